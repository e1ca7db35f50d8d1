// Backward pass of the gated token compressor (csa2_compress_bwd).
//
// Per entry and channel, with the softmax weights s_j over the window's rows (the block's m
// rows; overlapping form: and the previous block's m history rows) and E = sum s_j C_j:
//     g   = RoPE_-pos(dout)                      (with CSA2_W_ROPE)
//     dE  = r (g - E^ mean(E^ . g)), E^ = r E    (with CSA2_W_NORM, r the RMS factor; else g)
//     dC_j = s_j dE,   dZ_j = s_j dE (C_j - E),   dB_j = sum over entries of dZ_j
// The weights and E are computed again from the inputs; nothing of the forward is kept.
//
// Memory bound: every input row is read once and every gradient row written once.  A CTA takes
// a run of entries, a thread a few adjacent channels of each.  The usual windows (up to 8 rows:
// m = 1, 2, 3, 4, 8, and overlapping m = 1, 2, 3, 4) are compiled for their size: an entry's rows
// (contiguous stretches) come by bulk copies into a ring of stages in shared memory, several
// entries ahead of the arithmetic (loads into registers one entry ahead kept 41 KB an SM in
// flight, 3.7 TB/s over four streams of 131,072 tokens; now 448 us there, 5.4 TB/s), and stay in
// registers between the softmax and the gradients; other windows are read again (from the
// caches), m = 5, 6 and 7 among them.  The bias gradients are sums over all entries: each CTA sums its run in registers
// (long windows: in its slab of the workspace), and a last pass adds the CTAs' sums in order, so
// the results do not depend on timing.
#include <algorithm>
#include <atomic>

#include "attn_grad.cuh"
#include "sm100_ptx.cuh"

namespace {

// CTAs (of 152 SMs): what the registers keep resident at c = 512 -- windows of 1 or 2 rows 8 an SM; of 3 or 4
// rows 4; of 6 or 8 rows 2; of the general kernel 1,024 threads.
constexpr int CB_CTAS = 152 * 8;

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p);
template <>
__device__ __forceinline__ float4 ld4<float>(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 ld4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ void st4(T* p, const float (&v)[4]);
template <>
__device__ __forceinline__ void st4<float>(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void st4<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(ag_pack_bf16x2(v[0], v[1]), ag_pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void unpack4(const float4& u, float (&v)[4]) {
    v[0] = u.x;
    v[1] = u.y;
    v[2] = u.z;
    v[3] = u.w;
}

template <typename T>
struct CompressBwdArgs {
    const T *ca, *za, *cb, *zb, *prev_cb, *prev_zb;
    const float *ba, *bb;
    int64_t n_tokens, n_ent, entries;   // entries of one stream, of all
    int c, m;
    const int64_t* pos0;
    AgRope rope;
    unsigned flags;
    const void* dout;
    int dout_f32;
    int64_t dout_stride;
    T *dca, *dza, *dcb, *dzb, *dprev_cb, *dprev_zb;
    float* slab;              // [CTAs, (1 or 2) m, c] sums of dZ, or NULL (no bias gradient)
    int64_t run;              // entries per CTA
    int stages;               // usual windows: entries in the ring
    unsigned* st;
};

// Where the rows of an entry's window and their gradients are.
template <typename T>
struct Window {
    const T *c0, *z0, *c1, *z1;   // block rows, history rows (NULL: none)
    T *g0, *h0, *g1, *h1;         // their gradients (history: NULL = not wanted)
};

template <typename T>
__device__ __forceinline__ Window<T> window_of(const CompressBwdArgs<T>& a, int64_t b, int64_t i) {
    Window<T> w;
    const int64_t at = (b * a.n_tokens + i * a.m) * a.c, before = at - (int64_t)a.m * a.c;
    w.c0 = a.ca + at;
    w.z0 = a.za + at;
    w.g0 = a.dca + at;
    w.h0 = a.dza + at;
    w.c1 = w.z1 = nullptr;
    w.g1 = w.h1 = nullptr;
    if (a.cb) {
        if (i > 0) {
            w.c1 = a.cb + before;
            w.z1 = a.zb + before;
            w.g1 = a.dcb + before;
            w.h1 = a.dzb + before;
        } else if (a.prev_cb) {
            const int64_t p = b * (int64_t)a.m * a.c;
            w.c1 = a.prev_cb + p;
            w.z1 = a.prev_zb + p;
            if (a.dprev_cb) w.g1 = a.dprev_cb + p;
            if (a.dprev_zb) w.h1 = a.dprev_zb + p;
        }
    }
    return w;
}

// Sums of two values over the CTA's threads along x (at most 16 warps; others along y have the
// same values), two alternating buffers.
__device__ __forceinline__ void block_sum2(float& x, float& y, float2* red) {
    x = warp_sum(x);
    y = warp_sum(y);
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0 && threadIdx.y == 0) red[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    x = y = 0.0f;
    for (int i = 0; i < nw; ++i) {
        x += red[i].x;
        y += red[i].y;
    }
}

// CH adjacent channels from (to) memory.
__device__ __forceinline__ void get(const float* p, float (&x)[2]) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x;
    x[1] = v.y;
}
__device__ __forceinline__ void get(const float* p, float (&x)[4]) { unpack4(ld4<float>(p), x); }
__device__ __forceinline__ void get(const __nv_bfloat16* p, float (&x)[2]) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    x[0] = __uint_as_float(v << 16);
    x[1] = __uint_as_float(v & 0xFFFF0000u);
}
__device__ __forceinline__ void get(const __nv_bfloat16* p, float (&x)[4]) { unpack4(ld4<__nv_bfloat16>(p), x); }
__device__ __forceinline__ void st(float* p, const float (&v)[2]) { *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]); }
__device__ __forceinline__ void st(float* p, const float (&v)[4]) { st4<float>(p, v); }
__device__ __forceinline__ void st(__nv_bfloat16* p, const float (&v)[2]) {
    *reinterpret_cast<uint32_t*>(p) = ag_pack_bf16x2(v[0], v[1]);
}
__device__ __forceinline__ void st(__nv_bfloat16* p, const float (&v)[4]) { st4<__nv_bfloat16>(p, v); }

constexpr int CB_STAGES = 8;                     // most entries in the ring
constexpr long long CB_BUDGET = 1ll << 31;       // cycles a wait for a copy may take

// Bytes of one entry in the ring: gate and value rows of the block (and the history), dout's row.
__host__ __device__ inline size_t cb_stage_bytes(int rows, int c, size_t elem, size_t dout_elem) {
    return (size_t)c * (2 * rows * elem + dout_elem);
}

// Windows of M block rows and (OV) M history rows; CH channels a thread, c / CH threads.  The
// arithmetic, not the memory, came first here (about 350 instructions a thread and entry of two
// rows), so exponentials, the reciprocal and the square root are the hardware's approximations:
// the exponents are at most 0, where __expf is good to a few 2^-22 of every weight that counts.  In
// fp32, 4,096 tokens, the gradients are 0.8e-7 to 1.4e-7 off in norm (m = 2, 3, 4, 5 and 128); the
// same formulas in PyTorch's fp32 0.8e-7 to 2.0e-7.
template <typename T, int M, bool OV, int CH, bool BIAS>
__global__ void __launch_bounds__(1024 / CH, (OV ? 2 * M : M) <= 2 ? 4 : (CH == 4 ? 2 : 1)) compress_bwd_kernel(CompressBwdArgs<T> a) {
    using namespace sm100;
    constexpr int R = OV ? 2 * M : M;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 red[2][16];
    __shared__ uint64_t full[CB_STAGES];
    const int ch = CH * threadIdx.x, c = a.c;
    const float inv_c = 1.0f / (float)c;
    const int64_t e0 = (int64_t)blockIdx.x * a.run, e1 = min(a.entries, e0 + a.run);
    const uint32_t block_bytes = (uint32_t)(M * c * sizeof(T)), dout_bytes = (uint32_t)(c * (a.dout_f32 ? 4 : 2));
    const uint32_t stage_bytes = 2 * (R / M) * block_bytes + dout_bytes;
    if (threadIdx.x == 0) {
        for (int k = 0; k < a.stages; ++k) mbar_init(&full[k], 1);
        fence_mbar_init();
    }
    __syncthreads();
    // one thread copies an entry: [gates, values of the block][of the history][dout]
    auto fetch = [&](int64_t b, int64_t i, int stage) {
        const Window<T> w = window_of(a, b, i);
        uint8_t* dst = ring + (size_t)stage * stage_bytes;
        const bool hist = OV && w.c1;
        mbar_arrive_expect_tx(&full[stage], 2 * (hist ? 2 : 1) * block_bytes + dout_bytes);
        bulk_g2s(dst, w.z0, block_bytes, &full[stage]);
        bulk_g2s(dst + block_bytes, w.c0, block_bytes, &full[stage]);
        if (hist) {
            bulk_g2s(dst + 2 * block_bytes, w.z1, block_bytes, &full[stage]);
            bulk_g2s(dst + 3 * block_bytes, w.c1, block_bytes, &full[stage]);
        }
        bulk_g2s(dst + 2 * (R / M) * block_bytes,
                 reinterpret_cast<const uint8_t*>(a.dout) + (size_t)(b * a.dout_stride + i) * dout_bytes, dout_bytes,
                 &full[stage]);
    };
    auto step = [&](int64_t& b, int64_t& i) {
        if (++i == a.n_ent) {
            i = 0;
            ++b;
        }
    };
    int64_t b = e0 / a.n_ent, i = e0 - b * a.n_ent;
    int64_t fb = b, fi = i, fe = e0;             // the next entry to copy (thread 0)
    if (threadIdx.x == 0)
        for (int k = 0; k < a.stages && fe < e1; ++k, ++fe, step(fb, fi)) fetch(fb, fi, k);
    float db[BIAS ? R : 1][CH];
#pragma unroll
    for (int j = 0; j < (BIAS ? R : 1); ++j)
#pragma unroll
        for (int k = 0; k < CH; ++k) db[j][k] = 0.0f;
    int stage = 0;
    uint32_t par = 0;
    bool ok = true;
    // streams lie back to back, so entry e's block starts at row M e
    int64_t at = e0 * M * c + ch;
    for (int64_t e = e0; e < e1; ++e) {
        ok = mbar_wait(&full[stage], par, ok ? CB_BUDGET : 0, a.st) && ok;   // (a copy that never lands is flagged)
        const bool hist = OV && (i > 0 || a.prev_cb);
        const T* rows = reinterpret_cast<const T*>(ring + (size_t)stage * stage_bytes) + ch;
        float z[R][CH], v[R][CH], mx[CH], den[CH], E[CH], g[CH];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (!OV || j < M || hist) {
                const T* p = rows + (j < M ? j : j + M) * c;    // history gates follow the block's 2 M rows
                get(p, z[j]);
                get(p + M * c, v[j]);
            } else {
#pragma unroll
                for (int k = 0; k < CH; ++k) {                  // no history: logit -inf, value 0
                    z[j][k] = -INFINITY;
                    v[j][k] = 0.0f;
                }
            }
            const float* bias = j < M ? a.ba : a.bb;
            if (bias) {
                float x[CH];
                get(bias + (int64_t)(j < M ? j : j - M) * c + ch, x);
#pragma unroll
                for (int k = 0; k < CH; ++k) z[j][k] += x[k];
            }
        }
        const uint8_t* gd = ring + (size_t)stage * stage_bytes + 2 * (R / M) * block_bytes;
        if (a.dout_f32)
            get(reinterpret_cast<const float*>(gd) + ch, g);
        else
            get(reinterpret_cast<const __nv_bfloat16*>(gd) + ch, g);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            mx[k] = z[0][k];
#pragma unroll
            for (int j = 1; j < R; ++j) mx[k] = fmaxf(mx[k], z[j][k]);
            den[k] = E[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                z[j][k] = __expf(z[j][k] - mx[k]);
                den[k] += z[j][k];
                E[k] = fmaf(z[j][k], v[j][k], E[k]);
            }
            den[k] = __fdividef(1.0f, den[k]);
            E[k] *= den[k];
        }
        if ((a.flags & CSA2_W_ROPE) && ch >= c - 64) {
            const int64_t pos = (a.pos0 ? a.pos0[b] : 0) + (int64_t)M * i;
#pragma unroll
            for (int p = 0; p < CH / 2; ++p) {
                float cs, sn;
                ag_cos_sin(a.rope, pos, (ch + 2 * p - (c - 64)) >> 1, cs, sn);
                const float x0 = g[2 * p], x1 = g[2 * p + 1];
                g[2 * p] = x0 * cs + x1 * sn;
                g[2 * p + 1] = x1 * cs - x0 * sn;
            }
        }
        // (either barrier: every thread has read the stage)
        if (a.flags & CSA2_W_NORM) {
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                ss = fmaf(E[k], E[k], ss);
                dot = fmaf(E[k], g[k], dot);
            }
            block_sum2(ss, dot, red[(e - e0) & 1]);
            const float r = rsqrtf(fmaf(ss, inv_c, 1e-6f));
            const float d = dot * r * r * inv_c;
#pragma unroll
            for (int k = 0; k < CH; ++k) g[k] = r * fmaf(-E[k], d, g[k]);
        } else {
            __syncthreads();
        }
        if (threadIdx.x == 0 && fe < e1) {
            fetch(fb, fi, stage);
            ++fe;
            step(fb, fi);
        }
        if (++stage == a.stages) {
            stage = 0;
            par ^= 1;
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) g[k] *= den[k];             // dE / sum of the exponentials
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float dc[CH], dz[CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                dc[k] = z[j][k] * g[k];
                dz[k] = dc[k] * (v[j][k] - E[k]);
            }
            const int o = (j < M ? j : j - M) * c;
            if (!OV || j < M) {
                st(a.dca + at + o, dc);
                st(a.dza + at + o, dz);
            } else if (i > 0) {
                st(a.dcb + (at - M * c) + o, dc);
                st(a.dzb + (at - M * c) + o, dz);
            } else if (hist) {
                const int64_t p = b * (int64_t)M * c + o + ch;
                if (a.dprev_cb) st(a.dprev_cb + p, dc);
                if (a.dprev_zb) st(a.dprev_zb + p, dz);
            }
            if (BIAS && (!OV || j < M || hist))
#pragma unroll
                for (int k = 0; k < CH; ++k) db[BIAS ? j : 0][k] += dz[k];
        }
        if (OV && i == a.n_ent - 1) {
            // the stream's last block is nobody's history within this call
            float zero[CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) zero[k] = 0.0f;
            for (int j = 0; j < M; ++j) {
                st(a.dcb + at + (int64_t)j * c, zero);
                st(a.dzb + at + (int64_t)j * c, zero);
            }
        }
        step(b, i);
        at += M * c;
    }
    if (BIAS) {
        float* slab = a.slab + (int64_t)blockIdx.x * R * c + ch;
#pragma unroll
        for (int j = 0; j < (BIAS ? R : 1); ++j) st(slab + (int64_t)j * c, db[j]);
    }
}

// The usual windows; the bias sums' registers only where a bias gradient is wanted.  The ring
// takes half of an SM's shared memory for windows of 8 rows, a quarter for 4 rows (what the CTAs
// that the registers let in share evenly) and an eighth for the others: for 1 and 2 rows that is
// the even share as well, windows of 3 and 6 rows, of which 4 and 2 CTAs run, get less of it --
// three and two stages in bf16 at c = 512 -- and at least two stages everywhere.
template <typename T, int M, bool OV, int CH, bool BIAS>
csa2_status launch_window(const csa2_ctx* ctx, CompressBwdArgs<T> a, unsigned grid, cudaStream_t s) {
    constexpr int R = OV ? 2 * M : M;
    const size_t stage = cb_stage_bytes(R, a.c, sizeof(T), a.dout_f32 ? 4 : 2);
    const size_t share = (size_t)(226 * 1024) / (R == 8 ? 2 : (R == 4 ? 4 : 8)) - 2048;
    a.stages = (int)std::max<size_t>(2, std::min<size_t>(CB_STAGES, share / stage));
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (ctx->device & 63);
    auto kern = compress_bwd_kernel<T, M, OV, CH, BIAS>;
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        CSA2_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    kern<<<grid, (unsigned)(a.c / CH), (size_t)a.stages * stage, s>>>(a);
    return csa2_launch_status();
}

template <typename T, int M, bool OV, int CH>
csa2_status usual_window(const csa2_ctx* ctx, const CompressBwdArgs<T>& a, unsigned grid, cudaStream_t s) {
    return a.slab ? launch_window<T, M, OV, CH, true>(ctx, a, grid, s) : launch_window<T, M, OV, CH, false>(ctx, a, grid, s);
}

// Any m: four channels a thread; the window's rows are dealt out to groups of c / 4 threads, read once for the maximum, once for the sums and once for the gradients (the
// latter two from L2).  The groups' maxima and sums meet in shared memory, in group order.
// (512 entries of 128 rows, with biases: 197 us; one group for the whole window 431 us; groups of
// half as many threads, each with four rows' loads in flight, 256 us.)  __expf: the exponents are
// at most 0.
template <typename T>
__global__ void __launch_bounds__(1024) compress_bwd_any_kernel(CompressBwdArgs<T> a) {
    __shared__ float2 red[2][16];
    __shared__ __align__(16) float meet[2][4096];             // [group][channel]
    const int ch = 4 * threadIdx.x, grp = threadIdx.y, groups = blockDim.y;
    const int m = a.m, c = a.c;
    const int64_t e0 = (int64_t)blockIdx.x * a.run, e1 = min(a.entries, e0 + a.run);
    const int tables = a.cb ? 2 : 1;
    float* slab = a.slab ? a.slab + (int64_t)blockIdx.x * tables * m * c + ch : nullptr;
    // (the first entry writes the block rows' sums; one without history leaves the second table's as
    // they are, so those start at 0)
    if (slab)
        for (int j = e0 < e1 ? m + grp : grp; j < tables * m; j += groups) *reinterpret_cast<float4*>(slab + (int64_t)j * c) = make_float4(0.f, 0.f, 0.f, 0.f);
    auto mine = [&](int which, int g) { return reinterpret_cast<float4*>(&meet[which][g * c + ch]); };
    for (int64_t e = e0; e < e1; ++e) {
        const int64_t b = e / a.n_ent, i = e - b * a.n_ent;
        const Window<T> w = window_of(a, b, i);
        const int rows = w.c1 ? 2 * m : m;
        auto src = [&](const T* cur, const T* hist, int j) { return (j < m ? cur + (int64_t)j * c : hist + (int64_t)(j - m) * c) + ch; };
        auto logit = [&](int j, float (&z)[4]) {
            unpack4(ld4<T>(src(w.z0, w.z1, j)), z);
            const float* bias = j < m ? a.ba : a.bb;
            if (bias) {
                const float4 u = *reinterpret_cast<const float4*>(bias + (int64_t)(j < m ? j : j - m) * c + ch);
                z[0] += u.x;
                z[1] += u.y;
                z[2] += u.z;
                z[3] += u.w;
            }
        };
        float mx[4], den[4], E[4], g[4], t[4], x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mx[k] = -INFINITY;
            den[k] = E[k] = 0.0f;
        }
        const int64_t go = (b * a.dout_stride + i) * c + ch;
        unpack4(a.dout_f32 ? ld4<float>(reinterpret_cast<const float*>(a.dout) + go)
                           : ld4<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.dout) + go), g);
#pragma unroll 8
        for (int j = grp; j < rows; j += groups) {
            logit(j, t);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], t[k]);
        }
        *mine(0, grp) = make_float4(mx[0], mx[1], mx[2], mx[3]);
        __syncthreads();
        for (int o = 0; o < groups; ++o) {
            const float4 u = *mine(0, o);
            mx[0] = fmaxf(mx[0], u.x);
            mx[1] = fmaxf(mx[1], u.y);
            mx[2] = fmaxf(mx[2], u.z);
            mx[3] = fmaxf(mx[3], u.w);
        }
        __syncthreads();
#pragma unroll 4
        for (int j = grp; j < rows; j += groups) {
            logit(j, t);
            unpack4(ld4<T>(src(w.c0, w.c1, j)), x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float p = __expf(t[k] - mx[k]);
                den[k] += p;
                E[k] = fmaf(p, x[k], E[k]);
            }
        }
        *mine(0, grp) = make_float4(den[0], den[1], den[2], den[3]);
        *mine(1, grp) = make_float4(E[0], E[1], E[2], E[3]);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) den[k] = E[k] = 0.0f;
        for (int o = 0; o < groups; ++o) {
            const float4 u = *mine(0, o), v = *mine(1, o);
            den[0] += u.x;
            den[1] += u.y;
            den[2] += u.z;
            den[3] += u.w;
            E[0] += v.x;
            E[1] += v.y;
            E[2] += v.z;
            E[3] += v.w;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) E[k] /= den[k];
        if ((a.flags & CSA2_W_ROPE) && ch >= c - 64) {
            const int64_t pos = (a.pos0 ? a.pos0[b] : 0) + (int64_t)m * i;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float cs, sn;
                ag_cos_sin(a.rope, pos, (ch + 2 * p - (c - 64)) >> 1, cs, sn);
                const float x0 = g[2 * p], x1 = g[2 * p + 1];
                g[2 * p] = x0 * cs + x1 * sn;
                g[2 * p + 1] = x1 * cs - x0 * sn;
            }
        }
        if (a.flags & CSA2_W_NORM) {
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ss = fmaf(E[k], E[k], ss);
                dot = fmaf(E[k], g[k], dot);
            }
            block_sum2(ss, dot, red[(e - e0) & 1]);
            const float r = 1.0f / sqrtf(ss / (float)c + 1e-6f);
            const float d = dot * r * r / (float)c;
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] = r * fmaf(-E[k], d, g[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) den[k] = 1.0f / den[k];
#pragma unroll 4
        for (int j = grp; j < rows; j += groups) {
            logit(j, t);
            unpack4(ld4<T>(src(w.c0, w.c1, j)), x);
            float dc[4], dz[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                dc[k] = __expf(t[k] - mx[k]) * den[k] * g[k];
                dz[k] = dc[k] * (x[k] - E[k]);
            }
            const int64_t o = (int64_t)(j < m ? j : j - m) * c + ch;
            T* gc = j < m ? w.g0 : w.g1;
            T* gz = j < m ? w.h0 : w.h1;
            if (gc) st4<T>(gc + o, dc);
            if (gz) st4<T>(gz + o, dz);
            if (slab) {
                float4* d = reinterpret_cast<float4*>(slab + (int64_t)j * c);
                float4 u = e == e0 && j < m ? make_float4(0.f, 0.f, 0.f, 0.f) : *d;
                u.x += dz[0];
                u.y += dz[1];
                u.z += dz[2];
                u.w += dz[3];
                *d = u;
            }
        }
        if (a.cb && i == a.n_ent - 1) {
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            const int64_t at = (b * a.n_tokens + i * m) * c + ch;
            for (int j = grp; j < m; j += groups) {
                st4<T>(a.dcb + at + (int64_t)j * c, zero);
                st4<T>(a.dzb + at + (int64_t)j * c, zero);
            }
        }
    }
}

// db[x] = sum of the CTAs' slabs in a fixed order: warp w of a block takes slabs w, w + 32, ..
// of 32 adjacent columns, then the 32 sums are added.
__global__ void __launch_bounds__(1024) compress_bias_kernel(const float* slab, int ctas, int64_t cols, int64_t split,
                                                            float* dba, float* dbb) {
    __shared__ float red[32][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t x = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
#pragma unroll 8
    for (int i = w; i < ctas; i += 32) s += slab[(int64_t)i * cols + x];
    red[w][lane] = s;
    __syncthreads();
    if (w == 0) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][lane];
        float* d = x < split ? dba : dbb;
        if (d) d[x < split ? x : x - split] = s;
    }
}

// How a call is dealt out.  The launch and the workspace size both go by this: a CTA that sums bias
// gradients has a slab of its own.
struct Plan {
    bool usual;               // the window is compiled for its size
    int groups;               // groups of threads that share any other window's rows
    int64_t run, ctas;        // entries of a CTA; CTAs
};

Plan cb_plan(int64_t entries, int c, int m, bool overlap) {
    Plan p;
    const int rows = overlap ? 2 * m : m;
    p.usual = m <= 4 || (m == 8 && !overlap);
    // groups of the other windows: four rows each, as many as 1,024 threads take
    p.groups = p.usual ? 1 : std::max(1, std::min(4096 / c, rows / 4));
    const int64_t most = p.usual ? (rows > 4 ? CB_CTAS / 4 : rows > 2 ? CB_CTAS / 2 : CB_CTAS)
                                 : std::max(1, CB_CTAS * 128 / (c / 4 * p.groups));
    const int64_t run = (entries + most - 1) / most;
    p.ctas = run > 0 ? (entries + run - 1) / run : 0;
    p.run = p.ctas > 0 ? (entries + p.ctas - 1) / p.ctas : 0;
    return p;
}

struct CompressBwdCall {
    const void *ca, *za, *cb, *zb, *prev_cb, *prev_zb;
    const float *ba, *bb;
    int B;
    int64_t n_tokens;
    int c, m;
    const int64_t* pos0;
    float rope_base;
    unsigned flags;
    const void* dout;
    csa2_dtype dout_dt;
    int64_t dout_stride;
    void *dca, *dza, *dcb, *dzb, *dprev_cb, *dprev_zb;
    float *dba, *dbb, *slab;
};

template <typename T>
csa2_status cb_launch(const csa2_ctx* ctx, const CompressBwdCall& p, cudaStream_t s) {
    CompressBwdArgs<T> a;
    a.ca = reinterpret_cast<const T*>(p.ca);
    a.za = reinterpret_cast<const T*>(p.za);
    a.cb = reinterpret_cast<const T*>(p.cb);
    a.zb = reinterpret_cast<const T*>(p.zb);
    a.prev_cb = reinterpret_cast<const T*>(p.prev_cb);
    a.prev_zb = reinterpret_cast<const T*>(p.prev_zb);
    a.ba = p.ba;
    a.bb = p.bb;
    a.n_tokens = p.n_tokens;
    a.n_ent = p.n_tokens / p.m;
    a.entries = a.n_ent * p.B;
    a.c = p.c;
    a.m = p.m;
    a.pos0 = p.pos0;
    a.rope = make_ag_rope(p.rope_base);
    a.flags = p.flags;
    a.dout = p.dout;
    a.dout_f32 = p.dout_dt == CSA2_F32;
    a.dout_stride = p.dout_stride;
    a.dca = reinterpret_cast<T*>(p.dca);
    a.dza = reinterpret_cast<T*>(p.dza);
    a.dcb = reinterpret_cast<T*>(p.dcb);
    a.dzb = reinterpret_cast<T*>(p.dzb);
    a.dprev_cb = reinterpret_cast<T*>(p.dprev_cb);
    a.dprev_zb = reinterpret_cast<T*>(p.dprev_zb);
    a.slab = p.dba || p.dbb ? p.slab : nullptr;
    const Plan plan = cb_plan(a.entries, p.c, p.m, p.cb != nullptr);
    a.run = plan.run;
    a.stages = 0;
    a.st = ctx->status;
    csa2_status r = CSA2_OK;
    const unsigned grid = (unsigned)plan.ctas, c4 = (unsigned)(p.c / 4);
    if (!p.cb && p.m == 1)
        r = usual_window<T, 1, false, 4>(ctx, a, grid, s);
    else if (!p.cb && p.m == 2)
        r = usual_window<T, 2, false, 4>(ctx, a, grid, s);
    else if (!p.cb && p.m == 3)
        r = usual_window<T, 3, false, 4>(ctx, a, grid, s);
    else if (!p.cb && p.m == 4)
        r = usual_window<T, 4, false, 4>(ctx, a, grid, s);
    else if (!p.cb && p.m == 8)
        r = usual_window<T, 8, false, 2>(ctx, a, grid, s);
    else if (p.cb && p.m == 1)
        r = usual_window<T, 1, true, 4>(ctx, a, grid, s);
    else if (p.cb && p.m == 2)
        r = usual_window<T, 2, true, 4>(ctx, a, grid, s);
    else if (p.cb && p.m == 3)
        r = usual_window<T, 3, true, 2>(ctx, a, grid, s);
    else if (p.cb && p.m == 4)
        r = usual_window<T, 4, true, 2>(ctx, a, grid, s);
    else
        compress_bwd_any_kernel<T><<<grid, dim3(c4, (unsigned)plan.groups), 0, s>>>(a);
    if (r != CSA2_OK) return r;
    if (a.slab) {
        const int64_t split = (int64_t)p.m * p.c, cols = split * (p.cb ? 2 : 1);
        compress_bias_kernel<<<(unsigned)(cols / 32), 1024, 0, s>>>(a.slab, (int)plan.ctas, cols, split, p.dba, p.dbb);
    }
    return csa2_launch_status();
}

}  // namespace

extern "C" size_t csa2_compress_bwd_workspace_bytes(int B, int64_t n_tokens, int c, int m, int overlap) {
    if (B <= 0 || n_tokens <= 0 || c <= 0 || c % 128 || c > 1024 || m < 1) return 0;
    return (size_t)cb_plan(n_tokens / m * B, c, m, overlap != 0).ctas * (overlap ? 2 : 1) * m * c * sizeof(float);
}

extern "C" csa2_status csa2_compress_bwd(csa2_ctx* ctx, const void* ca, const void* za, const void* cb, const void* zb,
                                         csa2_dtype in_dt, const float* ba, const float* bb, const void* prev_cb,
                                         const void* prev_zb, int B, int64_t n_tokens, int c, int m,
                                         const int64_t* pos0, float rope_base, unsigned flags, const void* dout,
                                         csa2_dtype dout_dt, int64_t dout_seq_stride, void* dca, void* dza, void* dcb,
                                         void* dzb, void* dprev_cb, void* dprev_zb, float* dba, float* dbb, void* ws,
                                         size_t ws_bytes, void* stream) {
    if (!ctx || B < 0 || B > 65535 || n_tokens < 0 || m < 1 || c <= 0) return CSA2_ERR_INVALID_ARG;
    if (n_tokens % m || c % 128 || c > 1024) return CSA2_ERR_INVALID_ARG;
    if (!cb != !zb || !prev_cb != !prev_zb || (prev_cb && !cb)) return CSA2_ERR_INVALID_ARG;
    if (flags & ~(CSA2_W_NORM | CSA2_W_ROPE)) return CSA2_ERR_INVALID_ARG;
    if (in_dt != CSA2_F32 && in_dt != CSA2_BF16) return CSA2_ERR_UNSUPPORTED;
    if (dout_dt != CSA2_F32 && dout_dt != CSA2_BF16) return CSA2_ERR_UNSUPPORTED;
    if ((dbb || bb) && !cb) return CSA2_ERR_INVALID_ARG;
    if ((dprev_cb || dprev_zb) && !prev_cb) return CSA2_ERR_INVALID_ARG;
    for (const void* p : {ca, za, cb, zb, prev_cb, prev_zb, (const void*)ba, (const void*)bb, dout, (const void*)dca,
                          (const void*)dza, (const void*)dcb, (const void*)dzb, (const void*)dprev_cb,
                          (const void*)dprev_zb, (const void*)dba, (const void*)dbb, (const void*)ws})
        if (!aligned(p, 16)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(pos0, 8)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    if (B == 0 || n_tokens == 0) {
        const size_t e = in_dt == CSA2_F32 ? 4 : 2, prev = (size_t)B * m * c * e;
        if (prev && dprev_cb) CSA2_CHECK_CUDA(cudaMemsetAsync(dprev_cb, 0, prev, s));
        if (prev && dprev_zb) CSA2_CHECK_CUDA(cudaMemsetAsync(dprev_zb, 0, prev, s));
        if (dba) CSA2_CHECK_CUDA(cudaMemsetAsync(dba, 0, (size_t)m * c * 4, s));
        if (dbb) CSA2_CHECK_CUDA(cudaMemsetAsync(dbb, 0, (size_t)m * c * 4, s));
        return CSA2_OK;
    }
    if (!ca || !za || !dout || !dca || !dza || (cb && (!dcb || !dzb))) return CSA2_ERR_INVALID_ARG;
    if (dout_seq_stride < n_tokens / m && B > 1) return CSA2_ERR_INVALID_ARG;
    if ((dba || dbb) && (!ws || ws_bytes < csa2_compress_bwd_workspace_bytes(B, n_tokens, c, m, cb != nullptr)))
        return CSA2_ERR_INVALID_ARG;
    const CompressBwdCall p = {ca, za, cb, zb, prev_cb, prev_zb, ba, bb, B, n_tokens, c, m, pos0, rope_base, flags,
                               dout, dout_dt, dout_seq_stride, dca, dza, dcb, dzb, dprev_cb, dprev_zb, dba, dbb,
                               reinterpret_cast<float*>(ws)};
    return in_dt == CSA2_F32 ? cb_launch<float>(ctx, p, s) : cb_launch<__nv_bfloat16>(ctx, p, s);
}
