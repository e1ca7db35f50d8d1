// Trees of drafted tokens: the plan of a draft (positions and paths), the commit of an accepted
// path, and the attention of every node over its cache entries, the window ring and its own path
// (DSA-to-CSA/HCA page eqs. (18)-(19), (26), (27)) on the CUDA cores, in fp32 throughout.
//
// The CUDA-core attention takes 16 heads of one node a CTA, so that a row staged in shared memory
// serves 16 heads; its cost is shared-memory reads, so both products are tiled for few of them:
//   logits  a lane is a row, a warp an eighth of the 512 dims: 4 of the row's values (one 16-byte
//           read) meet 16 heads' (16 broadcasts) in 64 multiply-adds; the eight parts meet in
//           shared memory;
//   output  a thread holds 2 dims of 16 heads: one 8-byte read and 4 broadcasts, 32 multiply-adds.
// The softmax is online over chunks of 32 rows; few nodes split their rows over several CTAs,
// joined by log-sum-exp.  Measured: 2 x 13 nodes of 16 heads, 301 entries and a window of 100 each, 33 us of
// which 3.4 are their multiply-adds.  Large calls are bound by shared memory's port: 256 nodes of 64 heads over
// 640 slots keep it 78 % busy and the multiply-adds 35 %, and a warp waits for it 2.2 of the 7.1 cycles that an
// instruction takes (0.2 at barriers).  Calls that the tensor cores take too last 10 to 37 times as long here
// (8 x 32 nodes of 64 heads over FP4 pages 880 us, there 86; 4 x 64 over 4,096 bf16 entries 5,529 and 151).
#include <algorithm>

#include "csa2_internal.cuh"
#include "tree.cuh"
#include "tree_tc.cuh"

namespace {

constexpr int TS_C = 512;
constexpr int TS_HG = 16;                // heads of a CTA
constexpr int TS_KC = 32;                // rows of a chunk
constexpr int TS_THREADS = 256;
constexpr int TS_LD = TS_C + 4;          // floats between staged rows: lanes (rows) spread over all banks
constexpr int TS_MAX_T = 256;

// Positions and paths: a CTA a sequence, a thread a node; each walks up its parents in shared
// memory, once for its depth and once to write its path.
__global__ void __launch_bounds__(TS_MAX_T) tree_plan_kernel(const int32_t* parent, const int64_t* ctx_len, int T, int64_t* pos,
                                                             int16_t* path, unsigned* st) {
    __shared__ int par[TS_MAX_T];
    const int64_t b = blockIdx.x;
    const int i = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int64_t len = ctx_len[b];
    if (i < T) {
        int p = parent[b * T + i];
        if (p >= i || len < 0) {
            csa2_flag(st, CSA2_DEVBIT_RANGE);
            p = -2;
        }
        par[i] = max(p, -2);
    }
    int16_t* rows = path + b * T * T;
    for (int e = i; e < T * T; e += blockDim.x) rows[e] = -1;
    __syncthreads();
    if (i >= T) return;
    int depth = -1, j = i;
    while (j >= 0) {                     // parents are below their nodes, so this ends
        ++depth;
        j = par[j];
    }
    pos[b * T + i] = j == -1 ? len + depth : -1;
    if (j < -1) return;
    for (j = i; j >= 0; j = par[j]) rows[(int64_t)i * T + depth--] = (int16_t)j;
}

// The accepted path's rows into the ring: a CTA a (depth, sequence), 16 bytes a thread (no pieces: no ring, the
// lengths alone).
__global__ void __launch_bounds__(128) tree_commit_kernel(const uint4* draft, const int64_t* pos, const int16_t* path,
                                                          const int64_t* ctx_len, const int32_t* leaf, int T, int pieces, uint4* swa,
                                                          int64_t swa_cap, int64_t swa_pos0, int64_t* new_len, unsigned* st) {
    const int64_t b = blockIdx.y;
    const int d = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int l = leaf[b];
    const int64_t end = l >= 0 && l < T ? pos[b * T + l] : -1;
    if (d == 0 && threadIdx.x == 0) {    // the only reader of ctx_len, which new_len may be
        if (l >= T) csa2_flag(st, CSA2_DEVBIT_RANGE);
        if (new_len) new_len[b] = end >= 0 ? end + 1 : ctx_len[b];
    }
    const int j = end >= 0 ? path[(b * T + l) * (int64_t)T + d] : -1;
    if (j >= 0 && j < T && end - pos[b * T + j] < swa_cap) {
        const int64_t slot = ((pos[b * T + j] - swa_pos0) % swa_cap + swa_cap) % swa_cap;
        for (int u = threadIdx.x; u < pieces; u += blockDim.x)
            swa[(b * swa_cap + slot) * pieces + u] = draft[(b * T + j) * (int64_t)pieces + u];
    }
}

struct SimtArgs {
    TreeCall c;
    float* part;                         // [B*T, H, n_split, ATTN_PART] (n_split > 1)
    int n_split, spl;                    // splits of a node's rows, rows of a split (a multiple of TS_KC)
    unsigned* st;
};

__device__ __forceinline__ void load16f(const void* base, bool f32, int64_t row, int lane, float (&v)[16]) {
    if (f32) {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + row * TS_C + 16 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 u = p[i];
            v[4 * i] = u.x; v[4 * i + 1] = u.y; v[4 * i + 2] = u.z; v[4 * i + 3] = u.w;
        }
        return;
    }
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + row * TS_C + 16 * lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 u = p[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ void load16_fp4(const void* base, int64_t row, int lane, float (&v)[16]) {
    const uint8_t* r = reinterpret_cast<const uint8_t*>(base) + row * fp4_row_bytes(TS_C);
    const uint2 codes = *reinterpret_cast<const uint2*>(r + 8 * lane);
    const float s = e4m3_to_f32(r[TS_C / 2 + lane]);
    float lo[8], hi[8];
    e2m1x8_to_f32(codes.x, lo);
    e2m1x8_to_f32(codes.y, hi);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = lo[j] * s;
        v[8 + j] = hi[j] * s;
    }
}

__device__ __forceinline__ float sumsq16(const float (&v)[16]) {
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
    return warp_sum(ss);
}

// Factor of a warp's row whose squares sum to ss: its RMS factor, or 1 without a norm.  NaN for a row that
// holds a NaN or an infinity (without a norm its logits could all be -inf, which is no weight), or that is to be
// normalised and whose sum is not a number in fp32.
__device__ __forceinline__ float row_factor(const float (&v)[16], float ss, bool norm) {
    if (ss < INFINITY) return norm ? 1.0f / sqrtf(ss / (float)TS_C + 1e-6f) : 1.0f;
    bool bad = norm;
#pragma unroll
    for (int j = 0; j < 16; ++j) bad |= !(fabsf(v[j]) < INFINITY);
    return __any_sync(0xffffffffu, bad) ? __int_as_float(0x7FC00000) : 1.0f;
}

// A lane's 16 values to row[16 lane ..], its four pieces in an order that differs between the lanes of a
// store, so that eight lanes meet 32 banks (in the same order they would meet eight).
__device__ __forceinline__ void store16(float* row, int lane, const float (&v)[16]) {
    const bool one = lane & 2, two = lane & 4;
    float4 p[4], q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = one ? p[(j + 1) & 3] : p[j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4*>(row + 16 * lane)[(j + (lane >> 1)) & 3] = two ? q[(j + 2) & 3] : q[j];
}

struct SimtSmem {
    float xs[TS_KC * TS_LD];
    float qs[TS_HG * TS_C];
    float zp[7 * TS_HG * TS_KC];         // the parts of every logit that other warps than its head's have; cos, sin
    float ps[TS_KC * TS_HG];             // probability times RMS factor
    float rinv[TS_KC];                   // -1: no row
    float scale[TS_HG], m[TS_HG], l[TS_HG];
};
// Two CTAs an SM (1 KB each is the system's): with one, the rows' way from memory was in the open, and 256
// nodes of 64 heads over 640 slots took 1,292 us; with two 1,105, with the rows looked up a chunk ahead 975,
// stored without bank conflicts 908, with a look for infinities in them 923 (23 TFLOP/s).
static_assert(2 * (sizeof(SimtSmem) + 1024) <= 228 * 1024, "shared memory");

template <int KVK>                       // 0 fp32 rows, 1 bf16, 2 FP4
__global__ void __launch_bounds__(TS_THREADS, 2) tree_simt_kernel(const SimtArgs a) {
    extern __shared__ uint8_t raw[];
    SimtSmem& s = *reinterpret_cast<SimtSmem*>(raw);
    const TreeCall& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h0 = blockIdx.y * TS_HG;
    pdl_wait();
    pdl_trigger();
    const TreeNode n = tree_node(c.r, blockIdx.z);
    float *cs = s.zp, *sn = s.zp + 32;
    if (threadIdx.x < 32) ag_cos_sin(c.rope, n.t, lane, cs[lane], sn[lane]);
    if (threadIdx.x < TS_HG) {
        s.m[threadIdx.x] = -INFINITY;
        s.l[threadIdx.x] = 0.0f;
    }
    __syncthreads();
    // q^ of two heads a warp: normalised, rotated (dims 448 .. 511 are lanes 28 .. 31's, pairs in a lane)
    for (int h = warp; h < TS_HG; h += 8) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        if (h0 + h < c.H) load16f(c.q, c.q_dt == CSA2_F32, n.bt * c.H + h0 + h, lane, v);
        const float r = row_factor(v, sumsq16(v), c.flags & CSA2_QNORM);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= r;
        if ((c.flags & CSA2_ROPE) && lane >= 28) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = 8 * (lane - 28) + i;
                const float x0 = v[2 * i], x1 = v[2 * i + 1];
                v[2 * i] = x0 * cs[j] - x1 * sn[j];
                v[2 * i + 1] = x1 * cs[j] + x0 * sn[j];
            }
        }
        float4* dst = reinterpret_cast<float4*>(s.qs + h * TS_C + 16 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    float acc[TS_HG][2];
#pragma unroll
    for (int h = 0; h < TS_HG; ++h) acc[h][0] = acc[h][1] = 0.0f;
    const float inv_sqrt_c = 1.0f / sqrtf((float)TS_C);
    const int s_begin = blockIdx.x * a.spl, s_end = min(n.kq + n.nw, s_begin + a.spl);
    // lane i < 4 looks up the row of slot c0 + warp + 8 i, a chunk ahead
    int64_t at = -1;
    int what = TREE_NONE;
    const auto look_up = [&](int c0) {
        at = -1;
        what = TREE_NONE;
        if (lane < TS_KC / 8 && c0 + warp + 8 * lane < s_end) at = tree_slot(c.r, n, c0 + warp + 8 * lane, what, a.st, true);
    };
    look_up(s_begin);
    for (int c0 = s_begin; c0 < s_end; c0 += TS_KC) {
#pragma unroll
        for (int i0 = 0; i0 < TS_KC / 8; i0 += 2) {              // two rows at a time
            float v[2][16];
            int kind[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t row = __shfl_sync(0xffffffffu, at, i0 + i);
                kind[i] = __shfl_sync(0xffffffffu, what, i0 + i);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[i][j] = 0.0f;
                if (kind[i] == TREE_CACHE) {
                    if (KVK == 2) load16_fp4(c.kv, row, lane, v[i]);
                    else load16f(c.kv, KVK == 0, row, lane, v[i]);
                } else if (kind[i] != TREE_NONE) {
                    load16f(kind[i] == TREE_RING ? c.swa : c.draft, c.swa_dt == CSA2_F32, row, lane, v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = warp + 8 * (i0 + i);
                const float ss = sumsq16(v[i]);
                store16(s.xs + r * TS_LD, lane, v[i]);
                const float f = row_factor(v[i], ss, c.flags & CSA2_KVNORM);
                if (lane == 0) s.rinv[r] = kind[i] == TREE_NONE ? -1.0f : f;
            }
        }
        look_up(c0 + TS_KC);
        __syncthreads();
        // the softmax of heads `warp` and `warp + 8` is this warp's: its parts of their logits stay
        float mine[2] = {0.0f, 0.0f};
        {
            float z[TS_HG];
#pragma unroll
            for (int h = 0; h < TS_HG; ++h) z[h] = 0.0f;
            const float4* x = reinterpret_cast<const float4*>(s.xs + lane * TS_LD + 64 * warp);
            const float4* q = reinterpret_cast<const float4*>(s.qs + 64 * warp);
#pragma unroll 2
            for (int i = 0; i < 16; ++i) {
                const float4 xv = x[i];
#pragma unroll
                for (int h = 0; h < TS_HG; ++h) {
                    const float4 qv = q[h * (TS_C / 4) + i];
                    z[h] = fmaf(xv.x, qv.x, fmaf(xv.y, qv.y, fmaf(xv.z, qv.z, fmaf(xv.w, qv.w, z[h]))));
                }
            }
#pragma unroll
            for (int h = 0; h < TS_HG; ++h) {
                const int o = h & 7;
                if (o == warp) mine[h >> 3] = z[h];
                else s.zp[((warp < o ? warp : warp - 1) * TS_HG + h) * TS_KC + lane] = z[h];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = warp + 8 * i;
            float z = mine[i];
#pragma unroll
            for (int w = 0; w < 7; ++w) z += s.zp[(w * TS_HG + h) * TS_KC + lane];
            const float rinv = s.rinv[lane];
            z = rinv == -1.0f ? -INFINITY : z * rinv * inv_sqrt_c;
            // (a NaN, which fmaxf drops, counts as some logit: the row has one, whose sum is NaN)
            const float m_old = s.m[h], m_new = fmaxf(m_old, warp_max(z == z ? z : 0.0f));
            const float sc = m_new == -INFINITY ? 1.0f : expf(m_old - m_new);
            const float p = z == -INFINITY ? 0.0f : expf(z - m_new);
            const float l = warp_sum(p);
            s.ps[lane * TS_HG + h] = p * rinv;
            __syncwarp();
            if (lane == 0) {
                s.scale[h] = sc;
                s.m[h] = m_new;
                s.l[h] = s.l[h] * sc + l;
            }
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < TS_HG; ++h) {
            const float sc = s.scale[h];
            acc[h][0] *= sc;
            acc[h][1] *= sc;
        }
        const int here = min(TS_KC, s_end - c0);
#pragma unroll 4
        for (int r = 0; r < here; ++r) {
            const float2 x = *reinterpret_cast<const float2*>(s.xs + r * TS_LD + 2 * threadIdx.x);
#pragma unroll
            for (int h4 = 0; h4 < TS_HG / 4; ++h4) {
                const float4 p = *reinterpret_cast<const float4*>(s.ps + r * TS_HG + 4 * h4);
                const float pv[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[4 * h4 + j][0] = fmaf(pv[j], x.x, acc[4 * h4 + j][0]);
                    acc[4 * h4 + j][1] = fmaf(pv[j], x.y, acc[4 * h4 + j][1]);
                }
            }
        }
        __syncthreads();
    }
    if (a.n_split > 1) {
#pragma unroll
        for (int h = 0; h < TS_HG; ++h) {
            if (h0 + h >= c.H) break;
            float* part = a.part + ((n.bt * c.H + h0 + h) * (int64_t)a.n_split + blockIdx.x) * ATTN_PART;
            if (threadIdx.x == 0) {
                part[0] = s.m[h];
                part[1] = s.l[h];
            }
            *reinterpret_cast<float2*>(part + ATTN_PART_O + 2 * threadIdx.x) = make_float2(acc[h][0], acc[h][1]);
        }
        return;
    }
    if (threadIdx.x < 32) ag_cos_sin(c.rope, n.t, lane, cs[lane], sn[lane]);
    __syncthreads();
    const int j = (int)threadIdx.x - 224;            // this thread's pair of the last 64 dims
#pragma unroll
    for (int h = 0; h < TS_HG; ++h) {
        if (h0 + h >= c.H) break;
        const float zs = c.sink ? c.sink[h0 + h] : -INFINITY;
        const float m = s.m[h], top = fmaxf(m, zs);
        float den = 0.0f, sc = 0.0f;
        if (top != -INFINITY) {
            const float e = m == -INFINITY ? 0.0f : expf(m - top);
            den = s.l[h] * e + (zs == -INFINITY ? 0.0f : expf(zs - top));
            sc = e / den;
        }
        float x0 = acc[h][0] * sc, x1 = acc[h][1] * sc;
        if ((c.flags & CSA2_ROPE) && j >= 0) {
            const float y0 = x0 * cs[j] + x1 * sn[j];
            x1 = x1 * cs[j] - x0 * sn[j];
            x0 = y0;
        }
        const int64_t row = n.bt * c.H + h0 + h;
        if (c.out_dt == CSA2_F32)
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(c.out) + row * TS_C + 2 * threadIdx.x) = make_float2(x0, x1);
        else
            *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(c.out) + row * TS_C + 2 * threadIdx.x) =
                __floats2bfloat162_rn(x0, x1);
        if (c.lse && threadIdx.x == 0) c.lse[row] = top == -INFINITY ? -INFINITY : top + logf(den);
    }
}

// The splits of one (node, head), a warp each.
template <typename TO>
__global__ void __launch_bounds__(256) tree_combine_kernel(const SimtArgs a, int64_t rows) {
    __shared__ float cs[8][32], sn[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + warp;
    pdl_wait();
    pdl_trigger();
    if (r >= rows) return;
    const bool rope = a.c.flags & CSA2_ROPE;
    if (rope) ag_cos_sin(a.c.rope, a.c.r.pos[r / a.c.H], lane, cs[warp][lane], sn[warp][lane]);
    __syncwarp();
    const float sum = attn_combine_row<TO>(a.part + r * (int64_t)a.n_split * ATTN_PART, a.n_split,
                                           a.c.sink ? a.c.sink[r % a.c.H] : -INFINITY, rope ? cs[warp] : nullptr, sn[warp],
                                           reinterpret_cast<TO*>(a.c.out) + r * TS_C, a.c.lse ? a.c.lse + r : nullptr);
    if (sum != sum && a.c.lse && lane == 0) a.c.lse[r] = sum;         // NaN, as the outputs
}

// Splits that give every SM two CTAs, of 32 rows at least.
void simt_splits(const csa2_ctx* ctx, int64_t n_bt, int H, int64_t slots, int& n_split, int& spl) {
    const int64_t groups = n_bt * ((H + TS_HG - 1) / TS_HG), chunks = std::max<int64_t>(1, (slots + TS_KC - 1) / TS_KC);
    const int64_t want = std::min(chunks, std::max<int64_t>(1, 2 * (int64_t)ctx->num_sms / groups));
    const int64_t per = (chunks + want - 1) / want;
    spl = (int)(per * TS_KC);
    n_split = (int)((chunks + per - 1) / per);
}

size_t simt_ws(const csa2_ctx* ctx, int64_t n_bt, int H, int64_t slots) {
    int ns, spl;
    simt_splits(ctx, n_bt, H, slots, ns, spl);
    return ns > 1 ? (size_t)n_bt * H * ns * ATTN_PART * sizeof(float) : 0;
}

template <int KVK>
csa2_status launch_simt(const SimtArgs& a, cudaStream_t s) {
    auto kern = tree_simt_kernel<KVK>;
    CSA2_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SimtSmem)));
    const int64_t n_bt = (int64_t)a.c.B * a.c.r.T;
    csa2_status r = launch_pdl(kern, dim3((unsigned)a.n_split, (unsigned)((a.c.H + TS_HG - 1) / TS_HG), (unsigned)n_bt), dim3(TS_THREADS),
                               sizeof(SimtSmem), s, a);
    if (r == CSA2_OK && a.n_split > 1) {
        const int64_t rows = n_bt * a.c.H;
        const dim3 grid((unsigned)((rows + 7) / 8));
        r = a.c.out_dt == CSA2_F32 ? launch_pdl(tree_combine_kernel<float>, grid, dim3(256), 0, s, a, rows)
                                   : launch_pdl(tree_combine_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a, rows);
    }
    return r != CSA2_OK ? r : csa2_launch_status();
}

}  // namespace

extern "C" csa2_status csa2_tree_plan(csa2_ctx* ctx, const int32_t* parent, const int64_t* ctx_len, int B, int T,
                                      int64_t* pos, int16_t* path, void* stream) {
    if (!ctx || B < 0 || T < 1 || T > TS_MAX_T) return CSA2_ERR_INVALID_ARG;
    if (B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0) return CSA2_OK;
    if (!parent || !ctx_len || !pos || !path || !aligned(parent, 4) || !aligned(ctx_len, 8) || !aligned(pos, 8) || !aligned(path, 2))
        return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    const csa2_status l = launch_pdl(tree_plan_kernel, dim3((unsigned)B), dim3((unsigned)((T + 31) / 32 * 32)), 0, as_stream(stream), parent,
                                     ctx_len, T, pos, path, ctx->status);
    return l != CSA2_OK ? l : csa2_launch_status();
}

extern "C" csa2_status csa2_tree_commit(csa2_ctx* ctx, const void* draft, csa2_dtype dt, const int64_t* pos,
                                        const int16_t* path, const int64_t* ctx_len, const int32_t* leaf, int B, int T, int c,
                                        void* swa, int64_t swa_cap, int64_t swa_pos0, int64_t* new_len, void* stream) {
    const bool ring = draft || swa;                  // neither: the lengths alone
    if (!ctx || B < 0 || T < 1 || T > TS_MAX_T || (ring && swa_cap < 1)) return CSA2_ERR_INVALID_ARG;
    if (c != TS_C || (dt != CSA2_F32 && dt != CSA2_BF16) || B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0) return CSA2_OK;
    if (!pos || !path || !ctx_len || !leaf || (ring ? !draft || !swa : !new_len)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(draft, 16) || !aligned(swa, 16) || !aligned(pos, 8) || !aligned(path, 2) || !aligned(ctx_len, 8) ||
        !aligned(leaf, 4) || !aligned(new_len, 8))
        return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    const csa2_status l = launch_pdl(tree_commit_kernel, dim3(ring ? (unsigned)T : 1u, (unsigned)B), dim3(128), 0, as_stream(stream),
                                     reinterpret_cast<const uint4*>(draft), pos, path, ctx_len, leaf, T,
                                     ring ? c * (dt == CSA2_F32 ? 4 : 2) / 16 : 0, reinterpret_cast<uint4*>(swa), ring ? swa_cap : 1,
                                     swa_pos0, new_len, ctx->status);
    return l != CSA2_OK ? l : csa2_launch_status();
}

extern "C" size_t csa2_tree_attn_workspace_bytes(csa2_ctx* ctx, csa2_dtype q_dt, csa2_dtype kv_dt, csa2_dtype swa_dt, int B,
                                                 int T, int H, int k, int window, int dense, unsigned flags) {
    if (!ctx || B <= 0 || T <= 0 || H <= 0 || H > 128 || k < 0 || window < 0) return 0;
    if (tree_tc_applies(q_dt, kv_dt, swa_dt, flags)) return tree_tc_ws_bytes(ctx, B, T, H, k, window, dense != 0);
    return simt_ws(ctx, (int64_t)B * T, H, (int64_t)k + window);
}

extern "C" csa2_status csa2_tree_attn(csa2_ctx* ctx, const void* q, csa2_dtype q_dt, const void* kv, csa2_dtype kv_dt, int64_t N,
                                      const int32_t* table, int max_pages, int page, const int32_t* idx,
                                      const int64_t* n_visible, int k, const void* swa, csa2_dtype swa_dt, int64_t swa_cap,
                                      int64_t swa_pos0, int window, const void* draft, const int64_t* pos, const int16_t* path,
                                      const int64_t* ctx_len, const float* sink, int B, int T, int H, int c, float rope_base,
                                      unsigned flags, void* out, csa2_dtype out_dt, float* lse, void* ws, size_t ws_bytes,
                                      void* stream) {
    if (!ctx || B < 0 || T < 1 || T > TS_MAX_T || N < 0 || k < 0 || window < 0 || window > 1024 || H < 1 || H > 128)
        return CSA2_ERR_INVALID_ARG;
    if (idx && n_visible) return CSA2_ERR_INVALID_ARG;
    if (k > (n_visible ? 1 << 22 : 2048)) return CSA2_ERR_INVALID_ARG;
    if (flags & ~(unsigned)(CSA2_QNORM | CSA2_KVNORM | CSA2_ROPE)) return CSA2_ERR_INVALID_ARG;
    if (table && (page < 1 || page > 65536 || max_pages < 0 || N % page != 0)) return CSA2_ERR_INVALID_ARG;
    if (c != TS_C) return CSA2_ERR_UNSUPPORTED;
    if ((q_dt != CSA2_F32 && q_dt != CSA2_BF16) || (out_dt != CSA2_F32 && out_dt != CSA2_BF16) ||
        (swa_dt != CSA2_F32 && swa_dt != CSA2_BF16) || (kv_dt != CSA2_F32 && kv_dt != CSA2_BF16 && kv_dt != CSA2_FP4_E4M3x16))
        return CSA2_ERR_UNSUPPORTED;
    if ((int64_t)B * T > 65535 || N > 0x7FFFFFFF || (!table && B * N > 0x7FFFFFFF) || swa_cap < 0 || B * swa_cap > 0x7FFFFFFF)
        return CSA2_ERR_UNSUPPORTED;
    if (B == 0) return CSA2_OK;
    if (!q || !pos || !path || !ctx_len || !out) return CSA2_ERR_INVALID_ARG;
    if (k > 0 && ((!idx && !n_visible) || (N > 0 && !kv))) return CSA2_ERR_INVALID_ARG;
    if (window > 0 && (!swa || !draft || swa_cap < window)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(swa, 16) || !aligned(draft, 16) || !aligned(out, 16) || !aligned(ws, 16) ||
        !aligned(pos, 8) || !aligned(path, 2) || !aligned(ctx_len, 8) || !aligned(idx, 4) || !aligned(n_visible, 8) ||
        !aligned(table, 4) || !aligned(sink, 4) || !aligned(lse, 4))
        return CSA2_ERR_INVALID_ARG;
    const size_t need = csa2_tree_attn_workspace_bytes(ctx, q_dt, kv_dt, swa_dt, B, T, H, k, window, n_visible != nullptr, flags);
    if (need > 0 && (!ws || ws_bytes < need)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    SimtArgs a;
    TreeCall& t = a.c;
    t.r = {table, N, max_pages, page, idx, n_visible, k, window > 0 ? swa_cap : 1, swa_pos0, window, pos, path, ctx_len, T};
    t.q = q;
    t.q_dt = q_dt;
    t.kv = kv;
    t.kv_dt = kv_dt;
    t.swa = swa;
    t.draft = draft;
    t.swa_dt = swa_dt;
    t.sink = sink;
    t.B = B;
    t.H = H;
    t.rope = make_ag_rope(rope_base);
    t.flags = flags;
    t.out = out;
    t.out_dt = out_dt;
    t.lse = lse;
    if (tree_tc_applies(q_dt, kv_dt, swa_dt, flags)) return tree_tc_run(ctx, t, ws, s);
    a.part = reinterpret_cast<float*>(ws);
    a.st = ctx->status;
    simt_splits(ctx, (int64_t)B * T, H, (int64_t)k + window, a.n_split, a.spl);
    if (kv_dt == CSA2_F32) return launch_simt<0>(a, s);
    if (kv_dt == CSA2_BF16) return launch_simt<1>(a, s);
    return launch_simt<2>(a, s);
}
