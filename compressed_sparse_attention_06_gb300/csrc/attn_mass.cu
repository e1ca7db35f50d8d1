// Accumulated attention weight of the cache entries (csa2_attn_mass), from the forward's lse:
//     w[b,q,j] = sum over heads of exp(q^_h . k^_j / sqrt(c) - lse_h)
//     acc[b, entry of slot j] += w[b,q,j]
//
// The sums into acc do not depend on the order the queries finish in.  With one query per
// sequence an entry gets one addend (the same index twice gives equal addends), added
// straight to acc.  With more, the addends of a call meet as 64-bit integers in units of
// 2^-39 in the workspace (integer sums are the same in any order; an addend is at most H
// and B*Q*H at most 2^24, so the sum stays below 2^63), and a last pass adds them to acc.  An
// addend's rounding, 2^-40, is below fp32's of a weight of 2^-16 and more, and above it of a
// smaller one; a weight below 2^-40 counts 0 here, where one query's is kept.
#include <algorithm>
#include <atomic>

#include "attn_mass.cuh"

namespace {

constexpr int MS_KC = 32;
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

__global__ void __launch_bounds__(256) mass_finish_kernel(const unsigned long long* fix, float* acc, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const unsigned long long v = fix[i];
    if (v) acc[i] += __ull2float_rn(v) * (1.0f / MASS_FIX_ONE);
}

// q^ of every (query, head) in fp32; a warp per head row.
template <typename TQ>
__global__ void __launch_bounds__(256) mass_prep_kernel(const TQ* q, const int64_t* q_pos, int64_t n_rows, int H,
                                                        AgRope rope, unsigned flags, float* qh) {
    __shared__ float cs[8][32], sn[8][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + w;
    if (r >= n_rows) return;
    ag_cos_sin(rope, q_pos[r / H], lane, cs[w][lane], sn[w][lane]);
    __syncwarp();
    float v[16];
    ag_load16<TQ>(q + r * AG_C + 16 * lane, v);
    if (flags & CSA2_QNORM) {
        const float f = ag_rms_factor(warp_sum(ag_sumsq16(v)));
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= f;
    }
    if (flags & CSA2_ROPE) ag_rope16(v, lane, cs[w], sn[w], 1.0f);
    ag_store16<float>(qh + r * AG_C + 16 * lane, v);
}

// CUDA-core path (fp32): a CTA per (32 slots, query), rows staged in fp32, a warp per four
// heads at a time, which share the loads of a row from shared memory (its port is the bound with
// one head a warp, the FMAs with four).
__global__ void __launch_bounds__(256, 2) mass_simt_kernel(MassArgs a) {
    extern __shared__ float smem[];
    float* xs = smem;                                         // [32][512]
    float* ws = xs + MS_KC * AG_C;                            // [8][32]
    int64_t* rid = reinterpret_cast<int64_t*>(ws + 8 * 32);   // [32]
    const int64_t bq = blockIdx.y;
    const int s0 = blockIdx.x * MS_KC, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    {
        // rows w, w + 8, w + 16, w + 24: all looked up, then all loaded
        int64_t mine = -1;
        const int sr = s0 + w + 8 * lane;
        if (lane < MS_KC / 8 && sr < a.slots.k) mine = slot_row(a.slots, bq, sr, true);
        float v[MS_KC / 8][16];
#pragma unroll
        for (int j = 0; j < MS_KC / 8; ++j) {
            const int64_t row = __shfl_sync(0xffffffffu, mine, j);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[j][i] = 0.0f;
            if (row >= 0) ag_load_row16(a.kv, a.kv_dt, row, lane, v[j]);
        }
#pragma unroll
        for (int j = 0; j < MS_KC / 8; ++j) {
            const int64_t row = __shfl_sync(0xffffffffu, mine, j);
            const float f = (a.flags & CSA2_KVNORM) ? ag_rms_factor(warp_sum(ag_sumsq16(v[j]))) : 1.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[j][i] *= f;
            ag_store16<float>(xs + (w + 8 * j) * AG_C + 16 * lane, v[j]);
            if (lane == 0) rid[w + 8 * j] = row;
        }
    }
    __syncthreads();
    const float isc = 1.0f / sqrtf((float)AG_C);
    float sum = 0.0f;
    for (int h0 = 4 * w; h0 < a.H; h0 += 32) {
        float qv[4][16], z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float* qr = a.qh + (bq * a.H + min(h0 + e, a.H - 1)) * AG_C;
#pragma unroll
            for (int i = 0; i < 16; ++i) qv[e][i] = qr[lane + 32 * i];
        }
#pragma unroll 1
        for (int j0 = 0; j0 < MS_KC; j0 += 8) {
            float d[4][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e][j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = xs[(j0 + j) * AG_C + lane + 32 * i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e][j] = fmaf(qv[e][i], x, d[e][j]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = ag_sums_of_8(d[e], lane);
                if ((lane & 24) == j0) z[e] = t * isc;       // slots j0 .. j0 + 7 belong to these lanes
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lse = h0 + e < a.H ? a.lse[bq * a.H + h0 + e] : -INFINITY;
            if (lse != -INFINITY) sum += expf(z[e] - lse);
        }
    }
    ws[w * 32 + lane] = sum;
    __syncthreads();
    if (w == 0 && s0 + lane < a.slots.k) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += ws[i * 32 + lane];
        const int64_t row = rid[lane];
        if (row < 0) t = 0.0f;
        if (a.weights) a.weights[bq * a.slots.k + s0 + lane] = t;
        if (a.acc && row >= 0) add_mass(a.acc, a.fix, row, t);
    }
}

constexpr size_t MS_SMEM = (size_t)MS_KC * AG_C * 4 + 8 * 32 * 4 + MS_KC * 8;

csa2_status simt_run(const csa2_ctx* ctx, const MassArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (ctx->device & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        CSA2_CHECK_CUDA(cudaFuncSetAttribute(mass_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MS_SMEM));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t heads = a.n_bq * a.H;
    const unsigned hb = (unsigned)((heads + 7) / 8);
    float* qh = const_cast<float*>(a.qh);
    if (a.q_dt == CSA2_F32)
        mass_prep_kernel<float><<<hb, 256, 0, s>>>(reinterpret_cast<const float*>(a.q), a.slots.q_pos, heads, a.H, a.rope,
                                                  a.flags, qh);
    else
        mass_prep_kernel<__nv_bfloat16><<<hb, 256, 0, s>>>(reinterpret_cast<const __nv_bfloat16*>(a.q), a.slots.q_pos,
                                                          heads, a.H, a.rope, a.flags, qh);
    mass_simt_kernel<<<dim3((unsigned)((a.slots.k + MS_KC - 1) / MS_KC), (unsigned)a.n_bq), 256, MS_SMEM, s>>>(a);
    return csa2_launch_status();
}

// RMS factor of every bf16 row; a warp per row.
__global__ void __launch_bounds__(256) mass_rinv_kernel(const __nv_bfloat16* kv, int64_t rows, float* rinv) {
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    float v[16];
    ag_load16<__nv_bfloat16>(kv + row * AG_C + 16 * lane, v);
    const float f = ag_rms_factor(warp_sum(ag_sumsq16(v)));
    if (lane == 0) rinv[row] = f;
}

struct MassLayout {
    size_t qh, fix, rinv, passes, total;
    bool table;
};

MassLayout mass_layout(csa2_dtype kv_dt, int B, int Q, int H, int k, int64_t N, bool want_acc) {
    MassLayout L;
    // A table of the rows' RMS factors (one pass over the cache) or the factors of each tile from its
    // rows: 33,792 entries, 512 slots, 32 queries (0.5 slots an entry) 33 and 32 us, 66 queries 31 and
    // 36, 132 queries 31 and 55, 1,056 queries 100 and 315.
    L.table = kv_dt == CSA2_BF16 && 2 * (int64_t)Q * k >= N;
    L.qh = 0;
    L.fix = kv_dt == CSA2_F32 ? align_up((size_t)B * Q * H * AG_C * 4, 256) : 0;
    L.rinv = align_up(L.fix + (want_acc && Q > 1 ? (size_t)B * N * 8 : 0), 256);
    L.passes = align_up(L.rinv + (L.table ? (size_t)B * N * 4 : 0), 256);
    L.total = L.passes + (H > 64 ? (size_t)B * Q * k * 4 : 0);
    return L;
}

}  // namespace

extern "C" size_t csa2_attn_mass_workspace_bytes(csa2_ctx* ctx, csa2_dtype kv_dt, int B, int Q, int H, int k,
                                                 int64_t N, int want_acc) {
    if (!ctx || B <= 0 || Q <= 0 || H < 1 || H > 128 || k < 0 || N < 0) return 0;
    return mass_layout(kv_dt, B, Q, H, k, N, want_acc != 0).total;
}

extern "C" csa2_status csa2_attn_mass(csa2_ctx* ctx, const void* q, csa2_dtype q_dt, const void* kv, csa2_dtype kv_dt,
                                      int64_t N, const int32_t* idx, const int64_t* n_visible, int k,
                                      const int64_t* q_pos, const float* lse, int B, int Q, int H, int c,
                                      float rope_base, unsigned flags, float* weights, float* acc, void* ws,
                                      size_t ws_bytes, void* stream) {
    if (!ctx || B < 0 || Q < 0 || N < 0 || k < 0 || k > (1 << 22) || (idx && k > 2048)) return CSA2_ERR_INVALID_ARG;
    if (H < 1 || H > 128) return CSA2_ERR_INVALID_ARG;
    if (c != AG_C) return CSA2_ERR_UNSUPPORTED;
    if (flags & ~CSA2_ATTN_DEFAULT) return CSA2_ERR_INVALID_ARG;
    if (q_dt != CSA2_F32 && q_dt != CSA2_BF16) return CSA2_ERR_UNSUPPORTED;
    if (kv_dt != CSA2_F32 && kv_dt != CSA2_BF16 && kv_dt != CSA2_FP4_E4M3x16) return CSA2_ERR_UNSUPPORTED;
    if ((int64_t)B * Q > 65535) return CSA2_ERR_UNSUPPORTED;
    if (!weights && !acc) return CSA2_ERR_INVALID_ARG;
    if (B == 0 || Q == 0 || k == 0) return CSA2_OK;
    if (!q || !kv || !q_pos || !lse || (!idx == !n_visible)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(ws, 16) || !aligned(lse, 4) || !aligned(q_pos, 8) ||
        !aligned(idx, 4) || !aligned(n_visible, 8) || !aligned(weights, 4) || !aligned(acc, 4))
        return CSA2_ERR_INVALID_ARG;
    const MassLayout L = mass_layout(kv_dt, B, Q, H, k, N, acc != nullptr);
    if (ws_bytes < L.total || (L.total > 0 && !ws)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    MassArgs a;
    a.slots = {idx, n_visible, q_pos, N, 1, 0, k, 0, Q, (int64_t)B * N, ctx->status};
    a.q = q;
    a.q_dt = q_dt;
    a.kv = kv;
    a.kv_dt = kv_dt;
    a.rope = make_ag_rope(rope_base);
    a.n_bq = (int64_t)B * Q;
    a.passes = H > 64 && !weights ? reinterpret_cast<float*>(base + L.passes) : nullptr;
    a.qh = reinterpret_cast<const float*>(base + L.qh);
    a.lse = lse;
    a.H = H;
    a.flags = flags;
    a.weights = weights;
    a.acc = acc;
    a.fix = acc && Q > 1 ? reinterpret_cast<unsigned long long*>(base + L.fix) : nullptr;
    if (a.fix) CSA2_CHECK_CUDA(cudaMemsetAsync(a.fix, 0, (size_t)B * N * 8, s));
    a.rinv = nullptr;
    if (L.table) {
        float* t = reinterpret_cast<float*>(base + L.rinv);
        const int64_t rows = (int64_t)B * N;
        if (rows > 0)
            mass_rinv_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(reinterpret_cast<const __nv_bfloat16*>(kv), rows, t);
        a.rinv = t;
    }
    const csa2_status r = kv_dt == CSA2_F32 ? simt_run(ctx, a, s) : mass_tc_run(ctx, a, s);
    if (r != CSA2_OK) return r;
    const int64_t n = (int64_t)B * N;
    if (a.fix && n > 0) {
        mass_finish_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a.fix, acc, n);
    }
    return csa2_launch_status();
}
