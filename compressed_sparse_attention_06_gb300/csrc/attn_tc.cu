// Shared-KV MQA over the selected entries plus the sliding window on the tcgen05
// tensor cores (DSA-to-CSA/HCA page eqs. (18)-(19) and (27); CSA2 page «保留了 CSA
// 的骨架»): the same RMS-normalised row is key and value for all heads, the query
// is RMS-normalised and rotated by RoPE_t on its last 64 dims, the output is
// rotated back by RoPE_-t, and the sink adds e^{z'_h} to the denominator only.
//
// Work item = (query, range of 128-slot key tiles).  Per tile, two MMAs:
//   S^T[128 slots x 64 heads]  = X[128 x 512] . Qhat[64 x 512]^T       (K-major A, B)
//   O^T[512 dims x 64 heads]  += X^T[512 x 128] . P'[64 x 128]^T       (MN-major A, B)
// X is the tile of raw key rows (bf16; FP4 rows dequantised exactly into bf16),
// gathered once into shared memory in the 128-byte-swizzled layout and read by both
// MMAs; S and O live in tensor memory.  Each row's RMS factor r_s is applied to the
// logits and folded into the probabilities (P' = p r_s), so X is never rescaled.
//
// Softmax without a running maximum.  With both RMSNorms on, |qhat| and |xhat| are
// at most sqrt(512), so every logit qhat.xhat / sqrt(512) lies in [-22.7, 22.7].
// p = exp(logit - 24) is therefore in (e^-47, 1]: no overflow, no underflow in f32
// or bf16, and O accumulates across tiles without rescaling.  The denominator is the
// f32 sum of the unrounded p.  With several key splits each writes (24, sum,
// unnormalised O) and the log-sum-exp combine merges them.
//
// Precision: the normalised query and P' are rounded to bf16 for the MMA (fp32
// accumulation); key rows are exact.
//
// Warp roles (448 threads, one CTA per SM, persistent over work items):
//   warp 0      producer: the query image of each work item (one 64 KB bulk copy)
//   warp 1      MMA issuer; owns the tensor memory (O^T: columns 0-255, S^T: 256-319)
//   warps 2-5   softmax: one thread per slot; then the output epilogue, one thread per
//               output dim
//   warps 6-13  loaders, two groups of four warps with one thread per slot each, group
//               0 producing the 128-dim blocks {1, 0} ({0, 1} for bf16 tiles) and group
//               1 the blocks {2, 3}: bf16 rows gathered with 16-byte cp.async straight
//               into the swizzled tile (one commit group per block, so the next tile
//               streams in while the current PV finishes), FP4 rows staged in shared
//               memory and dequantised exactly into bf16, zero rows for empty slots,
//               and each row's RMS factor (group 0; read from a table precomputed once
//               per call when rows are gathered many times over, as in prefill)
// Every wait is bounded; a wait that expires flags a timeout and the roles wind down.
#include <algorithm>
#include <cstring>

#include "attn_tc.cuh"
#include "fp4_tile.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace sm100;

constexpr int TC_C = 512;
constexpr int TC_H = 64;
constexpr int TC_TILE = 128;
constexpr int TC_THREADS = 448;
constexpr float TC_SHIFT = 24.0f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int QIMG_BYTES = TC_H * TC_C * 2;     // 64 KB: 8 chunks of 64 rows x 128 B
constexpr int CHUNK_Q = TC_H * 128;
constexpr int CHUNK_K = TC_TILE * 128;          // 16 KB: 128 rows x 64 dims
constexpr int PART = ATTN_PART;
constexpr uint32_t DS_COL = 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr long long WAIT_BUDGET = 1ll << 31;
constexpr unsigned FULL = 0xffffffffu;

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + QIMG_BYTES;
constexpr int OFF_P = OFF_K + 8 * CHUNK_K;
constexpr int OFF_RINV = OFF_P + TC_TILE * 128;
constexpr int OFF_LW = OFF_RINV + TC_TILE * 4;
constexpr int OFF_SC = OFF_LW + 4 * TC_H * 4;        // [4 warps][64] output scale per head
constexpr int OFF_SCL = OFF_SC + 4 * TC_H * 4;       // [2 items][64] scales for the loader warps
constexpr int OFF_BAR = OFF_SCL + 2 * TC_H * 4;
constexpr int N_BAR = 20;
constexpr int OFF_TMEMPTR = OFF_BAR + N_BAR * 8;
constexpr int OFF_STGSC = (OFF_TMEMPTR + 16 + 15) / 16 * 16;   // [128 rows][32 B] staged FP4 scales
constexpr int OFF_SS = OFF_STGSC + TC_TILE * 32;              // [128] loader group 1's sums of squares
constexpr int SMEM_BYTES = OFF_SS + TC_TILE * 4 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

struct TcArgs {
    const uint8_t* qimg;          // [B*Q] query images
    const void* kv;               // bf16 [B, N, 512] or FP4 [B, N, 288]
    const uint8_t* swa;           // bf16 [B, swa_cap, 512]
    const float* rinv_kv;         // precomputed RMS factors of the bf16 rows, or NULL
    const float* rinv_swa;        // precomputed RMS factors of the window rows, or NULL
    int64_t N;
    const int32_t* idx;           // [B*Q, k]
    int k;
    const int64_t* dense_nv;      // dense mode: entries 0 .. dense_nv[bq]-1 (idx unused)
    int64_t swa_cap, swa_pos0;
    int window;
    const int64_t* q_pos;
    const float* sink;
    int Q, H;
    int Hs;                       // heads per query in out / lse (out, lse, sink start at this pass's head 0)
    RopeTable rope;
    unsigned flags;
    void* out;
    float* lse;
    float* part;                  // [B*Q, H, n_split, PART] when n_split > 1
    const float* rope_cs;         // [B*Q, 64]: cos, sin of the 32 RoPE angles at the query position
    int n_split, tps;             // splits per query, tiles per split
    int n_pass;                   // head passes of H (<= 64) heads in this launch (out, lse, sink
                                  // and q are then not offset: pass p takes heads 64p ..)
    int64_t n_bq;                 // queries (B * Q)
    int64_t items;
    unsigned int* st;
    long long budget;
    int stall;                    // test hook: the query-image producer issues nothing
    int cluster;                  // 1: a query's splits are one thread-block cluster (one item per
                                  // CTA) and merge their partials at the end of the kernel
};

struct ItemInfo {
    int64_t bq, b, t;
    int64_t v;                            // pass * n_bq + bq: the query image, the partials' block
    int64_t prow;                         // first row of this item's heads in the partials
    int pass, h0, H;                      // head pass, its first head, its heads
    int split, nw, kq, n_slots, t0, nt;   // kq: cache slots of this query, then nw window slots
};

__device__ __forceinline__ ItemInfo item_info(const TcArgs& a, int64_t item) {
    ItemInfo r;
    r.v = item / a.n_split;
    r.split = (int)(item % a.n_split);
    r.pass = (int)(r.v / a.n_bq);
    r.bq = r.v % a.n_bq;
    r.h0 = r.pass * TC_H;
    r.H = min(a.H, a.Hs - r.h0);
    r.prow = (int64_t)r.pass * TC_H * a.n_bq + r.bq * r.H;
    r.b = r.bq / a.Q;
    r.t = a.q_pos[r.bq];
    r.nw = (int)max((int64_t)0, min((int64_t)a.window, r.t + 1));
    r.kq = a.dense_nv ? (int)max((int64_t)0, min((int64_t)a.k, a.dense_nv[r.bq])) : a.k;
    r.n_slots = r.kq + r.nw;
    const int n_tiles = (r.n_slots + TC_TILE - 1) / TC_TILE;
    r.t0 = r.split * a.tps;
    r.nt = max(0, min(n_tiles, r.t0 + a.tps) - r.t0);
    return r;
}

// Source of a key slot: kind 0 = empty, 1 = selected cache row, 2 = window row.
struct SlotSrc {
    int kind;
    int64_t row;
};

__device__ __forceinline__ SlotSrc slot_source(const TcArgs& a, const ItemInfo& it, int slot, bool flag_range) {
    SlotSrc r;
    r.kind = 0;
    r.row = 0;
    if (slot >= it.n_slots) return r;
    if (slot < it.kq) {
        const int32_t id = a.dense_nv ? slot : a.idx[it.bq * a.k + slot];
        if (id >= 0) {
            if (id < a.N) {
                r.kind = 1;
                r.row = it.b * a.N + id;
            } else if (flag_range) {
                csa2_flag(a.st, CSA2_DEVBIT_RANGE);
            }
        }
    } else {
        const int64_t p = it.t - it.nw + 1 + (slot - it.kq);
        r.kind = 2;
        r.row = it.b * a.swa_cap + (((p - a.swa_pos0) % a.swa_cap) + a.swa_cap) % a.swa_cap;
    }
    return r;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void bf16x8_sumsq(const uint4& v, float& ss) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
        ss = fmaf(a, a, ss);
        ss = fmaf(b, b, ss);
    }
}

// Staged FP4 codes: 16-byte piece i (0..15) of row r, XOR-swizzled so that the eight
// rows a quarter-warp touches at once sit in eight different bank groups.
__device__ __forceinline__ uint32_t stg_code_offset(int r, int i) {
    return (uint32_t)r * 256u + ((uint32_t)(i ^ (r & 7)) << 4);
}

template <typename TQ>
__device__ __forceinline__ void load16(const TQ* src, float (&v)[16]);
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* src, float (&v)[16]) {
    const uint4* p = reinterpret_cast<const uint4*>(src);
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
template <>
__device__ __forceinline__ void load16<float>(const float* src, float (&v)[16]) {
    const float4* p = reinterpret_cast<const float4*>(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = p[i];
        v[4 * i] = u.x;
        v[4 * i + 1] = u.y;
        v[4 * i + 2] = u.z;
        v[4 * i + 3] = u.w;
    }
}

// Normalised, rotated query of every (query, head) as the bf16 image of the MMA's
// B operand: 8 chunks of [64 heads x 64 dims], 128-byte swizzled; heads >= H are 0.
// A CTA per (8 heads, query), a warp per head, 16 dims per lane.
template <typename TQ>
__global__ void __launch_bounds__(256) attn_qprep_kernel(const TQ* q, const int64_t* q_pos, int H, int Hs,
                                                         RopeTable rope, unsigned flags, uint8_t* qimg,
                                                         float* rope_cs) {
    __shared__ float cs[32], sn[32];
    pdl_wait();
    pdl_trigger();
    const int64_t bq = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the head row is loaded first, so its load and the position's overlap
    const int h = blockIdx.x * 8 + warp;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (h < H) load16<TQ>(q + ((bq * Hs + h) * (int64_t)TC_C + 16 * lane), v);
    if (threadIdx.x < 32) {
        rope_cos_sin(rope, q_pos[bq], threadIdx.x, cs[threadIdx.x], sn[threadIdx.x]);
        if (blockIdx.x == 0) {
            rope_cs[bq * 64 + threadIdx.x] = cs[threadIdx.x];
            rope_cs[bq * 64 + 32 + threadIdx.x] = sn[threadIdx.x];
        }
    }
    __syncthreads();
    // the image of (pass h / 64, query bq): passes side by side, gridDim.y queries each
    uint8_t* img = qimg + ((int64_t)(h >> 6) * gridDim.y + bq) * (int64_t)QIMG_BYTES;
    {
        if (flags & CSA2_QNORM) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
            ss = warp_sum(ss);
            const float r = 1.0f / sqrtf(ss / (float)TC_C + 1e-6f);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= r;
        }
        if ((flags & CSA2_ROPE) && lane >= 28) {      // dims 448..511, pairs (2j, 2j+1)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = 8 * (lane - 28) + i;
                const float c = cs[j], s = sn[j], x0 = v[2 * i], x1 = v[2 * i + 1];
                v[2 * i] = x0 * c - x1 * s;
                v[2 * i + 1] = x1 * c + x0 * s;
            }
        }
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pk[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        const int u0 = 2 * lane, chunk = u0 >> 3, uc = u0 & 7;
        const uint32_t hr = (uint32_t)(h & (TC_H - 1));     // row within the pass's image
        *reinterpret_cast<uint4*>(img + chunk * CHUNK_Q + sw128_offset(hr, uc)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<uint4*>(img + chunk * CHUNK_Q + sw128_offset(hr, uc + 1)) =
            make_uint4(pk[4], pk[5], pk[6], pk[7]);
    }
}

// RMS factor 1/sqrt(mean(x^2) + 1e-6) of every bf16 row of 512 values (a warp per row).
__global__ void __launch_bounds__(256) attn_rownorm_kernel(const uint8_t* rows, int64_t n_rows, float* rinv) {
    pdl_wait();
    pdl_trigger();
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= n_rows) return;
    const uint4* p = reinterpret_cast<const uint4*>(rows + row * (int64_t)(TC_C * 2)) + 2 * lane;
    float ss = 0.0f;
    bf16x8_sumsq(p[0], ss);
    bf16x8_sumsq(p[1], ss);
    ss = warp_sum(ss);
    if (lane == 0) rinv[row] = 1.0f / sqrtf(ss / (float)TC_C + 1e-6f);
}

// Output of a query whose split holds no key slot: the sink alone (O = 0).
template <typename TO>
__device__ void write_empty(const TcArgs& a, const ItemInfo& it, int d0) {
    for (int h = 0; h < it.H; ++h) {
        for (int d = d0; d < TC_C; d += 128) {
            if (a.n_split > 1)
                a.part[((it.prow + h) * a.n_split + it.split) * (int64_t)PART + ATTN_PART_O + d] = 0.0f;
            else
                reinterpret_cast<TO*>(a.out)[(it.bq * a.Hs + it.h0 + h) * (int64_t)TC_C + d] = from_f32<TO>(0.0f);
        }
    }
    if (d0 < it.H) {
        const int h = d0;
        if (a.n_split > 1) {
            float* p = a.part + ((it.prow + h) * a.n_split + it.split) * (int64_t)PART;
            p[0] = -INFINITY;
            p[1] = 0.0f;
        } else if (a.lse) {
            a.lse[it.bq * a.Hs + it.h0 + h] = a.sink ? a.sink[it.h0 + h] : -INFINITY;
        }
    }
}

// Output of heads [hbeg, hbeg + 32) of an item from O^T in tensor memory: the calling
// warp reads its 32-lane quarter `quad` (dims 32 quad + lane of every 128-dim block),
// scales by sc[h] (final output) and rotates back, or stores the unnormalised partial.
template <typename TO>
__device__ __forceinline__ void epilogue_heads(const TcArgs& a, const ItemInfo& it, uint32_t tmem, int quad, int lane,
                                               int hbeg, const float* sc) {
    const bool split = a.n_split > 1;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const int rr = quad * 32 + lane;
    const bool rot = !split && (a.flags & CSA2_ROPE) && quad >= 2;
    float rc = 1.0f, rs = 0.0f;
    if (rot) {
        const int j = (32 * quad + lane - 64) >> 1;
        rc = a.rope_cs[it.bq * 64 + j];
        rs = a.rope_cs[it.bq * 64 + 32 + j];
    }
    TO* obase = reinterpret_cast<TO*>(a.out) + (it.bq * a.Hs + it.h0 + hbeg) * (int64_t)TC_C + rr;
    float* pbase = a.part + ((it.prow + hbeg) * a.n_split + it.split) * (int64_t)PART + ATTN_PART_O + rr;
    const int64_t pstride = (int64_t)a.n_split * PART;
    // not unrolled: a CTA often runs this once (one item), from a cold instruction cache
#pragma unroll 1
    for (int db = 0; db < 4; ++db) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_base + (uint32_t)(db * TC_H + hbeg), o);
        tmem_wait_ld();
        if (split) {
            float* pb = pbase + db * 128;
#pragma unroll
            for (int h = 0; h < 32; ++h)
                if (hbeg + h < it.H) pb[h * pstride] = __uint_as_float(o[h]);
        } else {
            TO* ob = obase + db * 128;
            const bool rot_here = db == 3 && rot;
            float sc4[4];
#pragma unroll
            for (int h = 0; h < 32; ++h) {
                if ((h & 3) == 0) {
                    const float4 t4 = reinterpret_cast<const float4*>(sc + hbeg)[h >> 2];
                    sc4[0] = t4.x;
                    sc4[1] = t4.y;
                    sc4[2] = t4.z;
                    sc4[3] = t4.w;
                }
                float v = __uint_as_float(o[h]) * sc4[h & 3];
                if (rot_here) {
                    const float pv = __shfl_xor_sync(0xffffffffu, v, 1);
                    v = (lane & 1) ? v * rc - pv * rs : v * rc + pv * rs;
                }
                if (hbeg + h < it.H) ob[h * TC_C] = from_f32<TO>(v);
            }
        }
    }
}

// Merge of one (query, head)'s key splits by one warp, for this path's partials: every
// non-empty split used the same fixed offset (TC_SHIFT), so the unnormalised outputs
// and the sums of exponentials simply add up (an empty split holds zeros) and the
// output is scaled once, as a single split's epilogue does.  Every partial value is
// loaded in one batch (no pass over the splits' maxima first).  cs: RoPE cos, then
// sin, at the query position (NULL: no rotation).
template <typename TO>
__device__ __forceinline__ void tc_merge_row(const float* part, int ns, float zs, const float* cs, TO* o,
                                             float* lse) {
    const int lane = threadIdx.x & 31;
    float L = 0.0f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int sp = 0; sp < 8; ++sp) {
        if (sp >= ns) break;
        const float* pp = part + sp * (int64_t)PART;
        L += pp[1];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] += pp[ATTN_PART_O + lane + 32 * i];
    }
    float sc = 0.0f, ls = -INFINITY;
    if (L > 0.0f) {
        const float M = fmaxf(TC_SHIFT, zs);
        const float e = expf(TC_SHIFT - M);
        const float den = L * e + ((zs == -INFINITY) ? 0.0f : expf(zs - M));
        sc = e / den;
        ls = M + logf(den);
    } else if (zs != -INFINITY) {
        ls = zs;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= sc;
    if (cs) rope_lanes(acc, lane, cs, cs + 32, -1.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[lane + 32 * i] = from_f32<TO>(acc[i]);
    if (lse && lane == 0) *lse = ls;
}

template <bool FP4, typename TO>
// 14 warps: at most 128 registers a thread (four warps share one SM sub-partition's 16K registers)
__global__ void __launch_bounds__(TC_THREADS, 1) attn_tc_kernel(const TcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sQ = smem + OFF_Q;
    uint8_t* sK = smem + OFF_K;
    uint8_t* sP = smem + OFF_P;
    float* sRinv = reinterpret_cast<float*>(smem + OFF_RINV);
    float* sLw = reinterpret_cast<float*>(smem + OFF_LW);
    float* sSc = reinterpret_cast<float*>(smem + OFF_SC);
    float* sScL = reinterpret_cast<float*>(smem + OFF_SCL);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* qfull = bars + 0;
    uint64_t* qempty = bars + 1;
    uint64_t* kfull = bars + 2;        // [4] per 128-dim block of the tile
    uint64_t* kempty = bars + 6;       // [4]
    uint64_t* rfull = bars + 10;
    uint64_t* sfull = bars + 11;
    uint64_t* pfull = bars + 12;
    uint64_t* ofull = bars + 13;
    uint64_t* oempty = bars + 14;
    uint64_t* lred = bars + 15;
    uint64_t* scready = bars + 16;     // an item's output scales are in sScL
    uint64_t* stg = bars + 17;         // the tile's FP4 rows are staged (one arrival per loader thread)
    uint64_t* stgread = bars + 18;     // every loader warp has taken its rows' codes from the staging
    uint64_t* ssrdy = bars + 19;       // loader group 1's sums of squares are in sSS
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEMPTR);
    uint8_t* sStgSc = smem + OFF_STGSC;
    float* sSS = reinterpret_cast<float*>(smem + OFF_SS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&kfull[i], 4);
            mbar_init(&kempty[i], 1);
        }
        mbar_init(rfull, 4);
        mbar_init(sfull, 1);
        mbar_init(pfull, 4);
        mbar_init(ofull, 1);
        mbar_init(oempty, 8);
        mbar_init(scready, 1);
        mbar_init(lred, 4);
        mbar_init(stg, 2 * TC_TILE);
        mbar_init(stgread, 8);
        mbar_init(ssrdy, 4);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sTmem, TMEM_COLS);
        tmem_relinquish();
    }
    // everything above touches no global memory; the previous kernels (and their tensor
    // memory) are done before these CTAs can start, see pdl_wait()
    pdl_wait();                        // the query images, indices and rows are complete
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sTmem;

    if (warp == 0) {
        // ============================ producer ============================
        if (lane == 0) {
            int qi = 0, issued_q = -1;
            for (int64_t item = blockIdx.x; item < a.items && !a.stall; item += gridDim.x) {
                const ItemInfo it = item_info(a, item);
                if (it.nt == 0) continue;
                if (qi > 0 && !mbar_wait(qempty, (qi - 1) & 1, a.budget, a.st)) break;
                mbar_arrive_expect_tx(qfull, QIMG_BYTES);
                bulk_g2s(sQ, a.qimg + it.v * (int64_t)QIMG_BYTES, QIMG_BYTES, qfull);
                issued_q = qi++;
            }
            // the last copy must land before the CTA exits
            if (issued_q >= 0) mbar_wait(qfull, issued_q & 1, a.budget, a.st);
        }
    } else if (warp == 1) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            constexpr uint32_t IDESC_QK = idesc_f16(TC_TILE, TC_H, true);
            constexpr uint32_t IDESC_PV = idesc_f16_major(128, TC_H, true, true, true);
            const uint32_t q_base = smem_u32(sQ), k_base = smem_u32(sK), p_base = smem_u32(sP);
            int g = 0, qi = 0;
            bool ok = true;
            uint64_t* last_bar = nullptr;
            uint32_t last_par = 0;
            for (int64_t item = blockIdx.x; item < a.items && ok; item += gridDim.x) {
                const ItemInfo it = item_info(a, item);
                if (it.nt == 0) continue;
                if (!mbar_wait(qfull, qi & 1, a.budget, a.st)) {
                    ok = false;
                    break;
                }
                for (int tt = 0; tt < it.nt; ++tt, ++g) {
                    // logits: S^T = X . Qhat^T over 512 dims, the 128-dim blocks in the
                    // order the loaders produce them
                    for (int dbi = 0; dbi < 4 && ok; ++dbi) {
                        const int db = FP4 ? (dbi + 1) & 3 : dbi;
                        if (!mbar_wait(&kfull[db], g & 1, a.budget, a.st)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const int ch = 2 * db + (kk >> 2);
                            const uint32_t ko = (uint32_t)(kk & 3) * 32u;
                            mma_ss(tmem + DS_COL, sdesc_sw128(k_base + ch * CHUNK_K + ko),
                                   sdesc_sw128(q_base + ch * CHUNK_Q + ko), IDESC_QK, (dbi | kk) != 0);
                        }
                    }
                    if (!ok) break;
                    mma_commit(sfull);
                    last_bar = sfull;
                    last_par = g & 1;
                    if (tt == it.nt - 1) {
                        mma_commit(qempty);
                        last_bar = qempty;
                        last_par = qi & 1;
                    }
                    // output: O^T += X^T . P'^T over the tile's 128 slots
                    if (!mbar_wait(pfull, g & 1, a.budget, a.st) ||
                        (tt == 0 && qi > 0 && !mbar_wait(oempty, (qi - 1) & 1, a.budget, a.st))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int db = 0; db < 4; ++db) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            mma_ss(tmem + (uint32_t)db * TC_H,
                                   sdesc_sw128_mn(k_base + 2 * db * CHUNK_K + ks * 2048, CHUNK_K, 1024),
                                   sdesc_sw128_mn(p_base + ks * 2048, 1024, 1024), IDESC_PV, (tt > 0 || ks > 0));
                        }
                        mma_commit(&kempty[db]);
                    }
                    last_bar = &kempty[3];
                    last_par = g & 1;
                    if (tt == it.nt - 1) {
                        mma_commit(ofull);
                        last_bar = ofull;
                        last_par = qi & 1;
                    }
                }
                if (ok) ++qi;
            }
            // the MMAs must be complete before tensor memory is released
            if (last_bar) mbar_wait(last_bar, last_par, a.budget, a.st);
        }
    } else if (warp < 6) {
        // ============================ softmax + output ============================
        const int qd = warp & 3;
        const int r = qd * 32 + lane;                 // slot of the tile / dim of a 128-dim block
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        const float c1_base = LOG2E / sqrtf((float)TC_C);
        const float c0 = -TC_SHIFT * LOG2E;
        int g = 0, qi = 0;
        bool ok = true;
        for (int64_t item = blockIdx.x; item < a.items && ok; item += gridDim.x) {
            const ItemInfo it = item_info(a, item);
            if (it.nt == 0) {
                write_empty<TO>(a, it, r);
                continue;
            }
            float lacc[TC_H];
#pragma unroll
            for (int h = 0; h < TC_H; ++h) lacc[h] = 0.0f;
            for (int tt = 0; tt < it.nt; ++tt, ++g) {
                bool w = mbar_wait(sfull, g & 1, a.budget, a.st) && mbar_wait(rfull, g & 1, a.budget, a.st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float rinv = sRinv[r];
                const float c1 = rinv * c1_base;
                // heads 0..31, then 32..63 (half the logits live at a time)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t sv[32];
                    tmem_ld32(tmem + lane_base + DS_COL + 32 * hh, sv);
                    tmem_wait_ld();
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float p0 = ex2_approx(fmaf(__uint_as_float(sv[2 * i]), c1, c0));
                        float p1 = ex2_approx(fmaf(__uint_as_float(sv[2 * i + 1]), c1, c0));
                        if (rinv == 0.0f) p0 = p1 = 0.0f;
                        lacc[32 * hh + 2 * i] += p0;
                        lacc[32 * hh + 2 * i + 1] += p1;
                        pk[i] = pack_bf16x2(p0 * rinv, p1 * rinv);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        *reinterpret_cast<uint4*>(sP + sw128_offset((uint32_t)r, (uint32_t)(4 * hh + u))) =
                            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull);
            }
            if (!ok) break;
            // denominators: sum of p over the 128 slots (reduce-scatter: lane l ends
            // with heads 2l and 2l+1 of this warp's 32 slots)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const bool up = lane & 16;
                const float send = up ? lacc[i] : lacc[i + 32], keep = up ? lacc[i + 32] : lacc[i];
                lacc[i] = keep + __shfl_xor_sync(FULL, send, 16);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool up = lane & 8;
                const float send = up ? lacc[i] : lacc[i + 16], keep = up ? lacc[i + 16] : lacc[i];
                lacc[i] = keep + __shfl_xor_sync(FULL, send, 8);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool up = lane & 4;
                const float send = up ? lacc[i] : lacc[i + 8], keep = up ? lacc[i + 8] : lacc[i];
                lacc[i] = keep + __shfl_xor_sync(FULL, send, 4);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool up = lane & 2;
                const float send = up ? lacc[i] : lacc[i + 4], keep = up ? lacc[i + 4] : lacc[i];
                lacc[i] = keep + __shfl_xor_sync(FULL, send, 2);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool up = lane & 1;
                const float send = up ? lacc[i] : lacc[i + 2], keep = up ? lacc[i + 2] : lacc[i];
                lacc[i] = keep + __shfl_xor_sync(FULL, send, 1);
            }
            sLw[qd * TC_H + 2 * lane] = lacc[0];
            sLw[qd * TC_H + 2 * lane + 1] = lacc[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(lred);
            {
                const bool w = mbar_wait(lred, qi & 1, a.budget, a.st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
            }
            // per-head totals for heads lane and lane + 32; output scale and lse
            float sc2[2], lse2[2], L2[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = lane + 32 * j;
                const float L = sLw[h] + sLw[TC_H + h] + sLw[2 * TC_H + h] + sLw[3 * TC_H + h];
                const float zs = (a.sink && h < it.H) ? a.sink[it.h0 + h] : -INFINITY;
                float sc = 0.0f, ls = -INFINITY;
                if (L > 0.0f) {
                    const float M = fmaxf(TC_SHIFT, zs);
                    const float e = expf(TC_SHIFT - M);
                    const float den = L * e + ((zs == -INFINITY) ? 0.0f : expf(zs - M));
                    sc = e / den;
                    ls = M + logf(den);
                } else if (zs != -INFINITY) {
                    ls = zs;
                }
                sc2[j] = sc;
                lse2[j] = ls;
                L2[j] = L;
            }
            {
                const bool w = mbar_wait(ofull, qi & 1, a.budget, a.st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
            }
            tc_fence_after();
            const bool split = a.n_split > 1;
            // this warp's copy of the 64 output scales (lane holds heads lane, lane + 32);
            // warp 0 also publishes them for the loader warps, which store heads 32..63
            float* scw = sSc + qd * TC_H;
            scw[lane] = sc2[0];
            scw[lane + 32] = sc2[1];
            if (qd == 0) {
                sScL[(qi & 1) * TC_H + lane] = sc2[0];
                sScL[(qi & 1) * TC_H + lane + 32] = sc2[1];
            }
            __syncwarp();
            if (qd == 0 && lane == 0) mbar_arrive(scready);
            epilogue_heads<TO>(a, it, tmem, qd, lane, 0, scw);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
            if (qd == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = lane + 32 * j;
                    if (h >= it.H) continue;
                    if (split) {
                        float* p = a.part + ((it.prow + h) * a.n_split + it.split) * (int64_t)PART;
                        p[0] = L2[j] > 0.0f ? TC_SHIFT : -INFINITY;
                        p[1] = L2[j];
                    } else if (a.lse) {
                        a.lse[it.bq * a.Hs + it.h0 + h] = lse2[j];
                    }
                }
            }
            ++qi;
        }
    } else {
        // ============================ loaders ============================
        // two groups of four warps share the tile's slots, a thread per slot in each:
        // group 0 produces the 128-dim blocks {1, 0} of FP4 tiles ({0, 1} of bf16 tiles)
        // and the slot's RMS factor, group 1 the blocks {2, 3} and half of the squares
        const int lt = threadIdx.x - 192;
        const int hf = lt / TC_TILE;               // loader group
        const int r = lt % TC_TILE;                // slot of the tile
        const int quad = warp & 3;                 // tensor-memory lane quarter of this warp
        const int dbA = hf == 0 ? (FP4 ? 1 : 0) : 2;   // this group's blocks, in production order
        const int dbB = hf == 0 ? (FP4 ? 0 : 1) : 3;
        const uint8_t* kvb = reinterpret_cast<const uint8_t*>(a.kv);
        int g = 0, qi = 0;
        bool ok = true;
        // heads 32..63 of the previous item's output (group 0), stored once the next
        // item's first tile is on its way (or after the last item)
        ItemInfo pend;
        bool have_pend = false;
        auto run_pending = [&]() {
            bool w = mbar_wait(scready, (qi - 1) & 1, a.budget, a.st) && mbar_wait(ofull, (qi - 1) & 1, a.budget, a.st);
            if (!__all_sync(FULL, w)) {
                ok = false;
                return;
            }
            tc_fence_after();
            epilogue_heads<TO>(a, pend, tmem, quad, lane, 32, sScL + ((qi - 1) & 1) * TC_H);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
            have_pend = false;
        };
        for (int64_t item = blockIdx.x; item < a.items && ok; item += gridDim.x) {
            const ItemInfo it = item_info(a, item);
            for (int tt = 0; tt < it.nt && ok; ++tt, ++g) {
                const SlotSrc s = slot_source(a, it, (it.t0 + tt) * TC_TILE + r, true);
                const bool bf_row = s.kind == 2 || (s.kind == 1 && !FP4);
                const uint8_t* src = s.kind == 2 ? a.swa + s.row * (int64_t)(TC_C * 2)
                                                 : (bf_row ? kvb + s.row * (int64_t)(TC_C * 2) : nullptr);
                const float* pre = s.kind == 2 ? a.rinv_swa : (bf_row ? a.rinv_kv : nullptr);
                const float rpre = (hf == 0 && pre && s.kind != 0) ? pre[s.row] : 0.0f;
                const bool fp4_row = FP4 && s.kind == 1;
                const uint8_t* frow = fp4_row ? kvb + s.row * fp4_row_bytes(TC_C) : nullptr;
                // bf16 rows are copied cooperatively: per instruction the warp moves two of
                // its 32 rows, 256 contiguous bytes each (16 lanes x 16 B per row)
                const int wl = r >> 5, half = lane >> 4, piece = lane & 15;
                const uint8_t* srcj[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint64_t p = __shfl_sync(FULL, (uint64_t)(uintptr_t)(bf_row ? src : nullptr), 2 * j + half);
                    srcj[j] = reinterpret_cast<const uint8_t*>((uintptr_t)p);
                }
                float ss = 0.0f;
                bool w = true;
                uint4 kc[8];
                uint32_t ks[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < 8; ++i) kc[i] = make_uint4(0u, 0u, 0u, 0u);
                if (FP4) {
                    // the tile's FP4 rows are staged whole (codes in the space of block 0,
                    // whose PV reads finish first; scales beside), each group copying half
                    // of every row so that all copies are in flight together; each thread
                    // then takes its two blocks' codes into registers, and block 0 is
                    // written only after every loader warp has done so
                    if (g > 0) w = w && mbar_wait(&kempty[0], (g - 1) & 1, a.budget, a.st);
                    if (w && fp4_row) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            cp_async16(sK + stg_code_offset(r, 8 * hf + i), frow + 16 * (8 * hf + i));
                        cp_async16(sStgSc + r * 32 + 16 * hf, frow + 256 + 16 * hf);
                    }
                    cp_async_mbar_arrive_noinc(stg);
                    w = w && mbar_wait(stg, g & 1, a.budget, a.st);
                    if (w && fp4_row) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            kc[i] = *reinterpret_cast<const uint4*>(sK + stg_code_offset(r, 4 * dbA + i));
                            kc[4 + i] = *reinterpret_cast<const uint4*>(sK + stg_code_offset(r, 4 * dbB + i));
                        }
                        const uint2 sa = *reinterpret_cast<const uint2*>(sStgSc + r * 32 + 8 * dbA);
                        const uint2 sb = *reinterpret_cast<const uint2*>(sStgSc + r * 32 + 8 * dbB);
                        ks[0] = sa.x;
                        ks[1] = sa.y;
                        ks[2] = sb.x;
                        ks[3] = sb.y;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(stgread);
                }
#pragma unroll
                for (int bi = 0; bi < 2; ++bi) {
                    const int db = bi == 0 ? dbA : dbB;
                    if (g > 0 && !(FP4 && db == 0)) w = w && mbar_wait(&kempty[db], (g - 1) & 1, a.budget, a.st);
                    if (FP4 && db == 0) w = w && mbar_wait(stgread, g & 1, a.budget, a.st);
                    if (w) {
                        const int ch = 2 * db + (piece >> 3), u = piece & 7;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (srcj[j])
                                cp_async16(sK + ch * CHUNK_K + sw128_offset((uint32_t)(32 * wl + 2 * j + half), (uint32_t)u),
                                           srcj[j] + ch * 128 + u * 16);
                        }
                        if (fp4_row) {
                            ss += fp4_block_to_tile<CHUNK_K>(kc[4 * bi], kc[4 * bi + 1], kc[4 * bi + 2], kc[4 * bi + 3], ks[2 * bi],
                                                    ks[2 * bi + 1], sK, db, r);
                        } else if (!bf_row) {
#pragma unroll
                            for (int c2 = 2 * db; c2 < 2 * db + 2; ++c2)
#pragma unroll
                                for (int u2 = 0; u2 < 8; ++u2)
                                    *reinterpret_cast<uint4*>(sK + c2 * CHUNK_K + sw128_offset((uint32_t)r, (uint32_t)u2)) =
                                        make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    cp_async_commit();
                }
                // each 128-dim block is complete once its copy group has landed
                cp_async_wait<1>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kfull[dbA]);
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kfull[dbB]);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
                // squares of a bf16 row over this group's four 64-dim chunks (their copies
                // were made by this warp); not unrolled, for the same reason as the FP4 blocks
                if (bf_row && !pre) {
#pragma unroll 1
                    for (int ci = 0; ci < 4; ++ci) {
                        const int c = 2 * (ci < 2 ? dbA : dbB) + (ci & 1);
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            bf16x8_sumsq(*reinterpret_cast<const uint4*>(sK + c * CHUNK_K + sw128_offset((uint32_t)r, (uint32_t)u)),
                                         ss);
                    }
                }
                if (hf == 1) {
                    sSS[r] = ss;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ssrdy);
                    continue;
                }
                {
                    const bool w2 = mbar_wait(ssrdy, g & 1, a.budget, a.st);
                    if (!__all_sync(FULL, w2)) {
                        ok = false;
                        break;
                    }
                }
                float rv = 0.0f;
                if (s.kind != 0) rv = pre ? rpre : 1.0f / sqrtf((ss + sSS[r]) / (float)TC_C + 1e-6f);
                sRinv[r] = rv;
                __syncwarp();
                if (lane == 0) mbar_arrive(rfull);
                if (tt == 0 && have_pend) run_pending();
            }
            if (hf == 0 && it.nt > 0 && ok) {
                if (have_pend) run_pending();      // an item of a single tile: previous one first
                pend = it;
                have_pend = true;
                ++qi;
            }
        }
        if (hf == 0 && have_pend && ok) run_pending();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
    if (a.cluster) {
        // the query's splits merge here instead of in a combine kernel: once every CTA of
        // the cluster has written its partials (fence, then the cluster barrier), this
        // CTA merges its share of the heads from them, a warp per head
        __threadfence();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        const ItemInfo it = item_info(a, blockIdx.x);
        const int ns = a.n_split;
        const int hs = (it.H + ns - 1) / ns;
        const int h0 = it.split * hs, h1 = min(it.H, h0 + hs);
        const float* cs = (a.flags & CSA2_ROPE) ? a.rope_cs + it.bq * 64 : nullptr;
        for (int h = h0 + warp; h < h1; h += TC_THREADS / 32)
            tc_merge_row<TO>(a.part + (it.prow + h) * (int64_t)ns * PART, ns, a.sink ? a.sink[it.h0 + h] : -INFINITY,
                             cs, reinterpret_cast<TO*>(a.out) + (it.bq * a.Hs + it.h0 + h) * (int64_t)TC_C,
                             a.lse ? a.lse + it.bq * a.Hs + it.h0 + h : nullptr);
    }
}

void tc_splits(const csa2_ctx* ctx, int64_t n_bq, int k, int window, int& n_split, int& tps) {
    const int n_tiles = std::max(1, (k + window + TC_TILE - 1) / TC_TILE);
    // as many key splits as keep every (query, split) item in one wave of CTAs: a second
    // wave would put two items' tiles in a row on some SMs, and one wave lets a query's
    // splits run as one cluster that merges in the kernel
    int want = (int)std::min<int64_t>(n_tiles, std::max<int64_t>(1, ctx->num_sms / n_bq));
    tps = (n_tiles + want - 1) / want;
    n_split = (n_tiles + tps - 1) / tps;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Precomputed RMS factors pay off when the call gathers each cache row many times
// over (prefill: thousands of queries over one cache), not in decode.
bool want_row_table(int64_t n_bq, int k, int window, int64_t rows) {
    return rows > 0 && n_bq * (int64_t)(k + window) >= 4 * rows;
}

struct WsLayout {
    size_t part, qimg, rope, rinv_kv, rinv_swa, total;
    int n_split, tps;
    bool table;
};

WsLayout ws_layout(const csa2_ctx* ctx, int B, int Q, int H, int k, int window, int64_t N, int64_t swa_cap,
                   int n_pass = 1) {
    WsLayout L;
    const int64_t n_bq = (int64_t)B * Q;
    // every pass of every query is an item group of its own
    tc_splits(ctx, n_bq * n_pass, k, window, L.n_split, L.tps);
    if (n_pass > 1) H = TC_H * n_pass;                   // partial rows of all passes
    const int64_t kv_rows = (k > 0) ? (int64_t)B * std::max<int64_t>(N, 0) : 0;
    const int64_t sw_rows = (window > 0) ? (int64_t)B * std::max<int64_t>(swa_cap, 0) : 0;
    L.table = want_row_table(n_bq, k, window, kv_rows + sw_rows);
    L.part = 0;
    L.qimg = L.n_split > 1 ? align_up((size_t)n_bq * H * L.n_split * PART * sizeof(float), 1024) : 0;
    L.rope = L.qimg + (size_t)n_bq * n_pass * QIMG_BYTES;
    L.rinv_kv = align_up(L.rope + (size_t)n_bq * 64 * sizeof(float), 256);
    L.rinv_swa = align_up(L.rinv_kv + (L.table ? (size_t)kv_rows * sizeof(float) : 0), 256);
    L.total = L.rinv_swa + (L.table ? (size_t)sw_rows * sizeof(float) : 0);
    return L;
}

// Whether clusters of ns CTAs of this kernel can be resident (asked once per size).
template <bool FP4, typename TO>
bool tc_cluster_ok(int ns) {
    static int ok[9] = {-1, -1, -1, -1, -1, -1, -1, -1, -1};
    if (ns < 2 || ns > 8) return false;
    if (ok[ns] < 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ns);
        cfg.blockDim = dim3(TC_THREADS);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)ns;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        ok[ns] = cudaOccupancyMaxActiveClusters(&n, attn_tc_kernel<FP4, TO>, &cfg) == cudaSuccess && n > 0;
        (void)cudaGetLastError();
    }
    return ok[ns] == 1;
}

template <bool FP4, typename TO>
csa2_status launch_tc(const csa2_ctx* ctx, TcArgs& a, cudaStream_t s) {
    auto kern = attn_tc_kernel<FP4, TO>;
    static bool attr = false;
    if (!attr) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess)
            return CSA2_ERR_CUDA;
        attr = true;
    }
    // few queries (decode): one item per CTA, and a query's splits as one cluster that
    // merges its partials in the kernel
    a.cluster = a.n_split > 1 && a.n_split <= 8 && a.items <= ctx->num_sms && tc_cluster_ok<FP4, TO>(a.n_split);
    const int64_t grid = std::min<int64_t>(a.items, ctx->num_sms);
    if (!a.cluster) {
        const csa2_status r = launch_pdl(kern, dim3((unsigned)grid), dim3(TC_THREADS), SMEM_BYTES, s, a);
        return r != CSA2_OK ? r : csa2_launch_status();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.n_split;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see pdl_wait()
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return CSA2_ERR_CUDA;
    return csa2_launch_status();
}

}  // namespace

bool attn_tc_applies(const AttnTcCall& c) {
    if (c.q_dt != CSA2_BF16) return false;
    if (c.kv_dt != CSA2_BF16 && c.kv_dt != CSA2_FP4_E4M3x16) return false;
    if (c.window > 0 && c.swa_dt != CSA2_BF16) return false;
    if ((c.flags & (CSA2_QNORM | CSA2_KVNORM)) != (CSA2_QNORM | CSA2_KVNORM)) return false;
    if (c.H < 1 || c.H > TC_H) return false;
    return true;
}

size_t attn_tc_ws_bytes(const csa2_ctx* ctx, int B, int Q, int H, int k, int window, int64_t N, int64_t swa_cap) {
    if (!ctx || H < 1 || B <= 0 || Q <= 0) return 0;
    return ws_layout(ctx, B, Q, std::min(H, TC_H), k, window, N, swa_cap).total;
}

size_t attn_tc_ws_bytes_all_passes(const csa2_ctx* ctx, int B, int Q, int H, int k, int window, int64_t N,
                                   int64_t swa_cap) {
    if (!ctx || H < 1 || B <= 0 || Q <= 0) return 0;
    const int n_pass = (H + TC_H - 1) / TC_H;
    return ws_layout(ctx, B, Q, std::min(H, TC_H), k, window, N, swa_cap, n_pass).total;
}

const float* attn_tc_rope_table(const csa2_ctx* ctx, const AttnTcCall& c, void* ws) {
    const WsLayout L = ws_layout(ctx, c.B, c.Q, c.H, c.k, c.window, c.N, c.swa_cap, c.n_pass);
    return reinterpret_cast<const float*>(reinterpret_cast<uint8_t*>(ws) + L.rope);
}

namespace {

csa2_status attn_tc_prepare_into(const AttnTcCall& c, uint8_t* qimg, float* rope_cs, cudaStream_t s) {
    const int64_t n_bq = (int64_t)c.B * c.Q;
    const csa2_status rq =
        c.q_dt == CSA2_BF16
            ? launch_pdl(attn_qprep_kernel<__nv_bfloat16>, dim3(8 * c.n_pass, (unsigned)n_bq), dim3(256), 0, s,
                         reinterpret_cast<const __nv_bfloat16*>(c.q), c.q_pos, c.n_pass > 1 ? c.Hs : c.H, c.Hs, c.rope,
                         c.flags, qimg, rope_cs)
            : launch_pdl(attn_qprep_kernel<float>, dim3(8 * c.n_pass, (unsigned)n_bq), dim3(256), 0, s,
                         reinterpret_cast<const float*>(c.q), c.q_pos, c.n_pass > 1 ? c.Hs : c.H, c.Hs, c.rope,
                         c.flags, qimg, rope_cs);
    return rq != CSA2_OK ? rq : csa2_launch_status();
}

}  // namespace

csa2_status attn_tc_prepare(csa2_ctx* ctx, const AttnTcCall& c, void* ws, size_t ws_bytes, cudaStream_t s) {
    const WsLayout L = ws_layout(ctx, c.B, c.Q, c.H, c.k, c.window, c.N, c.swa_cap, c.n_pass);
    if (!ws || !aligned(ws, 16) || ws_bytes < L.rinv_kv) return CSA2_ERR_INVALID_ARG;
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    return attn_tc_prepare_into(c, base + L.qimg, reinterpret_cast<float*>(base + L.rope), s);
}

csa2_status attn_tc_run(csa2_ctx* ctx, const AttnTcCall& c, void* ws, size_t ws_bytes, cudaStream_t s,
                        int* n_split) {
    const int64_t n_bq = (int64_t)c.B * c.Q;
    const WsLayout L = ws_layout(ctx, c.B, c.Q, c.H, c.k, c.window, c.N, c.swa_cap, c.n_pass);
    if (!ws || !aligned(ws, 16) || ws_bytes < L.rinv_kv) return CSA2_ERR_INVALID_ARG;
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    uint8_t* qimg = base + L.qimg;
    float* rope_cs = reinterpret_cast<float*>(base + L.rope);
    // the query images and RoPE table (unless csa2_attn_prepare wrote them already)
    if (!(c.flags & CSA2_ATTN_PREPARED)) {
        const csa2_status rq = attn_tc_prepare_into(c, qimg, rope_cs, s);
        if (rq != CSA2_OK) return rq;
    }
    TcArgs a;
    a.rinv_kv = nullptr;
    a.rinv_swa = nullptr;
    if (L.table && ws_bytes >= L.total) {
        const bool kv_bf = c.kv_dt == CSA2_BF16 && c.k > 0 && c.N > 0;
        if (kv_bf) {
            float* t = reinterpret_cast<float*>(base + L.rinv_kv);
            const int64_t rows = (int64_t)c.B * c.N;
            attn_rownorm_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(reinterpret_cast<const uint8_t*>(c.kv),
                                                                          rows, t);
            a.rinv_kv = t;
        }
        if (c.window > 0) {
            float* t = reinterpret_cast<float*>(base + L.rinv_swa);
            const int64_t rows = (int64_t)c.B * c.swa_cap;
            attn_rownorm_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(reinterpret_cast<const uint8_t*>(c.swa),
                                                                          rows, t);
            a.rinv_swa = t;
        }
    }
    a.qimg = qimg;
    a.rope_cs = rope_cs;
    a.kv = c.kv;
    a.swa = reinterpret_cast<const uint8_t*>(c.swa);
    a.N = c.N;
    a.idx = c.idx;
    a.k = c.k;
    a.dense_nv = c.dense_nv;
    a.swa_cap = c.swa_cap;
    a.swa_pos0 = c.swa_pos0;
    a.window = c.window;
    a.q_pos = c.q_pos;
    a.sink = c.sink;
    a.Q = c.Q;
    a.H = c.H;
    a.Hs = c.Hs;
    a.rope = c.rope;
    a.flags = c.flags;
    a.out = c.out;
    a.lse = c.lse;
    a.part = reinterpret_cast<float*>(base + L.part);
    a.n_split = L.n_split;
    a.tps = L.tps;
    a.n_pass = c.n_pass;
    a.n_bq = n_bq;
    a.items = n_bq * c.n_pass * L.n_split;
    a.st = ctx->status;
    a.budget = WAIT_BUDGET;
    a.stall = 0;
    if (ctx->stall_next) {
        a.stall = 1;
        if (ctx->stall_budget > 0) a.budget = ctx->stall_budget;
        ctx->stall_next = 0;
    }
    *n_split = L.n_split;
    a.cluster = 0;
    const bool fp4 = c.kv_dt == CSA2_FP4_E4M3x16;
    const bool f32o = c.out_dt == CSA2_F32;
    const csa2_status r = fp4 ? (f32o ? launch_tc<true, float>(ctx, a, s) : launch_tc<true, __nv_bfloat16>(ctx, a, s))
                              : (f32o ? launch_tc<false, float>(ctx, a, s) : launch_tc<false, __nv_bfloat16>(ctx, a, s));
    if (a.cluster) *n_split = 1;           // merged in the kernel
    return r;
}
