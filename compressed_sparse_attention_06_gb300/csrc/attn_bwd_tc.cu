// Backward pass of the shared-KV MQA on the tcgen05 tensor cores (attn_bwd.cu has the
// formulas): bf16 query, rows, window and dout, both RMSNorms, head passes of 64.
//
// Work item = (head pass, query, range of 64-slot key tiles).  A query's stacked image --
// 128 rows of 512 dims, the normalised rotated heads q^ and the rotated gradients do',
// interleaved 16 by 16 -- stays in shared memory for the whole item; a tile of raw key rows
// X [64 slots x 512] is gathered once and read by two products, the image by two:
//   [S; dP] [128 x 64 slots]   = image . X^T           (S and dP of a head 16 lanes apart)
//   dQ^T    [512 dims x 64]   += X^T . (r dS)^T
//   dK^T    [512 dims x 64 slots] = image^T . [r dS; r P]
// p = exp(z - lse), dS = p (dP - D)/sqrt(c), r the row's RMS factor (folded in, so X is never
// rescaled and dK comes out as the row's contribution r dk^).  dQ accumulates in tensor memory
// over the item; dK leaves per tile, in 128-dim blocks through a ring of three accumulators, to
// its place in the sorted list of contributions, as bf16: the list is written and read once
// from device memory and its size is what bounds the row sums.  The addends' rounding
// (2^-8 at most, of values that p and dS rounded to bf16 made) is no larger than theirs; the
// sums over them are fp32.
//
// Warp roles (448 threads, one CTA per SM, persistent over items):
//   warp 0       the images (four 32 KB bulk copies, each freed by its dK block)
//   warp 1       MMA issuer; owns the tensor memory
//   warps 2-5    softmax: one thread per stacked row
//   warps 6-9    loaders: 16-byte cp.async into a ring of five 128-dim blocks of X
//   warps 10-13  drain: dK blocks every tile, dQ at the end of the item
// Every wait is bounded; a wait that expires flags a timeout and the roles wind down.
#include <algorithm>
#include <atomic>

#include "attn_bwd_tc.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace sm100;

constexpr int BT_C = 512;
constexpr int BT_H = 64;
constexpr int BT_TILE = 64;
constexpr int BT_THREADS = 448;
constexpr int IMG_CHUNK = 128 * 128;             // 128 stacked rows x 64 dims
constexpr int IMG_BYTES = 8 * IMG_CHUNK;
constexpr int X_CHUNK = BT_TILE * 128;           // 64 slots x 64 dims
constexpr int X_BLOCK = 2 * X_CHUNK;
constexpr int X_RING = 5;
constexpr int DK_RING = 3;
constexpr uint32_t COL_DQ = 0, COL_S = 256, COL_DK = 320;
constexpr uint32_t TMEM_COLS = 512;
constexpr long long WAIT_BUDGET = 1ll << 31;
constexpr unsigned FULL = 0xffffffffu;

constexpr int OFF_IMG = 0;
constexpr int OFF_X = OFF_IMG + IMG_BYTES;
constexpr int OFF_DSP = OFF_X + X_RING * X_BLOCK;       // [128 rows: r dS of 64 heads, r P][64 slots]
constexpr int OFF_RINV = OFF_DSP + 128 * 128;           // [4 warps][2 x 36]
constexpr int OFF_BAR = OFF_RINV + 4 * 72 * 4;
constexpr int N_BAR = 4 + 4 + X_RING + X_RING + 4 + 2 * DK_RING + 3;
constexpr int OFF_TMEMPTR = OFF_BAR + N_BAR * 8;
constexpr int SMEM_BYTES = OFF_TMEMPTR + 16 + 1024;
static_assert(OFF_BAR % 8 == 0, "barrier alignment");
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

struct Item {
    int64_t v;                   // pass * nb + query: the image
    int64_t bq;
    int q, pass, split;          // query within the chunk
    int kq, nw, n, t0, nt;       // cache slots, window slots, both; tiles t0 .. t0 + nt - 1
    int64_t kv0, sw0;            // row ids of the sequence's first cache row and window row
    int win0;                    // window row of the first window slot
};

__device__ __forceinline__ Item item_of(const BwdTcArgs& a, int64_t i) {
    Item r;
    r.v = i / a.n_split;
    r.split = (int)(i - r.v * a.n_split);
    r.pass = (int)(r.v / a.c.nb);
    r.q = (int)(r.v - (int64_t)r.pass * a.c.nb);
    r.bq = a.c.bq0 + r.q;
    const int64_t t = a.c.slots.q_pos[r.bq];
    r.nw = (int)max((int64_t)0, min((int64_t)a.c.slots.window, t + 1));
    r.kq = a.c.slots.dense_nv ? (int)max((int64_t)0, min((int64_t)a.c.slots.k, a.c.slots.dense_nv[r.bq])) : a.c.slots.k;
    r.n = r.kq + r.nw;
    const int tiles = (r.n + BT_TILE - 1) / BT_TILE;
    r.t0 = r.split * a.tps;
    r.nt = max(0, min(tiles, r.t0 + a.tps) - r.t0);
    const int64_t b = r.bq / a.c.slots.Q;
    r.kv0 = b * a.c.slots.N;
    r.sw0 = a.c.slots.n_kv + b * a.c.slots.swa_cap;
    r.win0 = 0;
    if (r.nw > 0) {
        const int64_t w = (t - r.nw + 1 - a.c.slots.swa_pos0) % a.c.slots.swa_cap;
        r.win0 = (int)(w < 0 ? w + a.c.slots.swa_cap : w);
    }
    return r;
}

// Row id (slot_row's) of position s of the item's slots -- its cache slots, then its window
// slots without the positions before 0 -- and in *slot the slot's number; -1 if it is empty.
__device__ __forceinline__ int64_t row_of(const BwdTcArgs& a, const Item& it, int s, int* slot) {
    *slot = 0;
    if (s >= it.n) return -1;
    if (s < it.kq) {
        *slot = s;
        const int id = a.c.slots.dense_nv ? s : a.c.slots.idx[it.bq * a.c.slots.k + s];
        return id >= 0 && id < a.c.slots.N ? it.kv0 + id : -1;
    }
    const int w = s - it.kq;
    *slot = a.c.slots.k + (a.c.slots.window - it.nw) + w;
    int64_t at = (int64_t)it.win0 + w;
    if (at >= a.c.slots.swa_cap) at -= a.c.slots.swa_cap;
    return it.sw0 + at;
}

// Position in a ring of n stages and the parity of its current round.
struct Ring {
    int i = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            ++round;
        }
    }
};

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Stacked images of the chunk's queries and D; a warp per head, 8 heads a CTA.  Image row of
// head h (within its pass): 32 (h / 16) + h % 16 for q^, 16 more for do'.  Heads past H are 0.
__global__ void __launch_bounds__(256) bwd_tc_prep_kernel(const __nv_bfloat16* q, const __nv_bfloat16* dout,
                                                          const __nv_bfloat16* out, const int64_t* q_pos, int64_t bq0,
                                                          int nb, int H, AgRope rope, unsigned flags, uint8_t* img,
                                                          float* D) {
    __shared__ float cs[32], sn[32];
    const int qi = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t bq = bq0 + qi;
    const int h = blockIdx.x * 8 + w;
    if (threadIdx.x < 32) ag_cos_sin(rope, q_pos[bq], lane, cs[lane], sn[lane]);
    float v[16], g[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = g[i] = 0.0f;
    if (h < H) {
        const int64_t o = (bq * H + h) * (int64_t)BT_C + 16 * lane;
        ag_load16<__nv_bfloat16>(q + o, v);
        ag_load16<__nv_bfloat16>(dout + o, g);
        float x[16], dot = 0.0f;
        ag_load16<__nv_bfloat16>(out + o, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) dot = fmaf(g[i], x[i], dot);
        dot = warp_sum(dot);
        if (lane == 0) D[bq * H + h] = dot;
    }
    __syncthreads();
    if (flags & CSA2_QNORM) {
        const float f = ag_rms_factor(warp_sum(ag_sumsq16(v)));
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= f;
    }
    if (flags & CSA2_ROPE) {
        ag_rope16(v, lane, cs, sn, 1.0f);
        ag_rope16(g, lane, cs, sn, 1.0f);
    }
    uint8_t* base = img + ((int64_t)(h >> 6) * nb + qi) * IMG_BYTES + (lane >> 2) * IMG_CHUNK;
    const uint32_t row = 32u * ((h & 63) >> 4) + (h & 15), u = 2u * (lane & 3);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = k == 0 ? ag_pack_bf16x2(v[2 * i], v[2 * i + 1]) : ag_pack_bf16x2(g[2 * i], g[2 * i + 1]);
        *reinterpret_cast<uint4*>(base + sw128_offset(row + 16 * k, u)) = make_uint4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<uint4*>(base + sw128_offset(row + 16 * k, u + 1)) = make_uint4(p[4], p[5], p[6], p[7]);
    }
}

// dq from dq^ (the sum of the item's splits): back through RoPE and the query's RMSNorm.  A
// warp per (query, head); a query that attends to nothing has no gradient.
__global__ void __launch_bounds__(256) bwd_tc_dq_kernel(BwdTcArgs a, const float* dqh, __nv_bfloat16* dq) {
    __shared__ float cs[8][32], sn[8][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + w;
    if (r >= (int64_t)a.c.nb * a.c.H) return;
    const int qi = (int)(r / a.c.H), h = (int)(r % a.c.H);
    const int64_t bq = a.c.bq0 + qi, o = (bq * a.c.H + h) * BT_C + 16 * lane;
    ag_cos_sin(a.c.rope, a.c.slots.q_pos[bq], lane, cs[w][lane], sn[w][lane]);
    __syncwarp();
    float g[16], v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = 0.0f;
    const int64_t item = ((int64_t)(h >> 6) * a.c.nb + qi) * a.n_split;
    for (int s = 0; s < a.n_split; ++s) {
        float p[16];
        ag_load16<float>(dqh + ((item + s) * BT_H + (h & 63)) * BT_C + 16 * lane, p);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] += p[i];
    }
    ag_load16<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.c.q) + o, v);
    const float f = ag_rms_factor(warp_sum(ag_sumsq16(v)));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= f;
    if (a.c.flags & CSA2_ROPE) ag_rope16(g, lane, cs[w], sn[w], -1.0f);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) dot = fmaf(v[i], g[i], dot);
    dot = warp_sum(dot) / (float)BT_C;
    const bool none = a.c.lse[bq * a.c.H + h] == -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = none ? 0.0f : f * (g[i] - v[i] * dot);
    ag_store16<__nv_bfloat16>(dq + o, g);
}

__global__ void __launch_bounds__(BT_THREADS, 1) attn_bwd_tc_kernel(const BwdTcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sImg = smem + OFF_IMG;
    uint8_t* sX = smem + OFF_X;
    uint8_t* sDsp = smem + OFF_DSP;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* imgfull = bars;                       // [4] 128-dim blocks of the image
    uint64_t* imgempty = bars + 4;                  // [4]
    uint64_t* xfull = bars + 8;                     // [X_RING]
    uint64_t* xempty = xfull + X_RING;              // [X_RING]
    uint64_t* sfull = xempty + X_RING;
    uint64_t* sempty = sfull + 1;
    uint64_t* dspfull = sfull + 2;
    uint64_t* dspempty = sfull + 3;
    uint64_t* dkfull = sfull + 4;                   // [DK_RING]
    uint64_t* dkempty = dkfull + DK_RING;           // [DK_RING]
    uint64_t* dqfull = dkempty + DK_RING;
    uint64_t* dqempty = dqfull + 1;
    uint64_t* alldone = dqfull + 2;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEMPTR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&imgfull[i], 1);
            mbar_init(&imgempty[i], 1);
        }
        for (int i = 0; i < X_RING; ++i) {
            mbar_init(&xfull[i], 4);
            mbar_init(&xempty[i], 1);
        }
        mbar_init(sfull, 1);
        mbar_init(sempty, 4);
        mbar_init(dspfull, 4);
        mbar_init(dspempty, 1);
        for (int i = 0; i < DK_RING; ++i) {
            mbar_init(&dkfull[i], 1);
            mbar_init(&dkempty[i], 4);
        }
        mbar_init(dqfull, 1);
        mbar_init(dqempty, 4);
        mbar_init(alldone, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sTmem, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sTmem;

    if (warp == 0) {
        // ============================ images ============================
        if (lane == 0) {
            int n = 0;                               // items with tiles so far
            bool ok = true;
            int issued = 0;                          // blocks issued in the last item, and their phase
            uint32_t par = 0;
            for (int64_t i = blockIdx.x; i < a.items && ok && !a.stall; i += gridDim.x) {
                const Item it = item_of(a, i);
                if (it.nt == 0) continue;
                issued = 0;
                par = n & 1;
                for (int db = 0; db < 4; ++db) {
                    if (n > 0 && !mbar_wait(&imgempty[db], (n - 1) & 1, a.budget, a.c.slots.st)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&imgfull[db], 2 * IMG_CHUNK);
                    bulk_g2s(sImg + db * 2 * IMG_CHUNK, a.img + it.v * (int64_t)IMG_BYTES + db * 2 * IMG_CHUNK,
                             2 * IMG_CHUNK, &imgfull[db]);
                    issued = db + 1;
                }
                ++n;
            }
            // the last copies must land before the CTA exits
            for (int db = 0; db < issued; ++db) mbar_wait(&imgfull[db], par, a.budget, a.c.slots.st);
        }
    } else if (warp == 1) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_f16(128, BT_TILE, true);
            constexpr uint32_t ID_DQ = idesc_f16_major(128, BT_H, true, true, false);
            constexpr uint32_t ID_DK = idesc_f16_major(128, BT_TILE, true, true, true);
            const uint32_t img = smem_u32(sImg), x0 = smem_u32(sX), dsp = smem_u32(sDsp);
            uint32_t g = 0;                          // tiles so far
            int n = 0;                               // items with tiles so far
            Ring xs, xq, dk;                         // X blocks of S and of dQ, dK accumulators
            bool ok = true;
            auto wait = [&](uint64_t* b, uint32_t par) {
                ok = ok && mbar_wait(b, par, a.budget, a.c.slots.st);
                return ok;
            };
            for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
                const Item it = item_of(a, i);
                if (it.nt == 0) continue;
                for (int tt = 0; tt < it.nt && ok; ++tt, ++g) {
                    const bool last = tt == it.nt - 1;
                    if (g > 0 && !wait(sempty, (g - 1) & 1)) break;
                    for (int db = 0; db < 4; ++db) {
                        if (tt == 0 && !wait(&imgfull[db], n & 1)) break;
                        if (!wait(&xfull[xs.i], xs.round & 1)) break;
                        tc_fence_after();
                        const uint64_t da = sdesc_sw128(img + 2 * db * IMG_CHUNK), dx = sdesc_sw128(x0 + xs.i * X_BLOCK);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ss(tmem + COL_S, da + (((kk >> 2) * IMG_CHUNK + (kk & 3) * 32) >> 4),
                                   dx + (((kk >> 2) * X_CHUNK + (kk & 3) * 32) >> 4), ID_S, (db | kk) != 0);
                        xs.next(X_RING);
                    }
                    if (!ok) break;
                    mma_commit(sfull);
                    if (!wait(dspfull, g & 1)) break;
                    if (tt == 0 && n > 0 && !wait(dqempty, (n - 1) & 1)) break;
                    tc_fence_after();
                    const uint64_t dds = sdesc_sw128(dsp);
                    for (int db = 0; db < 4; ++db) {
                        const uint64_t dx = sdesc_sw128_mn(x0 + xq.i * X_BLOCK, X_CHUNK, 1024);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ss(tmem + COL_DQ + db * BT_H, dx + (ks * 2048 >> 4), dds + (ks * 32 >> 4), ID_DQ,
                                   tt > 0 || ks > 0);
                        mma_commit(&xempty[xq.i]);
                        xq.next(X_RING);
                    }
                    if (last) mma_commit(dqfull);
                    const uint64_t dsp_mn = sdesc_sw128_mn(dsp, 1024, 1024);
                    for (int db = 0; db < 4; ++db) {
                        if (dk.round > 0 && !wait(&dkempty[dk.i], (dk.round - 1) & 1)) break;
                        tc_fence_after();
                        const uint64_t da = sdesc_sw128_mn(img + 2 * db * IMG_CHUNK, IMG_CHUNK, 1024);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            // image rows 16 ks .. : q^ (even ks) or do' (odd) of heads 16 (ks / 2) ..
                            const uint32_t row = 16u * (ks >> 1) + (ks & 1 ? 64u : 0u);
                            mma_ss(tmem + COL_DK + dk.i * BT_TILE, da + (ks * 2048 >> 4), dsp_mn + (row * 128 >> 4), ID_DK,
                                   ks > 0);
                        }
                        mma_commit(&dkfull[dk.i]);
                        if (last) mma_commit(&imgempty[db]);
                        dk.next(DK_RING);
                    }
                    if (!ok) break;
                    mma_commit(dspempty);
                }
                if (ok) ++n;
            }
            // the MMAs must be complete before tensor memory is released
            mma_commit(alldone);
            mbar_wait(alldone, 0, a.budget, a.c.slots.st);
        }
    } else if (warp < 6) {
        // ============================ softmax ============================
        const int qd = warp & 3;
        const int hl = 16 * qd + (lane & 15);                 // head of the pass
        const bool up = lane & 16;                            // this lane's slots: 32 .. 63 of the tile
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        float* rv = reinterpret_cast<float*>(smem + OFF_RINV) + qd * 72;
        const float isc = 1.0f / sqrtf((float)BT_C);
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            if (it.nt == 0) continue;
            const int h = it.pass * BT_H + hl;
            float lse2 = INFINITY, D = 0.0f;                  // p = 0 for heads past H and empty queries
            if (h < a.c.H) {
                const float l = a.c.lse[it.bq * a.c.H + h];
                if (l != -INFINITY) {
                    lse2 = l * AG_LOG2E;
                    D = a.c.D[it.bq * a.c.H + h];
                }
            }
            for (int tt = 0; tt < it.nt; ++tt, ++g) {
                // RMS factors of the tile's rows, 0 for empty slots (this warp's copy)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int slot;
                    const int64_t row = row_of(a, it, (it.t0 + tt) * BT_TILE + 32 * j + lane, &slot);
                    rv[36 * j + lane] = row >= 0 ? a.c.rinv[row] : 0.0f;
                }
                __syncwarp();
                bool w = mbar_wait(sfull, g & 1, a.budget, a.c.slots.st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t lo[32], hi[32];
                tmem_ld32(tmem + lane_base + COL_S, lo);
                tmem_ld32(tmem + lane_base + COL_S + 32, hi);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty);
                // lanes l and l + 16 hold S and dP of the same head: each takes 32 of the slots
                uint32_t ds[16], pp[16];
#pragma unroll
                for (int c4 = 0; c4 < 8; ++c4) {
                    const float4 r4 = *reinterpret_cast<const float4*>(rv + (up ? 36 : 0) + 4 * c4);
                    const float rr[4] = {r4.x, r4.y, r4.z, r4.w};
                    float dsv[4], pv[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 4 * c4 + k;
                        const float got = __uint_as_float(__shfl_xor_sync(FULL, up ? lo[c] : hi[c], 16));
                        const float s = up ? got : __uint_as_float(lo[c]);
                        const float dp = up ? __uint_as_float(hi[c]) : got;
                        const float r = rr[k];
                        float p = ex2_approx(fmaf(s * r, isc * AG_LOG2E, -lse2));
                        if (r == 0.0f) p = 0.0f;
                        pv[k] = p * r;
                        dsv[k] = p == 0.0f ? 0.0f : pv[k] * (fmaf(dp, r, -D) * isc);
                    }
                    ds[2 * c4] = ag_pack_bf16x2(dsv[0], dsv[1]);
                    ds[2 * c4 + 1] = ag_pack_bf16x2(dsv[2], dsv[3]);
                    pp[2 * c4] = ag_pack_bf16x2(pv[0], pv[1]);
                    pp[2 * c4 + 1] = ag_pack_bf16x2(pv[2], pv[3]);
                }
                if (g > 0) w = mbar_wait(dspempty, (g - 1) & 1, a.budget, a.c.slots.st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t unit = (up ? 4u : 0u) + u;
                    *reinterpret_cast<uint4*>(sDsp + sw128_offset((uint32_t)hl, unit)) =
                        make_uint4(ds[4 * u], ds[4 * u + 1], ds[4 * u + 2], ds[4 * u + 3]);
                    *reinterpret_cast<uint4*>(sDsp + sw128_offset(64u + hl, unit)) =
                        make_uint4(pp[4 * u], pp[4 * u + 1], pp[4 * u + 2], pp[4 * u + 3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(dspfull);
            }
        }
    } else if (warp < 10) {
        // ============================ loaders ============================
        const int lw = warp - 6;                              // slots 16 lw .. 16 lw + 15 of the tile
        const int half = lane >> 4, piece = lane & 15;        // a copy moves 256 bytes of two rows
        const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.c.kv);
        const uint8_t* swa = reinterpret_cast<const uint8_t*>(a.c.swa);
        Ring in, out;                                         // blocks issued, blocks signalled
        int behind = 0;                                       // in flight: issued, not signalled
        bool ok = true;
        auto signal = [&]() {                                 // the oldest block in flight
            if (behind == 4)
                cp_async_wait<3>();
            else if (behind == 3)
                cp_async_wait<2>();
            else if (behind == 2)
                cp_async_wait<1>();
            else
                cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&xfull[out.i]);
            out.next(X_RING);
            --behind;
        };
        for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            for (int tt = 0; tt < it.nt && ok; ++tt) {
                int slot;
                const int64_t row = lane < 16 ? row_of(a, it, (it.t0 + tt) * BT_TILE + 16 * lw + lane, &slot) : -1;
                const uint8_t* src = nullptr;
                if (row >= 0)
                    src = row < a.c.slots.n_kv ? kv + row * (BT_C * 2) : swa + (row - a.c.slots.n_kv) * (BT_C * 2);
                const uint8_t* from[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    from[j] = reinterpret_cast<const uint8_t*>(
                        (uintptr_t)__shfl_sync(FULL, (unsigned long long)(uintptr_t)src, 2 * j + half));
                for (int db = 0; db < 4; ++db) {
                    if (in.round > 0) {
                        const uint32_t par = (in.round - 1) & 1;
                        // blocks in flight are signalled before a wait that they may be needed for
                        if (!__all_sync(FULL, mbar_test(&xempty[in.i], par))) {
                            while (behind > 0) signal();
                            const bool w = mbar_wait(&xempty[in.i], par, a.budget, a.c.slots.st);
                            if (!__all_sync(FULL, w)) {
                                ok = false;
                                break;
                            }
                        }
                    }
                    uint8_t* dst = sX + in.i * X_BLOCK + (piece >> 3) * X_CHUNK;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint8_t* d = dst + sw128_offset((uint32_t)(16 * lw + 2 * j + half), (uint32_t)(piece & 7));
                        if (from[j])
                            cp_async16(d, from[j] + db * 256 + piece * 16);
                        else
                            *reinterpret_cast<uint4*>(d) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    cp_async_commit();
                    in.next(X_RING);
                    if (++behind > 3) signal();               // three blocks stay in flight
                }
            }
        }
        while (ok && behind > 0) signal();
        cp_async_wait_all();
    } else {
        // ============================ drain ============================
        const int qd = warp & 3;
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        // after the exchanges below lane l stores 8 dims (its group of 8 lanes') of the slots
        // s = 8 (l & 7 with its three bits reversed) .. + 7 of the tile
        const int sg = ((lane & 1) << 2) | (lane & 2) | ((lane & 4) >> 2);
        const int d0 = 32 * qd + (lane & 24);
        uint8_t* part = reinterpret_cast<uint8_t*>(a.c.part);
        const uint32_t row_bytes = (uint32_t)a.n_pass * BT_C * 2;
        Ring dk;
        int n = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            float* dqh = a.dqh + i * (int64_t)(BT_H * BT_C) + 32 * qd + lane;
            if (it.nt == 0) {
                for (int k = 0; k < BT_H * 4; ++k) dqh[(k >> 2) * BT_C + (k & 3) * 128] = 0.0f;
                continue;
            }
            uint8_t* base = part + it.pass * (BT_C * 2) + d0 * 2;
            for (int tt = 0; tt < it.nt && ok; ++tt) {
                // places of the tile's slots: slot s in register s >> 5 of lane s & 31
                int pl2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int slot, pl = -1;
                    const int64_t row = row_of(a, it, (it.t0 + tt) * BT_TILE + 32 * j + lane, &slot);
                    if (row >= 0)
                        pl = (int)(a.c.blk[row / BWD_SCAN_ROWS] + a.c.base[(int64_t)(it.q / a.c.group_q) * a.c.rows + row]) +
                             a.c.rank[(int64_t)it.q * a.c.n_slots + slot];
                    pl2[j] = pl;
                }
                for (int db = 0; db < 4; ++db) {
                    const bool w = mbar_wait(&dkfull[dk.i], dk.round & 1, a.budget, a.c.slots.st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t lo[32], hi[32];
                    tmem_ld32(tmem + lane_base + COL_DK + dk.i * BT_TILE, lo);
                    tmem_ld32(tmem + lane_base + COL_DK + dk.i * BT_TILE + 32, hi);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&dkempty[dk.i]);
                    dk.next(DK_RING);
                    // lane = dim, registers = slots -> 16-byte stores of 8 dims: lanes one, two and
                    // four apart swap the halves they do not keep (as bf16 pairs from the first
                    // swap on)
                    uint32_t u[32], v[16][2], x[8][4];
                    const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {            // slots k (even lanes), 32 + k (odd)
                        const uint32_t keep = b0 ? hi[k] : lo[k], got = __shfl_xor_sync(FULL, b0 ? lo[k] : hi[k], 1);
                        u[k] = ag_pack_bf16x2(__uint_as_float(b0 ? got : keep), __uint_as_float(b0 ? keep : got));
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint32_t keep = b1 ? u[16 + k] : u[k], got = __shfl_xor_sync(FULL, b1 ? u[k] : u[16 + k], 2);
                        v[k][0] = b1 ? got : keep;
                        v[k][1] = b1 ? keep : got;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t keep = b2 ? v[8 + k][e] : v[k][e];
                            const uint32_t got = __shfl_xor_sync(FULL, b2 ? v[k][e] : v[8 + k][e], 4);
                            x[k][e] = b2 ? got : keep;
                            x[k][2 + e] = b2 ? keep : got;
                        }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int slot = 8 * sg + k;
                        const int p0 = __shfl_sync(FULL, pl2[0], slot & 31), p1 = __shfl_sync(FULL, pl2[1], slot & 31);
                        const int pl = slot & 32 ? p1 : p0;
                        if (pl >= 0)
                            *reinterpret_cast<uint4*>(base + (uint64_t)(uint32_t)pl * row_bytes + db * 256) =
                                make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
                    }
                }
            }
            if (!ok) break;
            const bool w = mbar_wait(dqfull, n & 1, a.budget, a.c.slots.st);
            if (!__all_sync(FULL, w)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_base + COL_DQ + 32 * k, o);
                tmem_wait_ld();
                float* d = dqh + (int64_t)(32 * (k & 1)) * BT_C + (k >> 1) * 128;
#pragma unroll
                for (int h = 0; h < 32; ++h) d[h * BT_C] = __uint_as_float(o[h]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dqempty);
            ++n;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

}  // namespace

bool bwd_tc_applies(csa2_dtype q_dt, csa2_dtype kv_dt, int k, csa2_dtype swa_dt, int window, csa2_dtype out_dt,
                    unsigned flags) {
    return q_dt == CSA2_BF16 && (k == 0 || kv_dt == CSA2_BF16) && (window == 0 || swa_dt == CSA2_BF16) &&
           out_dt == CSA2_BF16 && (flags & (CSA2_QNORM | CSA2_KVNORM)) == (CSA2_QNORM | CSA2_KVNORM);
}

void bwd_tc_splits(int num_sms, int64_t queries, int n_slots, int* n_split, int* tps) {
    // as many key splits as keep every (query, split) item in one wave of CTAs
    const int tiles = std::max(1, (n_slots + BT_TILE - 1) / BT_TILE);
    const int want = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, num_sms / std::max<int64_t>(1, queries)));
    *tps = (tiles + want - 1) / want;
    *n_split = (tiles + *tps - 1) / *tps;
}

size_t bwd_tc_image_bytes() { return IMG_BYTES; }

csa2_status bwd_tc_chunk(csa2_ctx* ctx, BwdTcArgs& a, const void* dout, const void* out, float* D, uint8_t* img,
                         cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (ctx->device & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        CSA2_CHECK_CUDA(cudaFuncSetAttribute(attn_bwd_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    const BwdChunk& c = a.c;
    bwd_tc_prep_kernel<<<dim3((unsigned)(8 * a.n_pass), (unsigned)c.nb), 256, 0, s>>>(
        reinterpret_cast<const __nv_bfloat16*>(c.q), reinterpret_cast<const __nv_bfloat16*>(dout),
        reinterpret_cast<const __nv_bfloat16*>(out), c.slots.q_pos, c.bq0, c.nb, c.H, c.rope, c.flags, img, D);
    a.img = img;
    a.items = (int64_t)c.nb * a.n_pass * a.n_split;
    a.budget = WAIT_BUDGET;
    a.stall = 0;
    if (ctx->stall_next) {
        a.stall = 1;
        if (ctx->stall_budget > 0) a.budget = ctx->stall_budget;
        ctx->stall_next = 0;
    }
    const int64_t grid = std::min<int64_t>(a.items, ctx->num_sms);
    attn_bwd_tc_kernel<<<(unsigned)grid, BT_THREADS, SMEM_BYTES, s>>>(a);
    const int64_t heads = (int64_t)c.nb * c.H;
    bwd_tc_dq_kernel<<<(unsigned)((heads + 7) / 8), 256, 0, s>>>(a, a.dqh, reinterpret_cast<__nv_bfloat16*>(c.dq));
    return csa2_launch_status();
}
