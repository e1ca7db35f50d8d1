// Accumulated attention weight on the tcgen05 tensor cores (attn_mass.cu has the formulas):
// bf16 or FP4 rows, any flags, head passes of 64.
//
// The weights are fp32 results, so q^ enters the product as two bf16 numbers, hi = bf16(q^) and
// lo = bf16(q^ - hi) (2^-17 of q^ is left out).  They are the two halves of one operand: an
// image of 128 rows, hi of the 64 heads and then lo, so
//   [Z_hi  Z_lo] [128 slots x 128] = X . image^T
// is one MMA of N = 128 per 16 dims, which costs what N = 64 would.  The image stays in shared
// memory for a (query, head pass); the key rows X stream through a ring of three 128-dim blocks
// and are read once.  A softmax thread has a slot: it adds the two partial logits of each head,
// takes exp(z - lse) and sums over the heads, all in its own registers.  (With the heads in the
// lanes the sums went through shuffles and shared memory: 478 us for 4,096 queries of 512 slots.)
//
// Bound by the MMAs (32 a tile of 128 slots, 2,400 cycles) and, at about the same rate, by the
// rows' way from L2 (128 KB a tile).  An image is rewritten 64 dims at a time, behind the last
// tile that reads it, so that neither waits for the other's whole.
//
// Warp roles (one CTA per SM, persistent over items = (query, range of tiles)):
//   warps 0-3    softmax
//   warp 4       MMA issuer; owns the tensor memory (a ring of four [128 x 128] accumulators)
//   warps 5-12   image: norm, rotation, hi and lo of 8 heads each
//   warps 13-18  loaders, bf16 rows: 16-byte cp.async, a warp half of one block of the ring
//   warps 13-20  loaders, FP4 rows: a thread per slot, two groups of four warps in turn
// Every wait is bounded; a wait that expires flags a timeout and the roles wind down.
#include <algorithm>
#include <atomic>

#include "attn_mass.cuh"
#include "fp4_tile.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace sm100;

constexpr int MT_C = 512;
constexpr int MT_H = 64;
constexpr int MT_TILE = 128;
constexpr int CHUNK = 128 * 128;                 // 128 rows x 64 dims, image and tile alike
constexpr int BLOCK = 2 * CHUNK;                 // 128 dims
constexpr int X_RING = 3;
constexpr int S_RING = 4;
constexpr long long WAIT_BUDGET = 1ll << 31;
constexpr unsigned FULL = 0xffffffffu;
constexpr int threads_of(bool fp4) { return fp4 ? 672 : 608; }

constexpr int OFF_IMG = 0;
constexpr int OFF_X = OFF_IMG + 4 * BLOCK;
constexpr int OFF_RINV = OFF_X + X_RING * BLOCK;         // FP4: [2][128] RMS factors
constexpr int OFF_LSE = OFF_RINV + 2 * MT_TILE * 4;      // [4 warps][64 heads] -lse (base 2)
constexpr int OFF_BAR = OFF_LSE + 4 * MT_H * 4;
constexpr int N_BAR = 8 + 8 + 2 * X_RING + 2 * S_RING + 4 + 1;
constexpr int OFF_TMEMPTR = OFF_BAR + N_BAR * 8;
constexpr int SMEM_BYTES = OFF_TMEMPTR + 16;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

struct MassTcArgs {
    MassArgs m;
    int n_pass, n_split, tps;
    uint32_t items;
    long long budget;
    int stall;
};

struct Item {
    int64_t bq, kv0;
    int n, t0, nt;               // cache slots; tiles t0 .. t0 + nt - 1
};

__device__ __forceinline__ Item item_of(const MassTcArgs& a, uint32_t i) {
    Item r;
    const uint32_t bq = i / (uint32_t)a.n_split;
    r.bq = bq;
    const int split = (int)(i - bq * a.n_split);
    const SlotArgs& s = a.m.slots;
    r.n = s.dense_nv ? (int)max((int64_t)0, min((int64_t)s.k, s.dense_nv[r.bq])) : s.k;
    r.kv0 = (int64_t)(bq / (uint32_t)s.Q) * s.N;
    // all of the row's tiles: slots past a dense row's end are written as 0 too
    const int tiles = (s.k + MT_TILE - 1) / MT_TILE;
    r.t0 = split * a.tps;
    r.nt = max(0, min(tiles, r.t0 + a.tps) - r.t0);
    return r;
}

// Cache row of slot s, -1 if it is empty; an entry outside the cache is flagged if asked.
__device__ __forceinline__ int64_t row_of(const SlotArgs& a, const Item& it, int s, bool flag) {
    if (s >= it.n) return -1;
    const int id = a.dense_nv ? s : a.idx[it.bq * a.k + s];
    if (id < 0) return -1;
    if (id >= a.N) {
        if (flag) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
        return -1;
    }
    return it.kv0 + id;
}

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

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// RMS factors of the bf16 rows that the warp's lanes hold (row, -1 = none) from the rows
// themselves, eight at a time; a warp reads a row in two 512-byte pieces.
__device__ __forceinline__ float factors_of(const uint8_t* kv, int64_t row, int lane) {
    float mine = 0.0f;
#pragma unroll 1
    for (int j0 = 0; j0 < 32; j0 += 8) {
        uint4 v[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t r = __shfl_sync(FULL, row, j0 + j);
            const uint4* p = reinterpret_cast<const uint4*>(kv + max(r, (int64_t)0) * (MT_C * 2)) + lane;
#pragma unroll
            for (int e = 0; e < 2; ++e) v[j][e] = r >= 0 ? p[32 * e] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w[4] = {v[j][e].x, v[j][e].y, v[j][e].z, v[j][e].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = __uint_as_float(w[k] << 16), y = __uint_as_float(w[k] & 0xFFFF0000u);
                    ss = fmaf(x, x, ss);
                    ss = fmaf(y, y, ss);
                }
            }
            ss = warp_sum(ss);
            if (lane == j0 + j) mine = ag_rms_factor(ss);
        }
    }
    return mine;
}

template <typename TQ, bool FP4>
__global__ void __launch_bounds__(threads_of(FP4), 1) mass_tc_kernel(const MassTcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sImg = smem + OFF_IMG;
    uint8_t* sX = smem + OFF_X;
    float* sRinv = reinterpret_cast<float*>(smem + OFF_RINV);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* imgfull = bars;                       // [8] 64 dims of the image
    uint64_t* imgempty = bars + 8;                  // [8]
    uint64_t* xfull = bars + 16;                    // [X_RING]
    uint64_t* xempty = xfull + X_RING;              // [X_RING]
    uint64_t* sfull = xempty + X_RING;              // [S_RING]
    uint64_t* sempty = sfull + S_RING;              // [S_RING]
    uint64_t* rfull = sempty + S_RING;              // [2] FP4: RMS factors of a tile
    uint64_t* rempty = rfull + 2;                   // [2]
    uint64_t* alldone = rempty + 2;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEMPTR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* st = a.m.slots.st;

    if (smem_u32(smem) & 1023u) {                   // the operand tiles' layout needs it (never seen)
        if (threadIdx.x == 0) csa2_flag(st, CSA2_DEVBIT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&imgfull[i], 8);
            mbar_init(&imgempty[i], 1);
        }
        for (int i = 0; i < X_RING; ++i) {
            mbar_init(&xfull[i], FP4 ? 4 : 2);
            mbar_init(&xempty[i], 1);
        }
        for (int i = 0; i < S_RING; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&rfull[i], 4);
            mbar_init(&rempty[i], 4);
        }
        mbar_init(alldone, 1);
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(sTmem, 512);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sTmem;

    if (warp < 4) {
        // ============================ softmax ============================
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        float* nl = reinterpret_cast<float*>(smem + OFF_LSE) + warp * MT_H;
        const float c1 = AG_LOG2E / sqrtf((float)MT_C);
        const SlotArgs& sl = a.m.slots;
        float* wrow = a.m.weights ? a.m.weights : a.m.passes;
        uint32_t g = 0;                                       // tiles so far
        Ring sr;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            for (int pass = 0; pass < a.n_pass && ok; ++pass) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = pass * MT_H + 32 * j + lane;
                    const float l = h < a.m.H ? a.m.lse[it.bq * a.m.H + h] : -INFINITY;
                    // heads past H, and queries of no key, count 0
                    nl[32 * j + lane] = l != -INFINITY ? -l * AG_LOG2E : -INFINITY;
                }
                __syncwarp();
                int64_t next = row_of(sl, it, it.t0 * MT_TILE + 32 * warp + lane, pass == 0);
                for (int tt = 0; tt < it.nt; ++tt, ++g) {
                    const int own = (it.t0 + tt) * MT_TILE + 32 * warp + lane;      // this thread's slot
                    const int64_t row = next;
                    float r = 1.0f;
                    if (!FP4 && (a.m.flags & CSA2_KVNORM)) {
                        if (a.m.rinv)
                            r = row >= 0 ? a.m.rinv[row] : 1.0f;
                        else
                            r = factors_of(reinterpret_cast<const uint8_t*>(a.m.kv), row, lane);
                    }
                    if (tt + 1 < it.nt) next = row_of(sl, it, own + MT_TILE, pass == 0);
                    bool w = mbar_wait(&sfull[sr.i], sr.round & 1, a.budget, st);
                    if (FP4) w = w && mbar_wait(&rfull[g & 1], (g >> 1) & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (FP4) {
                        r = sRinv[(g & 1) * MT_TILE + 32 * warp + lane];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&rempty[g & 1]);
                    }
                    const float rz = r * c1;
                    const uint32_t at = tmem + lane_base + sr.i * MT_TILE;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {             // 16 heads
                        uint32_t hi[16], lo[16];
                        tmem_ld16(at + 16 * q, hi);
                        tmem_ld16(at + 64 + 16 * q, lo);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 l4 = *reinterpret_cast<const float4*>(nl + 16 * q + 4 * j);
                            const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                sum[k] += ex2_approx(fmaf(__uint_as_float(hi[4 * j + k]) + __uint_as_float(lo[4 * j + k]), rz, l[k]));
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sempty[sr.i]);
                    sr.next(S_RING);
                    if (own < sl.k) {
                        float t = row >= 0 ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.0f;
                        if (pass > 0) t += wrow[it.bq * sl.k + own];
                        if (wrow) wrow[it.bq * sl.k + own] = t;
                        if (a.m.acc && row >= 0 && pass == a.n_pass - 1) add_mass(a.m.acc, a.m.fix, row, t);
                    }
                }
            }
        }
    } else if (warp == 4) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            constexpr uint32_t ID = idesc_f16(128, MT_TILE, true);
            const uint32_t img = smem_u32(sImg), x0 = smem_u32(sX);
            Ring xr, sr;
            int n = 0;                                        // images so far
            bool ok = true;
            auto wait = [&](uint64_t* b, uint32_t par) {
                ok = ok && mbar_wait(b, par, a.budget, st);
                return ok;
            };
            for (uint32_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
                const Item it = item_of(a, i);
                for (int pass = 0; pass < a.n_pass && ok && it.nt > 0; ++pass, ++n) {
                    for (int tt = 0; tt < it.nt && ok; ++tt) {
                        if (sr.round > 0 && !wait(&sempty[sr.i], (sr.round - 1) & 1)) break;
                        for (int db = 0; db < 4; ++db) {
                            if (tt == 0 && (!wait(&imgfull[2 * db], n & 1) || !wait(&imgfull[2 * db + 1], n & 1))) break;
                            if (!wait(&xfull[xr.i], xr.round & 1)) break;
                            tc_fence_after();
                            const uint64_t da = sdesc_sw128(img + db * BLOCK), dx = sdesc_sw128(x0 + xr.i * BLOCK);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint64_t o = ((kk >> 2) * CHUNK + (kk & 3) * 32) >> 4;
                                mma_ss(tmem + sr.i * MT_TILE, dx + o, da + o, ID, (db | kk) != 0);
                                if (kk == 3 && tt == it.nt - 1) mma_commit(&imgempty[2 * db]);
                            }
                            if (tt == it.nt - 1) mma_commit(&imgempty[2 * db + 1]);
                            mma_commit(&xempty[xr.i]);
                            xr.next(X_RING);
                        }
                        if (!ok) break;
                        mma_commit(&sfull[sr.i]);
                        sr.next(S_RING);
                    }
                }
            }
            // the MMAs must be complete before tensor memory is released
            mma_commit(alldone);
            mbar_wait(alldone, 0, a.budget, st);
        }
    } else if (warp < 13) {
        // ============================ images ============================
        const int iw = warp - 5;
        const TQ* q = reinterpret_cast<const TQ*>(a.m.q);
        int n = 0;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < a.items && ok && !a.stall; i += gridDim.x) {
            const Item it = item_of(a, i);
            if (it.nt == 0) continue;
            const int64_t t = a.m.slots.q_pos[it.bq];
            float c1 = 1.0f, s1 = 0.0f;                       // lane j: angle j (64-bit arithmetic: one a lane)
            if (a.m.flags & CSA2_ROPE) ag_cos_sin(a.m.rope, t, lane, c1, s1);
            for (int pass = 0; pass < a.n_pass && ok; ++pass, ++n) {
                // this warp's 8 heads, four lanes a head: 16 of a chunk's 64 dims each.  The sum of
                // squares first, then chunk by chunk, AHEAD of them on their way.
                constexpr int NW = sizeof(TQ);                // 16-byte words of 16 channels
                constexpr int AHEAD = 8 / NW;
                const int part = lane & 3, hl = 8 * iw + (lane >> 2), h = pass * MT_H + hl;
                const bool there = h < a.m.H;
                const uint4* src = reinterpret_cast<const uint4*>(q + (it.bq * a.m.H + (there ? h : 0)) * (int64_t)MT_C + 16 * part);
                uint4 nx[AHEAD][NW];
                auto load = [&](int c, uint4 (&x)[NW]) {
#pragma unroll
                    for (int k = 0; k < NW; ++k) x[k] = src[c * 4 * NW + k];
                };
                float f = 1.0f;
                if (a.m.flags & CSA2_QNORM) {
                    float ss = 0.0f;
#pragma unroll 1
                    for (int c0 = 0; c0 < 8; c0 += AHEAD) {
#pragma unroll
                        for (int j = 0; j < AHEAD; ++j) load(c0 + j, nx[j]);
#pragma unroll
                        for (int j = 0; j < AHEAD; ++j) {
                            float v[16];
                            ag_load16<TQ>(reinterpret_cast<const TQ*>(nx[j]), v);
                            ss += ag_sumsq16(v);
                        }
                    }
                    ss += __shfl_xor_sync(FULL, ss, 1);
                    ss += __shfl_xor_sync(FULL, ss, 2);
                    f = ag_rms_factor(ss);
                }
                if (!there) f = 0.0f;
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) load(j, nx[j]);
#pragma unroll 1
                for (int c0 = 0; c0 < 8 && ok; c0 += AHEAD) {
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) {
                        const int c = c0 + j;
                        float v[16];
                        ag_load16<TQ>(reinterpret_cast<const TQ*>(nx[j]), v);
                        if (c + AHEAD < 8) load(c + AHEAD, nx[j]);
                        uint32_t ph[8], pl[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float x0 = there ? v[2 * k] * f : 0.0f, x1 = there ? v[2 * k + 1] * f : 0.0f;
                            if (j == AHEAD - 1 && c == 7 && (a.m.flags & CSA2_ROPE)) {      // the last 64 channels
                                const float co = __shfl_sync(FULL, c1, 8 * part + k), si = __shfl_sync(FULL, s1, 8 * part + k);
                                const float y0 = x0 * co - x1 * si;
                                x1 = x1 * co + x0 * si;
                                x0 = y0;
                            }
                            ph[k] = ag_pack_bf16x2(x0, x1);
                            pl[k] = ag_pack_bf16x2(x0 - __uint_as_float(ph[k] << 16), x1 - __uint_as_float(ph[k] & 0xFFFF0000u));
                        }
                        if (n > 0) {
                            const bool w = mbar_wait(&imgempty[c], (n - 1) & 1, a.budget, st);
                            if (!__all_sync(FULL, w)) {
                                ok = false;
                                break;
                            }
                        }
                        uint8_t* d = sImg + c * CHUNK;
                        const uint32_t u = 2u * part;
                        *reinterpret_cast<uint4*>(d + sw128_offset(hl, u)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                        *reinterpret_cast<uint4*>(d + sw128_offset(hl, u + 1)) = make_uint4(ph[4], ph[5], ph[6], ph[7]);
                        *reinterpret_cast<uint4*>(d + sw128_offset(64 + hl, u)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                        *reinterpret_cast<uint4*>(d + sw128_offset(64 + hl, u + 1)) = make_uint4(pl[4], pl[5], pl[6], pl[7]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&imgfull[c]);
                    }
                }
            }
        }
    } else if (FP4) {
        // ============================ loaders, FP4 rows ============================
        const int lt = threadIdx.x - 416, grp = lt >> 7, r = lt & 127;
        const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.m.kv);
        Ring xr;
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            for (int tp = 0; tp < it.nt * a.n_pass && ok; ++tp, ++g) {
                const int tt = tp % it.nt;
                if ((int)(g & 1) != grp) {                    // the other group's tile
                    for (int db = 0; db < 4; ++db) xr.next(X_RING);
                    continue;
                }
                const int64_t row = row_of(a.m.slots, it, (it.t0 + tt) * MT_TILE + r, false);
                const uint8_t* src = kv + row * fp4_row_bytes(MT_C);
                uint4 code[4];
                uint2 sc = make_uint2(0u, 0u);
                auto fetch = [&](int db) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) code[k] = make_uint4(0u, 0u, 0u, 0u);
                    sc = make_uint2(0u, 0u);
                    if (row >= 0) {
                        const uint4* p = reinterpret_cast<const uint4*>(src + 64 * db);
#pragma unroll
                        for (int k = 0; k < 4; ++k) code[k] = p[k];
                        sc = *reinterpret_cast<const uint2*>(src + 256 + 8 * db);
                    }
                };
                fetch(0);
                // Once the tile before is written whole, every place of the ring has been emptied as
                // often as the waits below take for granted, but for the last time: no parity of
                // theirs can be taken for the one two rounds ago.
                if (g > 0) {
                    const bool w = mbar_wait(&rfull[(g - 1) & 1], ((g - 1) >> 1) & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                }
                float ss = 0.0f;
                for (int db = 0; db < 4; ++db) {
                    uint4 c0 = code[0], c1 = code[1], c2 = code[2], c3 = code[3];
                    const uint2 s0 = sc;
                    if (db < 3) fetch(db + 1);                // in flight during this block
                    if (xr.round > 0) {
                        const bool w = mbar_wait(&xempty[xr.i], (xr.round - 1) & 1, a.budget, st);
                        if (!__all_sync(FULL, w)) {
                            ok = false;
                            break;
                        }
                    }
                    ss += fp4_block_to_tile<CHUNK>(c0, c1, c2, c3, s0.x, s0.y, sX + xr.i * BLOCK, 0, r);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&xfull[xr.i]);
                    xr.next(X_RING);
                }
                if (!ok) break;
                const int rb = g & 1;
                if (g >= 2) {
                    const bool w = mbar_wait(&rempty[rb], ((g >> 1) - 1) & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                }
                sRinv[rb * MT_TILE + r] = row < 0 ? -1.0f : (a.m.flags & CSA2_KVNORM) ? ag_rms_factor(ss) : 1.0f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&rfull[rb]);
            }
        }
    } else {
        // ============================ loaders, bf16 rows ============================
        // A warp fills one half (64 dims) of one block of the ring, every third block.
        const int w6 = warp - 13, x = w6 >> 1, half = w6 & 1;
        const int sub = lane >> 3, piece = lane & 7;          // a copy moves 128 bytes of four rows
        const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.m.kv) + half * 128 + piece * 16;
        // rows 8 apart have the same swizzle
        uint8_t* dst0 = sX + x * BLOCK + half * CHUNK + sw128_offset((uint32_t)sub, (uint32_t)piece);
        uint8_t* dst4 = sX + x * BLOCK + half * CHUNK + sw128_offset((uint32_t)(sub + 4), (uint32_t)piece);
        uint32_t b = 0, c = 0;                                // blocks of the stream; filled by this warp
        bool ok = true;
        for (uint32_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            // a slot's entry, or -1; read a tile ahead
            int code[4], next[4];
            auto look = [&](int tt, int (&o)[4]) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int s = (it.t0 + tt) * MT_TILE + 32 * q + lane;
                    o[q] = s >= it.n ? -1 : a.m.slots.dense_nv ? s : a.m.slots.idx[it.bq * a.m.slots.k + s];
                }
            };
            if (it.nt > 0) look(0, next);
            for (int tp = 0; tp < it.nt * a.n_pass && ok; ++tp) {
#pragma unroll
                for (int q = 0; q < 4; ++q) code[q] = next[q] >= 0 && next[q] < a.m.slots.N ? next[q] : -1;
                if (tp + 1 < it.nt * a.n_pass) look((tp + 1) % it.nt, next);
#pragma unroll 1
                for (int db = 0; db < 4; ++db, ++b) {
                    if (b % X_RING != x) continue;
                    bool w = true;
                    if (c > 0) w = mbar_wait(&xempty[x], (c - 1) & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                    ++c;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {             // eight addresses, then eight copies
                        const uint8_t* src[8];
                        bool read[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int o = __shfl_sync(FULL, code[q], 4 * j + sub);
                            read[j] = o >= 0;
                            src[j] = kv + ((it.kv0 + max(o, 0)) * (MT_C * 2) + db * 256);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            cp_async16_or_zero((j & 1 ? dst4 : dst0) + (4 * q + (j >> 1)) * 1024, src[j], read[j]);
                    }
                    cp_async_wait_all();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&xfull[x]);
                }
            }
        }
        cp_async_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, 512);
}

template <typename TQ, bool FP4>
csa2_status launch(csa2_ctx* ctx, const MassTcArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (ctx->device & 63);
    auto kern = mass_tc_kernel<TQ, FP4>;
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        CSA2_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES));
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t grid = std::min<int64_t>(a.items, ctx->num_sms);
    kern<<<(unsigned)grid, threads_of(FP4), SMEM_BYTES, s>>>(a);
    return csa2_launch_status();
}

}  // namespace

csa2_status mass_tc_run(csa2_ctx* ctx, const MassArgs& m, cudaStream_t s) {
    MassTcArgs a;
    a.m = m;
    a.n_pass = (m.H + MT_H - 1) / MT_H;
    // as many ranges of tiles as keep every (query, range) item in one wave of CTAs
    const int tiles = (m.slots.k + MT_TILE - 1) / MT_TILE;
    const int want = (int)std::min<int64_t>(tiles, std::max<int64_t>(1, ctx->num_sms / m.n_bq));
    a.tps = (tiles + want - 1) / want;
    a.n_split = (tiles + a.tps - 1) / a.tps;
    a.items = (uint32_t)m.n_bq * a.n_split;
    a.budget = WAIT_BUDGET;
    a.stall = 0;
    if (ctx->stall_next) {
        a.stall = 1;
        if (ctx->stall_budget > 0) a.budget = ctx->stall_budget;
        ctx->stall_next = 0;
    }
    const bool fp4 = m.kv_dt == CSA2_FP4_E4M3x16;
    if (m.q_dt == CSA2_F32) return fp4 ? launch<float, true>(ctx, a, s) : launch<float, false>(ctx, a, s);
    return fp4 ? launch<__nv_bfloat16, true>(ctx, a, s) : launch<__nv_bfloat16, false>(ctx, a, s);
}
