// Accumulated attention weight on the tcgen05 tensor cores (attn_mass.cu has the formulas):
// bf16 or FP4 rows, any flags, head passes of 64.
//
// The weights are fp32 results, so q^ enters the product as two bf16 numbers, hi = bf16(q^) and
// lo = bf16(q^ - hi) (2^-17 of q^ is left out).  They are the two halves of one operand: an
// image of 128 stacked rows, hi and lo of the 64 heads interleaved 16 by 16, so one MMA of
// M = 128, N = 128 slots makes both partial logits of a head, 16 lanes apart, and costs what
// N = 64 would.  The image stays in shared memory for a (query, head pass); the key rows stream
// through a ring of three 128-dim blocks and are read once.  Per tile of 128 slots the softmax
// warps add the two partial logits, take exp(z - lse), and sum over the heads (a butterfly over
// a warp's 16 heads, then the four warps).
//
// Bound by shared memory: the MMAs of a tile read 256 KB (32 at 39.5 ns would be 1.27 us), the
// copies write 128 KB, 3,072 cycles of the 128-byte port (1.6 us).  So the rows' squares are not
// taken from there when rows are gathered many times over: a table of RMS factors is made once.
//
// Warp roles (672 threads, one CTA per SM, persistent over items = (query, range of tiles)):
//   warps 0-3    softmax: one thread per stacked row; owns one slot of the tile's result
//   warp 4       MMA issuer; owns the tensor memory (a ring of four [128 x 128] accumulators)
//   warps 5-12   image: norm, rotation, hi and lo of 8 heads each, loaded while the previous
//                image is in use
//   warps 13-20  loaders: bf16 rows by 16-byte cp.async, a warp 16 slots of every tile; FP4 rows a
//                thread per slot, the two groups of four warps taking tiles in turn
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
constexpr int MT_THREADS = 672;
constexpr int CHUNK = 128 * 128;                 // 128 rows x 64 dims, image and tile alike
constexpr int BLOCK = 2 * CHUNK;                 // 128 dims
constexpr int X_RING = 3;
constexpr int S_RING = 4;
constexpr long long WAIT_BUDGET = 1ll << 31;
constexpr unsigned FULL = 0xffffffffu;

constexpr int OFF_IMG = 0;
constexpr int OFF_X = OFF_IMG + 4 * BLOCK;
constexpr int OFF_RINV = OFF_X + X_RING * BLOCK;         // [2][128] RMS factors, -1 = empty slot
constexpr int OFF_RED = OFF_RINV + 2 * MT_TILE * 4;      // [4 owners][3 other warps][32] partial sums
constexpr int OFF_BAR = OFF_RED + 4 * 3 * 32 * 4;
constexpr int N_BAR = 2 + 2 * X_RING + 2 * S_RING + 4 + 2 + 1;
constexpr int OFF_TMEMPTR = OFF_BAR + N_BAR * 8;
constexpr int SMEM_BYTES = OFF_TMEMPTR + 16;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

struct MassTcArgs {
    MassArgs m;
    int n_pass, n_split, tps;
    int64_t items;
    long long budget;
    int stall;
};

struct Item {
    int64_t bq, kv0;
    int n, t0, nt;               // cache slots; tiles t0 .. t0 + nt - 1
};

__device__ __forceinline__ Item item_of(const MassTcArgs& a, int64_t i) {
    Item r;
    r.bq = i / a.n_split;
    const int split = (int)(i - r.bq * a.n_split);
    const SlotArgs& s = a.m.slots;
    r.n = s.dense_nv ? (int)max((int64_t)0, min((int64_t)s.k, s.dense_nv[r.bq])) : s.k;
    r.kv0 = (r.bq / s.Q) * s.N;
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <typename TQ, bool FP4>
__global__ void __launch_bounds__(MT_THREADS, 1) mass_tc_kernel(const MassTcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sImg = smem + OFF_IMG;
    uint8_t* sX = smem + OFF_X;
    float* sRinv = reinterpret_cast<float*>(smem + OFF_RINV);
    float* sRed = reinterpret_cast<float*>(smem + OFF_RED);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* imgfull = bars;
    uint64_t* imgempty = bars + 1;
    uint64_t* xfull = bars + 2;                     // [X_RING]
    uint64_t* xempty = xfull + X_RING;              // [X_RING]
    uint64_t* sfull = xempty + X_RING;              // [S_RING]
    uint64_t* sempty = sfull + S_RING;              // [S_RING]
    uint64_t* rfull = sempty + S_RING;              // [2]
    uint64_t* rempty = rfull + 2;                   // [2]
    uint64_t* redfull = rempty + 2;                 // the softmax warps' sums are in sRed / have been read
    uint64_t* redempty = redfull + 1;
    uint64_t* alldone = redfull + 2;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEMPTR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* st = a.m.slots.st;

    if (smem_u32(smem) & 1023u) {                   // the operand tiles' layout needs it (never seen)
        if (threadIdx.x == 0) csa2_flag(st, CSA2_DEVBIT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(imgfull, 8);
        mbar_init(imgempty, 1);
        for (int i = 0; i < X_RING; ++i) {
            mbar_init(&xfull[i], FP4 ? 4 : 8);
            mbar_init(&xempty[i], 1);
        }
        for (int i = 0; i < S_RING; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&rfull[i], FP4 ? 4 : 8);
            mbar_init(&rempty[i], 4);
        }
        mbar_init(redfull, 4);
        mbar_init(redempty, 4);
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
        const int hl = 16 * warp + (lane & 15);               // head of the pass
        const bool up = lane & 16;                            // this lane's slots: 64 .. 127 of the tile
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const float c1 = AG_LOG2E / sqrtf((float)MT_C);
        uint32_t g = 0;                                       // tiles so far
        Ring sr;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            float* wrow = (a.m.weights ? a.m.weights : a.m.passes);
            for (int pass = 0; pass < a.n_pass && ok; ++pass) {
                const int h = pass * MT_H + hl;
                float lse2 = INFINITY;                        // heads past H, and queries of no key, count 0
                if (h < a.m.H) {
                    const float l = a.m.lse[it.bq * a.m.H + h];
                    if (l != -INFINITY) lse2 = l * AG_LOG2E;
                }
                const bool count = lse2 != INFINITY;
                for (int tt = 0; tt < it.nt; ++tt, ++g) {
                    const int own = (it.t0 + tt) * MT_TILE + 32 * warp + lane;      // the slot this thread reports
                    const int64_t row = own < a.m.slots.k ? row_of(a.m.slots, it, own, pass == 0) : -1;
                    const int rb = g & 1;
                    bool w = mbar_wait(&rfull[rb], (g >> 1) & 1, a.budget, st) &&
                             mbar_wait(&sfull[sr.i], sr.round & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float* rv = sRinv + rb * MT_TILE + (up ? 64 : 0);
                    if (g > 0) {
                        w = mbar_wait(redempty, (g - 1) & 1, a.budget, st);
                        if (!__all_sync(FULL, w)) {
                            ok = false;
                            break;
                        }
                    }
                    float mine = 0.0f;
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {             // slots (up ? 64 : 0) + 16 b ..
                        uint32_t lo[16], hi[16];
                        tmem_ld16(tmem + lane_base + sr.i * MT_TILE + 16 * b, lo);
                        tmem_ld16(tmem + lane_base + sr.i * MT_TILE + 64 + 16 * b, hi);
                        tmem_wait_ld();
                        float p[16];
#pragma unroll
                        for (int c4 = 0; c4 < 4; ++c4) {
                            const float4 r4 = *reinterpret_cast<const float4*>(rv + 16 * b + 4 * c4);
                            const float rr[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int c = 4 * c4 + k;
                                const float z = __uint_as_float(up ? hi[c] : lo[c]) +
                                                __uint_as_float(__shfl_xor_sync(FULL, up ? lo[c] : hi[c], 16));
                                p[c] = count && rr[k] >= 0.0f ? ex2_approx(fmaf(z * rr[k], c1, -lse2)) : 0.0f;
                            }
                        }
                        // sum over the warp's 16 heads: every lane ends with one slot, 16 b + (lane & 15)
#pragma unroll
                        for (int d = 8; d >= 1; d >>= 1) {
                            const bool top = lane & d;
#pragma unroll
                            for (int k = 0; k < d; ++k) {
                                const float send = top ? p[k] : p[k + d], keep = top ? p[k + d] : p[k];
                                p[k] = keep + __shfl_xor_sync(FULL, send, d);
                            }
                        }
                        // the four warps' sums meet at the slot's owner
                        const int dest = (up ? 2 : 0) + (b >> 1);
                        if (dest != warp)
                            sRed[(dest * 3 + (warp < dest ? warp : warp - 1)) * 32 + 16 * (b & 1) + (lane & 15)] = p[0];
                        const float v = __shfl_sync(FULL, p[0], ((warp & 2) << 3) | (lane & 15));
                        if (b == 2 * (warp & 1) + (lane >> 4)) mine = v;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sempty[sr.i]);
                        mbar_arrive(&rempty[rb]);
                    }
                    sr.next(S_RING);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(redfull);
                    w = mbar_wait(redfull, g & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                    float t = 0.0f;
#pragma unroll
                    for (int o = 0; o < 4; ++o)
                        t += o == warp ? mine : sRed[(warp * 3 + (o < warp ? o : o - 1)) * 32 + lane];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(redempty);
                    if (own < a.m.slots.k) {
                        if (pass > 0) t += wrow[it.bq * a.m.slots.k + own];
                        if (wrow) wrow[it.bq * a.m.slots.k + own] = t;
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
            for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
                const Item it = item_of(a, i);
                for (int pass = 0; pass < a.n_pass && ok && it.nt > 0; ++pass, ++n) {
                    if (!wait(imgfull, n & 1)) break;
                    for (int tt = 0; tt < it.nt && ok; ++tt) {
                        if (sr.round > 0 && !wait(&sempty[sr.i], (sr.round - 1) & 1)) break;
                        for (int db = 0; db < 4; ++db) {
                            if (!wait(&xfull[xr.i], xr.round & 1)) break;
                            tc_fence_after();
                            const uint64_t da = sdesc_sw128(img + db * BLOCK), dx = sdesc_sw128(x0 + xr.i * BLOCK);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint64_t o = ((kk >> 2) * CHUNK + (kk & 3) * 32) >> 4;
                                mma_ss(tmem + sr.i * MT_TILE, da + o, dx + o, ID, (db | kk) != 0);
                            }
                            mma_commit(&xempty[xr.i]);
                            xr.next(X_RING);
                        }
                        if (!ok) break;
                        mma_commit(&sfull[sr.i]);
                        sr.next(S_RING);
                    }
                    if (ok) mma_commit(imgempty);
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
        for (int64_t i = blockIdx.x; i < a.items && ok && !a.stall; i += gridDim.x) {
            const Item it = item_of(a, i);
            if (it.nt == 0) continue;
            const int64_t t = a.m.slots.q_pos[it.bq];
            float c1 = 1.0f, s1 = 0.0f;                       // lane j: angle j (64-bit arithmetic: one a lane)
            if (a.m.flags & CSA2_ROPE) ag_cos_sin(a.m.rope, t, lane, c1, s1);
            for (int pass = 0; pass < a.n_pass && ok; ++pass, ++n) {
                // this warp's 8 heads, two at a time: half a warp a head, lane l its channels
                // 16 (l & 15) + 256 e, e = 0, 1.  The first two are loaded, the others are on their
                // way to L2, before the image is free.  (Kept small and not unrolled: a decode
                // call runs it once, from a cold instruction cache.)
                constexpr int NW = sizeof(TQ);                // 16-byte words of 16 channels, twice over / 2
                const int sub = lane >> 4, l16 = lane & 15;
                const int h0 = pass * MT_H + 8 * iw + sub;
                uint4 nx[2][NW];
                auto load = [&](int h) {
                    const uint4* src = reinterpret_cast<const uint4*>(q + (it.bq * a.m.H + h) * (int64_t)MT_C + 16 * l16);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int k = 0; k < NW; ++k)
                            nx[e][k] = h < a.m.H ? src[e * 16 * NW + k] : make_uint4(0u, 0u, 0u, 0u);
                };
                load(h0);
                for (int j = 2; j < 8; j += 2)
                    if (h0 + j < a.m.H) {
                        const TQ* src = q + (it.bq * a.m.H + h0 + j) * (int64_t)MT_C + 16 * l16;
                        prefetch_l2(src);
                        prefetch_l2(src + 256);
                    }
                if (n > 0) {
                    const bool w = mbar_wait(imgempty, (n - 1) & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                }
#pragma unroll 1
                for (int j = 0; j < 8; j += 2) {
                    float v[2][16];
#pragma unroll
                    for (int e = 0; e < 2; ++e) ag_load16<TQ>(reinterpret_cast<const TQ*>(nx[e]), v[e]);
                    if (j < 6) load(h0 + j + 2);
                    float f = ag_sumsq16(v[0]) + ag_sumsq16(v[1]);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) f += __shfl_xor_sync(FULL, f, o);
                    f = (a.m.flags & CSA2_QNORM) ? ag_rms_factor(f) : 1.0f;
                    const int hl = 8 * iw + j + sub;
                    const uint32_t r = 32u * (hl >> 4) + (hl & 15), u = 2u * (l16 & 3);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t ph[8], pl[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float x0 = v[e][2 * k] * f, x1 = v[e][2 * k + 1] * f;
                            if (e == 1) {                     // lanes l16 = 12 .. 15: channels 448 .. 511, pair 8 (l16 - 12) + k
                                const float c = __shfl_sync(FULL, c1, (8 * l16 + k) & 31);
                                const float s = __shfl_sync(FULL, s1, (8 * l16 + k) & 31);
                                if (l16 >= 12) {
                                    const float y0 = x0 * c - x1 * s;
                                    x1 = x1 * c + x0 * s;
                                    x0 = y0;
                                }
                            }
                            ph[k] = ag_pack_bf16x2(x0, x1);
                            pl[k] = ag_pack_bf16x2(x0 - __uint_as_float(ph[k] << 16),
                                                   x1 - __uint_as_float(ph[k] & 0xFFFF0000u));
                        }
                        uint8_t* c = sImg + ((l16 >> 2) + 4 * e) * CHUNK;
                        *reinterpret_cast<uint4*>(c + sw128_offset(r, u)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                        *reinterpret_cast<uint4*>(c + sw128_offset(r, u + 1)) = make_uint4(ph[4], ph[5], ph[6], ph[7]);
                        *reinterpret_cast<uint4*>(c + sw128_offset(r + 16, u)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                        *reinterpret_cast<uint4*>(c + sw128_offset(r + 16, u + 1)) = make_uint4(pl[4], pl[5], pl[6], pl[7]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(imgfull);
            }
        }
    } else if (FP4) {
        // ============================ loaders, FP4 rows ============================
        const int lt = threadIdx.x - 416, grp = lt >> 7, r = lt & 127;
        const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.m.kv);
        Ring xr;
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            for (int tp = 0; tp < it.nt * a.n_pass && ok; ++tp, ++g) {
                const int tt = tp % it.nt;
                if ((int)(g & 1) != grp) {
                    // the other group's tile: wait as it does, so that a later wait of this group's
                    // is never two rounds ahead of a ring slot
                    for (int db = 0; db < 4 && ok; ++db) {
                        if (xr.round > 0) {
                            const bool w = mbar_wait(&xempty[xr.i], (xr.round - 1) & 1, a.budget, st);
                            ok = __all_sync(FULL, w);
                        }
                        xr.next(X_RING);
                    }
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
        const int lw = warp - 13;                             // slots 16 lw .. 16 lw + 15 of the tile
        const int half = lane >> 4, piece = lane & 15;        // a copy moves 256 bytes of two rows
        const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.m.kv);
        Ring in, out;                                         // blocks issued, blocks signalled
        int behind = 0, odb = 0;                              // in flight; dim block of the oldest
        uint32_t og = 0, g = 0;                               // tile of the oldest, tiles issued
        unsigned live[2] = {0u, 0u};                          // valid slots of the last two tiles
        float known[2] = {0.0f, 0.0f};                        // lanes 0-15: their RMS factors from the table
        float ss[8];
        bool ok = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[j] = 0.0f;
        auto signal = [&]() {                                 // the oldest block in flight
            if (behind == 3)
                cp_async_wait<2>();
            else if (behind == 2)
                cp_async_wait<1>();
            else
                cp_async_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&xfull[out.i]);
            // squares of the pieces this lane copied (before the block can be overwritten: the
            // ring comes back here only through this warp)
            const uint8_t* src = sX + out.i * BLOCK + (piece >> 3) * CHUNK;
            if (!a.m.rinv)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 v = *reinterpret_cast<const uint4*>(
                    src + sw128_offset((uint32_t)(16 * lw + 2 * j + half), (uint32_t)(piece & 7)));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = __uint_as_float(w[k] << 16), y = __uint_as_float(w[k] & 0xFFFF0000u);
                    ss[j] = fmaf(x, x, ss[j]);
                    ss[j] = fmaf(y, y, ss[j]);
                }
            }
            out.next(X_RING);
            --behind;
            if (++odb < 4) return;
            odb = 0;
            // the tile is complete: its rows' RMS factors
            const int rb = og & 1;
            if (og >= 2) {
                const bool w = mbar_wait(&rempty[rb], ((og >> 1) - 1) & 1, a.budget, st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    return;
                }
            }
            const unsigned lv = rb ? live[1] : live[0];
            if (a.m.rinv) {
                if (lane < 16) sRinv[rb * MT_TILE + 16 * lw + lane] = rb ? known[1] : known[0];
            } else
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float s = ss[j];
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
                if (piece == j) {
                    const int slot = 2 * j + half;
                    sRinv[rb * MT_TILE + 16 * lw + slot] =
                        !((lv >> slot) & 1u) ? -1.0f : (a.m.flags & CSA2_KVNORM) ? ag_rms_factor(s) : 1.0f;
                }
                ss[j] = 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&rfull[rb]);
            ++og;
        };
        for (int64_t i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it = item_of(a, i);
            for (int tp = 0; tp < it.nt * a.n_pass && ok; ++tp, ++g) {
                const int tt = tp % it.nt;
                const int64_t row = lane < 16 ? row_of(a.m.slots, it, (it.t0 + tt) * MT_TILE + 16 * lw + lane, false) : -1;
                const unsigned lv = __ballot_sync(FULL, row >= 0);
                const float kn = !a.m.rinv || row < 0 ? -1.0f : (a.m.flags & CSA2_KVNORM) ? a.m.rinv[row] : 1.0f;
                if (g & 1) {
                    live[1] = lv;
                    known[1] = kn;
                } else {
                    live[0] = lv;
                    known[0] = kn;
                }
                const uint8_t* src = row >= 0 ? kv + row * (MT_C * 2) : nullptr;
                const uint8_t* from[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    from[j] = reinterpret_cast<const uint8_t*>(
                        (uintptr_t)__shfl_sync(FULL, (unsigned long long)(uintptr_t)src, 2 * j + half));
                for (int db = 0; db < 4 && ok; ++db) {
                    if (in.round > 0) {
                        const uint32_t par = (in.round - 1) & 1;
                        // blocks in flight are signalled before a wait that they may be needed for
                        if (!__all_sync(FULL, mbar_test(&xempty[in.i], par))) {
                            while (behind > 0 && ok) signal();
                            if (!ok) break;
                            const bool w = mbar_wait(&xempty[in.i], par, a.budget, st);
                            if (!__all_sync(FULL, w)) {
                                ok = false;
                                break;
                            }
                        }
                    }
                    uint8_t* dst = sX + in.i * BLOCK + (piece >> 3) * CHUNK;
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
                    if (++behind > 2) signal();
                }
            }
        }
        while (ok && behind > 0) signal();
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
    kern<<<(unsigned)grid, MT_THREADS, SMEM_BYTES, s>>>(a);
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
    a.items = m.n_bq * a.n_split;
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
