// Backward pass of the shared-KV MQA on the tcgen05 tensor cores (attn_bwd.cu has the
// formulas): bf16 query, rows, window and dout, both RMSNorms, head passes of 64.
//
// Work item = (head pass, query, range of 128-slot tiles).  A query's image -- 128 rows of 512
// dims, the normalised rotated heads q^ and then the rotated gradients do' -- stays in shared
// memory for the whole item.  A tile's raw key rows X [128 slots x 512] pass through a ring of
// four 64-dim chunks; the second half of them stays there from the logits to dQ, the first half
// is read again (from L2):
//   [S  dP] [128 slots x 128]  = X . image^T
//   dQ^T [512 dims x 64 heads] += X^T . (r dS)
//   dK [128 slots x 512 dims]  = [r dS  r P] . image
// p = exp(z - lse), dS = p (dP - D)/sqrt(c), r the row's RMS factor (folded in, so X is never
// rescaled and dK comes out as the row's contribution r dk^).  dQ accumulates in tensor memory
// over the item; dK leaves per tile, in 128-dim blocks, to its place in the sorted list of
// contributions, as bf16: the list is written and read once from device memory and its size is
// what bounds the row sums.  The addends' rounding (2^-8 at most, of values that p and dS rounded
// to bf16 made) is no larger than theirs; the sums over them are fp32.  dq^ leaves as fp32: a
// query of few keys has one that is nearly parallel to q^, and the norm's backward pass takes
// that part away (as bf16, 50 us less at 2,048 queries, its rounding was 3 times the rest there).
//
// What bounds it: the MMAs (96 a tile; one of M = 128 costs the same for N = 64 and N = 128, 81
// cycles K-major and 92 to 105 with MN-major operands here, about 9,000 a tile) and the waits
// between them: for chunks on their way from L2 (2,000 cycles under load, with room for half a
// tile only) and for the softmax (1,300).  2,048 queries of 640 slots: 618 us, 15,000 cycles a
// tile.  What was measured against it (product kernel, the same call):
//   870 us  64 slots a tile, so that S, dQ and dK all run at N = 64
//   919 us  X kept in shared memory between its two uses, half a tile at a time: 64 MMAs for S
//           instead of 32, and every half waits for the one before
//   922 us  a lane storing its own slot's 32-byte pieces of dK; whole 128-byte lines by a 4 x 4
//           exchange between neighbouring lanes, as below: 704
//   1,132 us  two CTAs of a cluster with 256 dims each (every product N >= 128, but the halves of
//           S and dP are summed through distributed shared memory, 48 KB a tile at 12 bytes a cycle)
//
// Warp roles (448 threads of 128 registers, so nothing spills -- beside 226 KB of shared memory
// there is no L1, and a spilled register is read from L2; one CTA per SM, persistent):
//   warp 0        the images (four 32 KB bulk copies, each freed by its dK block)
//   warp 1        MMA issuer; owns the tensor memory
//   warps 2-5     softmax: one thread per slot
//   warps 6-9     loaders: 16-byte cp.async, a warp one place of the ring
//   warps 10-13   drain: dK blocks, one thread per slot; dQ at the end of the item
// Every wait is bounded; a wait that expires flags a timeout and the roles wind down.
#include <algorithm>
#include <atomic>

#include "attn_bwd_tc.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace sm100;

constexpr int BT_C = 512;
constexpr int BT_H = 64;
constexpr int BT_TILE = 128;
constexpr int BT_THREADS = 448;
constexpr int CHUNK = 128 * 128;                 // 128 rows (of the image, or slots) x 64 dims
constexpr int IMG_BYTES = 8 * CHUNK;
constexpr int X_RING = 4;                        // chunks of X (the roles below count on four)
constexpr uint32_t COL_DQ = 0, COL_S = 256, COL_DK = 384;
constexpr uint32_t TMEM_COLS = 512;
constexpr long long WAIT_BUDGET = 1ll << 31;
constexpr unsigned FULL = 0xffffffffu;

constexpr int OFF_IMG = 0;
constexpr int OFF_X = OFF_IMG + IMG_BYTES;
constexpr int OFF_DSP = OFF_X + X_RING * CHUNK;  // r dS, then r P: [128 slots][64 heads]
constexpr int OFF_LD = OFF_DSP + 2 * CHUNK;      // [4 warps][64 heads] -lse (base 2), -D / sqrt(c)
constexpr int OFF_START = OFF_LD + 4 * BT_H * 8;
constexpr int OFF_BAR = OFF_START + 16;
constexpr int N_BAR = 4 + 4 + 2 * X_RING + 9;
constexpr int OFF_TMEMPTR = OFF_BAR + N_BAR * 8;
constexpr int SMEM_BYTES = OFF_TMEMPTR + 16;
static_assert(OFF_START % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

// The 8 words lo of the upper lane of a pair `d` apart and hi of the lower one change places.
__device__ __forceinline__ void swap_pieces(uint32_t* lo, uint32_t* hi, int d, bool upper) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t got = __shfl_xor_sync(FULL, upper ? lo[i] : hi[i], d);
        if (upper)
            lo[i] = got;
        else
            hi[i] = got;
    }
}

// The slots of a query that hold something, in order -- its cache slots, then the window slots
// whose position is not before 0 -- as the roles below want them: code[q][s] = a cache row's
// number, -2 - a window row's, or -1 (empty); fac[q][s] = the row's RMS factor, 0 if empty;
// place[q][s] = its contribution's place, -1 if empty; n_of[q] = how many, tile0[q] = the tiles
// they fill (scanned afterwards: the tiles of the queries before).  A chain of three
// dependent lookups a slot, made here with every slot at once and read back in one access.
__global__ void __launch_bounds__(256) bwd_tc_slots_kernel(BwdTcArgs a, int32_t* code, float* fac, int32_t* place,
                                                           int32_t* n_of, uint32_t* tile0) {
    const SlotArgs& sl = a.c.slots;
    const int q = blockIdx.y, s = blockIdx.x * 256 + threadIdx.x;
    if (s >= a.n_pad) return;
    const int64_t bq = a.c.bq0 + q, t = sl.q_pos[bq];
    const int nw = (int)max((int64_t)0, min((int64_t)sl.window, t + 1));
    const int kq = sl.dense_nv ? (int)max((int64_t)0, min((int64_t)sl.k, sl.dense_nv[bq])) : sl.k;
    const int slot = s < kq ? s : s < kq + nw ? sl.k + (sl.window - nw) + (s - kq) : -1;
    const int64_t row = slot >= 0 ? slot_row(sl, bq, slot, false) : -1;
    const int64_t at = (int64_t)q * a.n_pad + s;
    code[at] = row < 0 ? -1 : row < sl.n_kv ? (int32_t)row : (int32_t)(-2 - (row - sl.n_kv));
    fac[at] = row >= 0 ? a.c.rinv[row] : 0.0f;
    place[at] = row >= 0 ? (int32_t)(a.c.blk[row / BWD_SCAN_ROWS] + a.c.base[(int64_t)(q / a.c.group_q) * a.c.rows + row]) +
                               a.c.rank[(int64_t)q * a.c.n_slots + slot]
                         : -1;
    if (s == 0) {
        n_of[q] = kq + nw;
        tile0[q] = (uint32_t)((kq + nw + BT_TILE - 1) / BT_TILE);
        if (q == 0) tile0[a.c.nb] = 0u;
    }
}

// The (pass, query) pairs v = pass * nb + query are dealt out whole, one a CTA and wave, as long as
// that fills the wave; the tiles of the rest are shared evenly, so there a query's may go to
// several CTAs (whose dq^ are added) and a CTA have the end of one query and the beginning of
// another.  (Whole queries, or equal parts of them, to the end leave the last wave half empty:
// 666 pairs of 9 tiles took 399 us.  Even shares of everything, 410 us and 2,048 queries 10 %
// more: neighbouring queries' contributions are neighbours in the list, and are written
// together only if they run together.)
struct Tail {
    uint32_t first, before, all, per;                // first pair; tiles before it and in all; a CTA's share
};

__device__ __forceinline__ Tail tail_of(const BwdTcArgs& a) {
    const uint32_t total = a.tile0[a.c.nb];
    Tail r;
    r.first = a.waves * a.ctas;
    r.before = r.first / a.c.nb * total + a.tile0[r.first % a.c.nb];
    r.all = total * a.n_pass;
    r.per = max(1u, (r.all - r.before + a.ctas - 1) / a.ctas);
    return r;
}

struct Item {
    int v;                       // pass * nb + query: the image
    int q, pass;                 // query within the chunk
    int t0, nt;                  // tiles t0 .. t0 + nt - 1 of the query's
    int dq;                      // its dq^: v in the waves, v + CTA in the shared rest
};

// Where a CTA's share of the rest begins, and how many tiles it has.
struct Start {
    int pass, q, t0, tiles;
};

// (by one warp: the last query whose tiles begin at or before the share's first)
__device__ __forceinline__ Start find_start(const BwdTcArgs& a, int lane) {
    const Tail tail = tail_of(a);
    const uint32_t total = a.tile0[a.c.nb], g = tail.before + blockIdx.x * tail.per;
    Start r = {0, 0, 0, 0};
    if (g >= tail.all) return r;
    r.tiles = (int)min(tail.per, tail.all - g);
    r.pass = (int)(g / total);
    const uint32_t t = g - r.pass * total;
    int lo = 0, n = a.c.nb;                          // the query is one of lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const unsigned le = __ballot_sync(FULL, at < lo + n && a.tile0[min(at, a.c.nb)] <= t);
        const int k = 31 - __clz(le);                // (lane 0's is one of them)
        n = min(step, n - k * step);
        lo += k * step;
    }
    r.q = lo;
    r.t0 = (int)(t - a.tile0[lo]);
    return r;
}

// The CTA's items one after the other (one without tiles where a query has none); the next
// one's number of slots is read ahead.
struct Items {
    const BwdTcArgs& a;
    uint32_t v, step;                                // the next item's pair; pairs to the one after it
    int t0, left, n;                                 // its first tile; the rest's tiles; its slots
    __device__ __forceinline__ Items(const BwdTcArgs& args, const Start& s)
        : a(args), v(blockIdx.x), step(args.ctas), t0(0), left(s.tiles) {
        if (a.waves == 0) rest(s);
        n = a.n_of[v % a.c.nb];
    }
    __device__ __forceinline__ void rest(const Start& s) {
        v = (uint32_t)(s.pass * a.c.nb + s.q);
        step = 1;
        t0 = s.t0;
    }
    __device__ __forceinline__ bool more() const { return step > 1 || left > 0; }
    __device__ __forceinline__ Item next(const Start& s) {
        const int tiles = (n + BT_TILE - 1) / BT_TILE;
        Item r;
        r.v = (int)v;
        r.pass = r.v / a.c.nb;
        r.q = r.v - r.pass * a.c.nb;
        r.t0 = t0;
        r.dq = r.v;
        r.nt = tiles;
        if (step > 1) {
            v += step;
            if (v >= a.waves * a.ctas) rest(s);
        } else {
            r.dq += blockIdx.x;
            r.nt = min(tiles - t0, left);
            left -= r.nt;
            t0 = 0;
            ++v;
        }
        n = a.n_of[v % a.c.nb];
        return r;
    }
};

__device__ __forceinline__ void st_global32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Images of the chunk's queries and D; a warp per head, 8 heads a CTA.  Image row of head h
// (within its pass): h for q^, 64 + h for do'.  Heads past H are 0.
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
    uint8_t* base = img + ((int64_t)(h >> 6) * nb + qi) * IMG_BYTES + (lane >> 2) * CHUNK;
    const uint32_t row = h & 63, u = 2u * (lane & 3);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = k == 0 ? ag_pack_bf16x2(v[2 * i], v[2 * i + 1]) : ag_pack_bf16x2(g[2 * i], g[2 * i + 1]);
        *reinterpret_cast<uint4*>(base + sw128_offset(row + 64 * k, u)) = make_uint4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<uint4*>(base + sw128_offset(row + 64 * k, u + 1)) = make_uint4(p[4], p[5], p[6], p[7]);
    }
}

// dq from dq^ (the sum over the CTAs that had tiles of the query): back through RoPE and the query's RMSNorm.  A
// warp per (query, head); a query that attends to nothing has no gradient.
__global__ void __launch_bounds__(256) bwd_tc_dq_kernel(BwdTcArgs a, const float* dqh, __nv_bfloat16* dq) {
    __shared__ float cs[8][32], sn[8][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + w;
    if (r >= (int64_t)a.c.nb * a.c.H) return;
    const int qi = (int)(r / a.c.H), h = (int)(r % a.c.H);
    const int64_t bq = a.c.bq0 + qi, o = (bq * a.c.H + h) * BT_C + 16 * lane;
    const int pass = h >> 6;
    const uint32_t v0 = (uint32_t)pass * a.c.nb + qi;
    auto sum_at = [&](uint32_t k) { return dqh + ((int64_t)k * BT_H + (h & 63)) * BT_C + 16 * lane; };
    const bool whole = v0 < a.waves * a.ctas;
    float g[16], v[16];
    if (whole) ag_load16<float>(sum_at(v0), g);
    ag_load16<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.c.q) + o, v);
    const uint32_t tiles = a.tile0[qi + 1] - a.tile0[qi];
    ag_cos_sin(a.c.rope, a.c.slots.q_pos[bq], lane, cs[w][lane], sn[w][lane]);
    __syncwarp();
    if (!whole || tiles == 0) {                      // (nobody wrote the sum of a query without keys)
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = 0.0f;
    }
    if (!whole && tiles > 0) {
        const Tail tail = tail_of(a);
        const uint32_t begin = pass * a.tile0[a.c.nb] + a.tile0[qi] - tail.before;
        const uint32_t last = (begin + tiles - 1) / tail.per;
        for (uint32_t s = begin / tail.per; s <= last; ++s) {
            float p[16];
            ag_load16<float>(sum_at(v0 + s), p);
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] += p[i];
        }
    }
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
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sImg = smem + OFF_IMG;
    uint8_t* sX = smem + OFF_X;
    uint8_t* sDsp = smem + OFF_DSP;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* imgfull = bars;                       // [4] 128-dim blocks of the image
    uint64_t* imgempty = bars + 4;                  // [4]
    uint64_t* xfull = bars + 8;                     // [X_RING]
    uint64_t* xempty = xfull + X_RING;              // [X_RING]
    uint64_t* sfull = xempty + X_RING;              // per tile
    uint64_t* sempty = sfull + 1;
    uint64_t* dspfull = sfull + 2;                  // per tile
    uint64_t* dspempty = sfull + 3;
    uint64_t* dkfull = sfull + 4;                   // per dK block
    uint64_t* dkempty = sfull + 5;
    uint64_t* dqfull = sfull + 6;                   // per item
    uint64_t* dqempty = sfull + 7;
    uint64_t* alldone = sfull + 8;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEMPTR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned* st = a.c.slots.st;

    if (smem_u32(smem) & 1023u) {                   // the operand tiles' layout needs it (never seen)
        if (threadIdx.x == 0) csa2_flag(st, CSA2_DEVBIT_TIMEOUT);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&imgfull[i], 1);
            mbar_init(&imgempty[i], 1);
        }
        for (int i = 0; i < X_RING; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 1);
        }
        mbar_init(sfull, 1);
        mbar_init(sempty, 4);
        mbar_init(dspfull, 4);
        mbar_init(dspempty, 1);
        mbar_init(dkfull, 1);
        mbar_init(dkempty, 4);
        mbar_init(dqfull, 1);
        mbar_init(dqempty, 4);
        mbar_init(alldone, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sTmem, TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 2) {
        const Start s = find_start(a, lane);
        if (lane == 0) *reinterpret_cast<Start*>(smem + OFF_START) = s;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sTmem;
    const Start* start = reinterpret_cast<const Start*>(smem + OFF_START);

    if (warp == 0) {
        // ============================ images ============================
        if (lane == 0) {
            int n = 0;                               // items with tiles so far
            bool ok = true;
            int issued = 0;                          // blocks issued in the last item, and their phase
            uint32_t par = 0;
            for (Items items(a, *start); items.more() && ok && !a.stall;) {
                const Item it = items.next(*start);
                if (it.nt == 0) continue;
                issued = 0;
                par = n & 1;
                for (int db = 0; db < 4; ++db) {
                    if (n > 0 && !mbar_wait(&imgempty[db], (n - 1) & 1, a.budget, st)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&imgfull[db], 2 * CHUNK);
                    bulk_g2s(sImg + db * 2 * CHUNK, a.img + (int64_t)it.v * IMG_BYTES + db * 2 * CHUNK, 2 * CHUNK,
                             &imgfull[db]);
                    issued = db + 1;
                }
                ++n;
            }
            // the last copies must land before the CTA exits
            for (int db = 0; db < issued; ++db) mbar_wait(&imgfull[db], par, a.budget, st);
        }
    } else if (warp == 1) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc_f16(128, 128, true);
            constexpr uint32_t ID_DQ = idesc_f16_major(128, BT_H, true, true, true);
            constexpr uint32_t ID_DK = idesc_f16_major(128, 128, true, false, true);
            const uint32_t img = smem_u32(sImg), x0 = smem_u32(sX), dsp = smem_u32(sDsp);
            uint32_t g = 0, t = 0, k = 0;            // tiles with logits; tiles done; dK blocks
            int n = 0;                               // items with tiles so far
            bool ok = true;
            auto wait = [&](uint64_t* b, uint32_t par) {
                ok = ok && mbar_wait(b, par, a.budget, st);
                return ok;
            };
            // A place of the ring is filled three times a tile: with chunk x and chunk x + 4 for the
            // logits -- the latter stays for dQ -- and with chunk x again for dQ.
            // chunk ch (64 dims) of the logits of tile g
            auto scores = [&](int ch) {
                const int x = ch & 3;
                if (!wait(&xfull[x], (3 * g + (ch >> 2)) & 1)) return;
                tc_fence_after();
                const uint64_t dx = sdesc_sw128(x0 + x * CHUNK), di = sdesc_sw128(img + ch * CHUNK);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(tmem + COL_S, dx + (kk * 32 >> 4), di + (kk * 32 >> 4), ID_S, (ch | kk) != 0);
                if (ch < 4) mma_commit(&xempty[x]);
                if (ch == 7) {
                    mma_commit(sfull);
                    ++g;
                }
            };
            // dims block db of dQ, from two places of the ring
            auto dq = [&](int db, bool fresh) {
                const int x = 2 * (db & 1);
                if (db < 2 && (!wait(&xfull[x], (3 * t + 2) & 1) || !wait(&xfull[x + 1], (3 * t + 2) & 1))) return;
                tc_fence_after();
                const uint64_t dx = sdesc_sw128_mn(x0 + x * CHUNK, CHUNK, 1024), dds = sdesc_sw128_mn(dsp, CHUNK, 1024);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ss(tmem + COL_DQ + db * BT_H, dx + (ks * 2048 >> 4), dds + (ks * 2048 >> 4), ID_DQ, !fresh || ks > 0);
                mma_commit(&xempty[x]);
                mma_commit(&xempty[x + 1]);
            };
            auto dk = [&](int db, bool last) {
                if (k > 0 && !wait(dkempty, (k - 1) & 1)) return;
                tc_fence_after();
                const uint64_t da = sdesc_sw128(dsp), di = sdesc_sw128_mn(img + 2 * db * CHUNK, CHUNK, 1024);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ss(tmem + COL_DK, da + (((ks >> 2) * CHUNK + (ks & 3) * 32) >> 4), di + (ks * 2048 >> 4), ID_DK, ks > 0);
                mma_commit(dkfull);
                ++k;
                if (last) mma_commit(&imgempty[db]);
                if (db == 3) mma_commit(dspempty);
            };
            for (Items items(a, *start); items.more() && ok;) {
                const Item it = items.next(*start);
                if (it.nt == 0) continue;
                if (g > 0 && !wait(sempty, (g - 1) & 1)) break;
                for (int ch = 0; ch < 8 && ok; ++ch)
                    if ((ch & 1) || wait(&imgfull[ch >> 1], n & 1)) scores(ch);
                for (int tt = 0; tt < it.nt && ok; ++tt, ++t) {
                    const bool last = tt == it.nt - 1;
                    if (tt == 0 && n > 0 && !wait(dqempty, (n - 1) & 1)) break;
                    if (!wait(dspfull, t & 1)) break;
                    // the dK blocks run where the others would wait for chunks that were just made room for
                    dq(2, tt == 0);
                    if (ok) dq(3, tt == 0);
                    if (ok) dk(0, last);
                    if (ok) dq(0, tt == 0);
                    if (ok) dq(1, tt == 0);
                    if (ok && last) mma_commit(dqfull);
                    if (ok) dk(1, last);
                    if (ok) dk(2, last);
                    if (ok && !last && wait(sempty, (g - 1) & 1))
                        for (int ch = 0; ch < 8 && ok; ++ch) {
                            scores(ch);
                            if (ch == 3 && ok) dk(3, false);
                        }
                    if (ok && last) dk(3, true);
                }
                if (ok) ++n;
            }
            // the MMAs must be complete before tensor memory is released
            mma_commit(alldone);
            mbar_wait(alldone, 0, a.budget, st);
        }
    } else if (warp < 6) {
        // ============================ softmax ============================
        const int qd = warp & 3;
        const uint32_t slot = 32 * qd + lane;                 // of the tile
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        float2* ld = reinterpret_cast<float2*>(smem + OFF_LD) + qd * BT_H;
        const float isc = 1.0f / sqrtf((float)BT_C);
        uint32_t t = 0;
        bool ok = true;
        for (Items items(a, *start); items.more() && ok;) {
            const Item it = items.next(*start);
            if (it.nt == 0) continue;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = it.pass * BT_H + 32 * j + lane;
                float2 v = make_float2(-INFINITY, 0.0f);      // p = 0 for heads past H and empty queries
                if (h < a.c.H) {
                    const int64_t o = (a.c.bq0 + it.q) * a.c.H + h;
                    const float l = a.c.lse[o], d = a.c.D[o];
                    if (l != -INFINITY) v = make_float2(-l * AG_LOG2E, -d * isc);
                }
                ld[32 * j + lane] = v;
            }
            __syncwarp();
            // the row's RMS factor, 0 for an empty slot, read a tile ahead
            const float* fac = a.fac + (int64_t)it.q * a.n_pad + it.t0 * BT_TILE + slot;
            float next = *fac;
            for (int tt = 0; tt < it.nt; ++tt, ++t) {
                const float r = next, rs = r * isc, rz = rs * AG_LOG2E;
                if (tt + 1 < it.nt) next = fac[(tt + 1) * BT_TILE];
                bool w = mbar_wait(sfull, t & 1, a.budget, st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (t > 0) w = mbar_wait(dspempty, (t - 1) & 1, a.budget, st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    break;
                }
                // 16 heads at a time; the next ones are read from tensor memory meanwhile
                uint32_t s[2][16], d[2][16];
                tmem_ld16(tmem + lane_base + COL_S, s[0]);
                tmem_ld16(tmem + lane_base + COL_S + 64, d[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_wait_ld();
                    if (q < 3) {
                        tmem_ld16(tmem + lane_base + COL_S + 16 * (q + 1), s[(q + 1) & 1]);
                        tmem_ld16(tmem + lane_base + COL_S + 64 + 16 * (q + 1), d[(q + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sempty);
                    }
                    uint32_t ds[8], pp[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 h2 = *reinterpret_cast<const float4*>(&ld[16 * q + 2 * j]);   // two heads
                        float v0 = ex2_approx(fmaf(__uint_as_float(s[q & 1][2 * j]), rz, h2.x)) * r;
                        float v1 = ex2_approx(fmaf(__uint_as_float(s[q & 1][2 * j + 1]), rz, h2.z)) * r;
                        if (r == 0.0f) v0 = v1 = 0.0f;
                        pp[j] = ag_pack_bf16x2(v0, v1);
                        ds[j] = ag_pack_bf16x2(v0 * fmaf(__uint_as_float(d[q & 1][2 * j]), rs, h2.y),
                                               v1 * fmaf(__uint_as_float(d[q & 1][2 * j + 1]), rs, h2.w));
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint8_t* dst = sDsp + sw128_offset(slot, 2 * q + u);
                        *reinterpret_cast<uint4*>(dst) = make_uint4(ds[4 * u], ds[4 * u + 1], ds[4 * u + 2], ds[4 * u + 3]);
                        *reinterpret_cast<uint4*>(dst + CHUNK) = make_uint4(pp[4 * u], pp[4 * u + 1], pp[4 * u + 2], pp[4 * u + 3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(dspfull);
            }
        }
    } else if (warp < 10) {
        // ============================ loaders ============================
        // A warp fills one place of the ring, every fourth chunk: copies in flight in one warp then
        // never wait for another's.
        const int x = warp - 6;
        const int sub = lane >> 3, piece = lane & 7;          // a copy moves 128 bytes of four rows
        // (an empty slot's copy reads nothing; its address is a row of whichever array there is)
        const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.c.kv ? a.c.kv : a.c.swa) + piece * 16;
        const uint8_t* swa = reinterpret_cast<const uint8_t*>(a.c.swa) + piece * 16;
        // rows 8 apart have the same swizzle
        uint8_t* dst0 = sX + x * CHUNK + sw128_offset((uint32_t)sub, (uint32_t)piece);
        uint8_t* dst4 = sX + x * CHUNK + sw128_offset((uint32_t)(sub + 4), (uint32_t)piece);
        uint32_t c = 0;                                       // chunks filled
        bool ok = true;
        // chunks x and, for the logits, x + 4 of a tile; code[q]: slot 32 q + lane
        auto stream = [&](const int (&code)[4], int end) {
#pragma unroll 1
            for (int ch = x; ch < end && ok; ch += 4, ++c) {
                bool w = true;
                if (c > 0) w = mbar_wait(&xempty[x], (c - 1) & 1, a.budget, st);
                if (!__all_sync(FULL, w)) {
                    ok = false;
                    return;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {                 // eight addresses, then eight copies
                    const uint8_t* src[8];
                    bool read[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int o = __shfl_sync(FULL, code[q], 4 * j + sub);
                        read[j] = o != -1;
                        src[j] = (o >= -1 ? kv : swa) + ((uint64_t)(uint32_t)(o >= -1 ? max(o, 0) : -2 - o) * (BT_C * 2) + ch * 128);
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
        };
        for (Items items(a, *start); items.more() && ok;) {
            const Item it = items.next(*start);
            if (it.nt == 0) continue;
            const int32_t* codes = a.code + (int64_t)it.q * a.n_pad + it.t0 * BT_TILE + lane;
            int code[4], next[4];                             // read a tile ahead
#pragma unroll
            for (int q = 0; q < 4; ++q) code[q] = next[q] = codes[32 * q];
            stream(code, 8);                                  // logits
            for (int tt = 0; tt < it.nt && ok; ++tt) {
                if (tt + 1 < it.nt)
#pragma unroll
                    for (int q = 0; q < 4; ++q) next[q] = codes[(tt + 1) * BT_TILE + 32 * q];
                stream(code, 4);                              // dQ
                if (ok && tt + 1 < it.nt) stream(next, 8);    // the next tile's logits
#pragma unroll
                for (int q = 0; q < 4; ++q) code[q] = next[q];
            }
        }
    } else {
        // ============================ drain ============================
        const int qd = warp & 3;
        const uint32_t slot = 32 * qd + lane;                 // of the tile
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        const uint32_t row_bytes = (uint32_t)a.n_pass * BT_C * 2;
        uint32_t k = 0;
        int n = 0;
        bool ok = true;
        for (Items items(a, *start); items.more() && ok;) {
            const Item it = items.next(*start);
            if (it.nt == 0) continue;
            // (slot: here the dim of a block)
            float* dqh = a.dqh + (int64_t)it.dq * (BT_H * BT_C) + slot;
            uint8_t* base = reinterpret_cast<uint8_t*>(a.c.part) + it.pass * (BT_C * 2) + (lane & 3) * 32;
            // the place of the slot's contribution (-1: empty), read a tile ahead
            const int32_t* place = a.place + (int64_t)it.q * a.n_pad + it.t0 * BT_TILE + slot;
            int next = *place;
            for (int tt = 0; tt < it.nt && ok; ++tt) {
                const int pl = next;
                if (tt + 1 < it.nt) next = place[(tt + 1) * BT_TILE];
                // four neighbouring lanes store 128 bytes of one of their slots at a time
                uint8_t* dst[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int o = __shfl_sync(FULL, pl, (lane & 28) + j);
                    dst[j] = o >= 0 ? base + (uint64_t)(uint32_t)o * row_bytes : nullptr;
                }
#pragma unroll 1
                for (int db = 0; db < 4; ++db, ++k) {
                    const bool w = mbar_wait(dkfull, k & 1, a.budget, st);
                    if (!__all_sync(FULL, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t u[64];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint32_t v[16];
                        tmem_ld16(tmem + lane_base + COL_DK + 16 * q, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            u[8 * q + j] = ag_pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dkempty);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {    // 64 dims: 4 x 4 pieces of 16 change lanes
                        uint32_t* w = u + 32 * half;
#pragma unroll
                        for (int j = 0; j < 4; j += 2) swap_pieces(w + 8 * j, w + 8 * (j + 1), 1, lane & 1);
#pragma unroll
                        for (int j = 0; j < 2; ++j) swap_pieces(w + 8 * j, w + 8 * (j + 2), 2, lane & 2);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (dst[j]) st_global32(dst[j] + db * 256 + half * 128, w + 8 * j);
                    }
                }
            }
            if (!ok) break;
            const bool w = mbar_wait(dqfull, n & 1, a.budget, st);
            if (!__all_sync(FULL, w)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {                     // heads 32 (j & 1) .. of dims block j >> 1
                uint32_t o[32];
                tmem_ld32(tmem + lane_base + COL_DQ + 32 * j, o);
                tmem_wait_ld();
                float* d = dqh + (int64_t)(32 * (j & 1)) * BT_C + (j >> 1) * 128;
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

int pad_slots(int n) { return std::max(1, (n + BT_TILE - 1) / BT_TILE) * BT_TILE; }

// CTAs for `queries` (times head passes): one a tile, at most one an SM (sizes are also asked for
// without a GPU).
int64_t ctas_for(int num_sms, int64_t queries, int n_slots) {
    return std::min<int64_t>(std::max(1, num_sms), queries * (pad_slots(n_slots) / BT_TILE));
}

}  // namespace

bool bwd_tc_applies(csa2_dtype q_dt, csa2_dtype kv_dt, int k, csa2_dtype swa_dt, int window, csa2_dtype out_dt,
                    unsigned flags) {
    return q_dt == CSA2_BF16 && (k == 0 || kv_dt == CSA2_BF16) && (window == 0 || swa_dt == CSA2_BF16) &&
           out_dt == CSA2_BF16 && (flags & (CSA2_QNORM | CSA2_KVNORM)) == (CSA2_QNORM | CSA2_KVNORM);
}

// dq^ of every (query, CTA that has tiles of it).
size_t bwd_tc_dq_bytes(int num_sms, int64_t queries, int n_slots) {
    return (size_t)(queries + ctas_for(num_sms, queries, n_slots) - 1) * BT_H * BT_C * 4;
}

size_t bwd_tc_image_bytes() { return IMG_BYTES; }

size_t bwd_tc_slots_bytes(int64_t nb, int n_slots) {
    return (size_t)(nb * (3 * (int64_t)pad_slots(n_slots) + 2) + 1) * 4;
}

csa2_status bwd_tc_chunk(csa2_ctx* ctx, BwdTcArgs& a, const void* dout, const void* out, float* D, uint8_t* img,
                         void* slots, cudaStream_t s) {
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
    a.n_pad = pad_slots(c.n_slots);
    int32_t* code = reinterpret_cast<int32_t*>(slots);
    int32_t* place = code + (int64_t)c.nb * a.n_pad;
    float* fac = reinterpret_cast<float*>(place + (int64_t)c.nb * a.n_pad);
    int32_t* n_of = reinterpret_cast<int32_t*>(fac + (int64_t)c.nb * a.n_pad);
    uint32_t* tile0 = reinterpret_cast<uint32_t*>(n_of + c.nb);
    a.code = code;
    a.place = place;
    a.fac = fac;
    a.n_of = n_of;
    a.tile0 = tile0;
    bwd_tc_slots_kernel<<<dim3((unsigned)((a.n_pad + 255) / 256), (unsigned)c.nb), 256, 0, s>>>(a, code, fac, place, n_of, tile0);
    bwd_scan(tile0, (int64_t)c.nb + 1, s);
    a.ctas = (uint32_t)ctas_for(ctx->num_sms, (int64_t)c.nb * a.n_pass, c.n_slots);
    a.budget = WAIT_BUDGET;
    a.stall = 0;
    if (ctx->stall_next) {
        a.stall = 1;
        if (ctx->stall_budget > 0) a.budget = ctx->stall_budget;
        ctx->stall_next = 0;
    }
    a.waves = a.ctas > 1 ? (uint32_t)c.nb * a.n_pass / a.ctas : 0;      // (a step of 1 marks the shared rest)
    attn_bwd_tc_kernel<<<a.ctas, BT_THREADS, SMEM_BYTES, s>>>(a);
    const int64_t heads = (int64_t)c.nb * c.H;
    bwd_tc_dq_kernel<<<(unsigned)((heads + 7) / 8), 256, 0, s>>>(a, a.dqh, reinterpret_cast<__nv_bfloat16*>(c.dq));
    return csa2_launch_status();
}
