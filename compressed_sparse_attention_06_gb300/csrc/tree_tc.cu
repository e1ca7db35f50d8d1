// Attention of drafted trees on the tcgen05 tensor cores (DSA-to-CSA/HCA page eqs. (18)-(19), (26),
// (27)): the same RMS-normalised row is key and value for all heads of a node and, in the dense
// form, for all nodes of a tree.
//
// A work item is a group of up to 128 query rows that read the same slots (a node's heads; dense:
// those of up to 8 nodes) and a range of tiles of 128 slots.  Two CTAs (a cluster) share an item,
// each with half of the 512 dims: the fp32 output of 128 rows x 512 dims alone is all of an SM's
// tensor memory, and 64 rows would leave half of every MMA unused (N = 64 costs what N = 128 does).
//   S[128 rows x 128 slots]  = Q^[128 x 256] . X[128 x 256]^T     this CTA's half of the logits
//   O[128 rows x 256 dims]  += P'[128 x 128] . X[128 x 256]       P' = p f, read from tensor memory
// f = RMS factor of the slot's row / (sqrt(512) ln 2): it scales the logits (to base 2) and, folded
// into P', makes a row's value its normalised form, so X is never rescaled.  Both norms bound a logit
// by sqrt(512), 32.7 in base 2: p = 2^z needs no running maximum (sums of 4 million of them stay below
// 2^55), and the splits of a group's slots simply add up.
//
// Each CTA weighs half of a tile's slots for both: it gets the peer's half logits of its 64 slots as 16-bit
// multiples of 1/992 in base 2 (TT_FIX), adds them to its own fp32 ones and sends P' (bf16) back, 16 KB each
// way.  The half logits of a query that lies along a row reach 32.7: as fp16 they were off by up to 2^-6
// there, which moved log-sum-exps by 3e-3; a fixed step moves a weight by 3.5e-4 at most, wherever the logit
// stands.  (The rounding of q^'s 64 rotated dims to bf16 is what is left: 2^-8 / sqrt(3) of the root of the sum of
// their products' squares, 1e-3 for a query along a row.)  (With whole tiles of logits exchanged and every
// exponential taken by both, 64 nodes over 4,096 entries took 184 us instead of 174.)  The peer's P' go from shared to tensor memory by the tensor core's own copies, in
// order with the products.
//
// tree_prep_kernel runs first: q^ (rotated, its RMS factor but for a power of two left to the logits) as
// the swizzled image of the A operand, the RoPE table, and for every slot its row (-1: none), f (the window's rows: once for all nodes), and as
// bits which nodes attend to it.  (A row's squares need all of its dims, of which a CTA has half: with
// the sums exchanged like the logits, and the rows through registers for them, the loaders were what a
// tile waited for.)  It reads the row of every slot once: of 8 x 24 nodes of 128 heads, 133 of them used, 136,192
// rows of 1 KB in 24.7 us, 5.6 TB/s, beside 50 MB of queries read and images written.
//
// Warps (768 threads, one CTA an SM):
//   0       query images (bulk copies)
//   1       half logits; owns tensor memory (O: columns 0-255, S / P': two buffers of 128)
//   2       the tiles' masks and factors
//   3       products.  (Both kinds of MMA from one thread: its time to issue them, 3.4K cycles a tile, was
//           what a tile took; 174 us instead of 159.)
//   4-11    softmax, two warps a lane quarter (32 of the CTA's 64 slots each)
//   12-19   loaders, 16 rows of a tile each: bf16 rows that follow one another by tensor copies, others
//           by 16-byte asynchronous copies into the swizzled tile, FP4 rows dequantised (exactly) from
//           registers that are filled a tile ahead
//   20-23   outputs, a row a thread.  (By the loaders: 8 x 32 nodes over FP4 pages 104 us, not 97.)
// Every wait is bounded; the CTAs meet at the cluster's barrier before either one exits.
//
// Two tiles are in flight (they fill shared memory, their logits tensor memory): each is loaded (1.0-1.3K
// cycles; FP4 2.4K), multiplied (1.5K), weighed (2.2K), multiplied again (1.4K) before the next but one is,
// so that a tile takes 3.6K cycles where its MMAs take 2.2K and its shared-memory traffic 2.6K.  Tiles of 64
// slots, four in flight, were slower (216 us where 128 took 184: a half logit's MMA of N = 64 reads as much
// of Q^), as were 4 or 16 loader warps (at 16 the registers of a thread no longer hold the softmax).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "fp4_tile.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"
#include "tree_tc.cuh"

namespace {

using namespace sm100;

constexpr unsigned FULL = 0xffffffffu;
constexpr int TT_C = 512, TT_HALF = 256;
constexpr int TT_ROWS = 128, TT_TILE = 128;
constexpr int TT_G = 8;                          // nodes of a group at most
constexpr int TT_LOADERS = 8;                    // warps
constexpr int TT_OUT = 4;                        // warps that store outputs
constexpr int TT_THREADS = 32 * (12 + TT_LOADERS + TT_OUT);
constexpr int TT_CHUNK = TT_TILE * 128;          // 16 KB: 128 rows x 64 dims
constexpr int TT_TILE_BYTES = 4 * TT_CHUNK;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr long long TT_BUDGET = 1ll << 31;
// Half logits as 16-bit integers: y * TT_FIX + TT_FIX_AT in fp32 has the rounded multiple plus 2^15 in its low 16
// bits.  A half logit is at most sqrt(512) / ln 2 = 32.65, 2^-8 more with the rotated dims rounded to bf16:
// 32.78 * 992 = 32,515, inside 16 bits.
constexpr float TT_FIX = 992.0f, TT_FIX_AT = 8388608.0f + 32768.0f;

constexpr int OFF_Q = 0;
constexpr int OFF_Y = 65536;                             // the peer's P': [2 groups][4 units of 8 slots][128 rows] x 16 B
constexpr int OFF_X = OFF_Y + 16384;                     // its half logits, the same
constexpr int OFF_K = OFF_X + 16384;
constexpr int OFF_F = OFF_K + 2 * TT_TILE_BYTES;         // [2][128] the factors f
constexpr int OFF_L = OFF_F + 1024;                      // [2][128] sums of exponentials, by softmax warp of a lane quarter
constexpr int OFF_MASK = OFF_L + 1024;                   // [2][TT_G][4] x 32 bits
constexpr int OFF_BAR = OFF_MASK + 2 * TT_G * 16;
constexpr int N_BAR = 18 + 8 + 2 * 8;
constexpr int OFF_TMEM = OFF_BAR + N_BAR * 8;
constexpr int TT_SMEM = OFF_TMEM + 16;
static_assert(TT_SMEM <= 227 * 1024, "shared memory");

// What the prep kernel leaves for the main one.
struct TtLists {
    uint8_t* qimg;                // [groups][2 halves][4 chunks][R8 rows x 128 B]
    float* qm;                    // [groups][R8] what the image's rows are yet to be multiplied by, in [1, 2)
    int32_t* erow;                // [eg][lde] rows of the entry slots (eg: nodes; dense: sequences)
    float* ef;                    // [eg][lde] their factors f
    uint32_t* eok;                // [eg][lde / 32] which of them there are
    int32_t* wrow;                // [groups][ldw] rows of the window slots: the ring's, then drafts
    uint32_t* wmask;              // [groups][ldw / 32][TT_G] who attends to them
    float* rf;                    // [B][window] factors of the ring's last rows: position ctx_len - window + j
    float* df;                    // [B*T] of the drafts
    int4* info;                   // [groups] entry slots (a multiple of 32), all, the ring's, their first j in rf
    float* rope_cs;               // [B*T, 64] cos, sin of the 32 angles
    int lde, ldw;
    int64_t drafts;               // B*T
    int H, G, R8, gps;            // heads, nodes of a group, image rows, groups of a sequence
};

struct TtArgs {
    TtLists l;
    TreeRows r;
    const uint8_t* kv;
    const uint8_t* swa;
    const uint8_t* draft;
    const float* sink;
    int groups, rounds, clusters; // cluster c has groups c, c + clusters, .. whole, `rounds` of them
    int share, tiles;             // and of the others' tiles (at most `tiles` a group) `share`
    unsigned flags;
    void* out;
    int out_f32;
    float* lse;
    int pieces;                   // in which the others are dealt out, at most
    float* part_o;                // [the others * pieces][G*H rows][512] (pieces > 1)
    float* part_l;                // [the others * pieces][G*H rows]
    unsigned* st;
    long long budget;
    int stall;
};

struct TtMaps {                   // bf16 rows of 512, boxes of 64 dims x the rows of a loader: cache, ring, drafts
    CUtensorMap m[3];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of p in CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// 128 rows of 32 bytes into tensor memory: units of 16 bytes a row, 8 rows of a unit side by side
// (sdesc_plain).  In order with the MMAs that the same thread issues.
__device__ __forceinline__ void tmem_cp_128x256b(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// A K-major matrix without swizzle: `lbo` bytes from one 16-byte unit of a row to the next, `sbo` from
// 8 rows of a unit to the next 8.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | (uint64_t)1 << 46;
}
// An arrival at the barrier of the same address in CTA `rank` of the cluster, when everything this
// thread has issued to the tensor cores is done.
__device__ __forceinline__ void mma_commit_to(uint64_t* bar, uint32_t rank) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)(1u << rank))
                 : "memory");
}

// An arrival at a barrier of the peer's that says "read": the values read are in registers, and
// nothing this thread wrote is behind it, so it carries no fence (a release at the cluster's scope
// waits for every access of the thread).
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Stores into the peer's shared memory that count their bytes at one of its barriers.
__device__ __forceinline__ void peer_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void peer_st1(uint32_t addr, uint32_t a, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(a), "r"(bar) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two fp32 values in a register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t two(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 two_of(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 32 bytes to global memory: one access, so that a thread with a row of its own writes whole sectors, or two
// where the address is a multiple of 16 only.
__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8], bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// A cluster's items: `rounds` whole groups, then its share of the groups that are left over: their tiles
// stand one behind the other, `tiles` a group (a shorter one leaves its last ones out), and cluster c has
// `share` of them from c * share on.
struct TtItem {
    int v, b, n0, gv;             // group, sequence, first node in it, nodes
    int kq, slots, ring, rf;      // entry slots, all slots, the ring's among the others, the first one's j in rf
    int t0, nt;                   // tiles t0 .. t0 + nt - 1
    int piece, pieces;            // of the group
    int part;                     // its first piece's place among the partial outputs
};

struct TtWalk {
    int cluster, round;
    int v, at, left;              // leftover group, tile in it, tiles left to the cluster
    int4 info;                    // the next item's group's, loaded an item ahead

    __device__ __forceinline__ int group(const TtArgs& a) const {        // of the next item, -1: none
        return round < a.rounds ? round * a.clusters + cluster : (left > 0 ? a.rounds * a.clusters + v : -1);
    }
    __device__ __forceinline__ void load(const TtArgs& a) {
        const int g = group(a);
        info = g >= 0 ? a.l.info[g] : make_int4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void start(const TtArgs& a, int c) {
        cluster = c;
        round = 0;
        const int64_t f0 = (int64_t)c * a.share, rest = (int64_t)(a.groups - a.rounds * a.clusters) * a.tiles;
        v = (int)(f0 / a.tiles);
        at = (int)(f0 - (int64_t)v * a.tiles);
        left = (int)max((int64_t)0, min((int64_t)a.share, rest - f0));
        load(a);
    }
    // The next item; false at the end.  One without slots (an empty group, a short one's last tiles) gets a
    // tile of masked slots, so that no role meets a special case.
    __device__ __forceinline__ bool next(const TtArgs& a, TtItem& r) {
        r.v = group(a);
        if (r.v < 0) return false;
        r.b = r.v / a.l.gps;
        r.n0 = (r.v - r.b * a.l.gps) * a.l.G;
        r.gv = min(a.l.G, a.r.T - r.n0);
        r.kq = info.x;
        r.slots = info.y;
        r.ring = info.z;
        r.rf = info.w;
        int to = a.tiles;
        r.t0 = 0;
        r.piece = 0;
        r.pieces = 1;
        if (round < a.rounds) {
            ++round;
        } else {
            to = min(a.tiles, at + left);
            r.t0 = at;
            if (a.pieces > 1) {
                const int64_t g0 = (int64_t)v * a.tiles;
                const int c0 = (int)(g0 / a.share);
                r.piece = cluster - c0;
                r.pieces = (int)((g0 + a.tiles - 1) / a.share) - c0 + 1;
                r.part = v * a.pieces;
            }
            left -= to - at;
            ++v;
            at = 0;
        }
        r.nt = max(1, min((r.slots + TT_TILE - 1) / TT_TILE, to) - r.t0);
        load(a);
        return true;
    }
};

// Factor of window slot j of an item, whose row is `row`.
__device__ __forceinline__ float window_factor(const TtArgs& a, const TtItem& it, int j, int row) {
    return j < it.ring ? a.l.rf[(int64_t)it.b * a.r.window + it.rf + j] : (row >= 0 ? a.l.df[row] : 0.0f);
}

// Output scale 1 / (L + e^zs) (for O of P' = p f: times ln 2 sqrt(512)) and log-sum-exp of a row with
// the sum L of its exponentials and the sink logit zs; a row without either gives 0 and -inf.
__device__ __forceinline__ float2 finish_row(float L, float zs) {
    if (L == 0.0f) return make_float2(0.0f, zs);
    const float l = logf(L);
    const float w = zs == -INFINITY ? 1.0f : 1.0f / (1.0f + expf(zs - l));
    const float lse = zs == -INFINITY ? l : fmaxf(l, zs) + log1pf(expf(-fabsf(l - zs)));
    return make_float2(w / L * (LN2 * sqrtf((float)TT_C)), lse);
}

// ---------------------------------------------------------------- before the main kernel
struct PrepArgs {
    TtLists l;
    TreeRows r;
    const __nv_bfloat16* q;
    const uint8_t* kv;
    const uint8_t* swa;
    const uint8_t* draft;
    int fp4;
    // warps: of query rows, of entry slots (32 each), of window slots (32), of the ring's rows (8), of drafts (8)
    int64_t q_warps, e_warps, w_warps, r_warps, d_warps;
    int ew, ww, rw;               // of a list of entries, of a group's window, of a sequence's ring rows
    AgRope rope;
    unsigned flags;
    unsigned* st;
};

// The squares of a lane's 16 values of a bf16 or an FP4 row.
__device__ __forceinline__ float lane_squares(const uint4& u0, const uint4& u1) {
    float q = 0.0f;
    const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xFFFF0000u);
        q = fmaf(lo, lo, fmaf(hi, hi, q));
    }
    return q;
}
__device__ __forceinline__ float lane_squares(const uint2& c, uint32_t scale) {
    const float s = e4m3_to_f32(scale);
    uint32_t q = 0;                              // 4 x code^2 by table, summed as bytes
    const uint32_t w[4] = {c.x & 0x77777777u, (c.x >> 16) & 0x7777u, c.y & 0x77777777u, (c.y >> 16) & 0x7777u};
#pragma unroll
    for (int i = 0; i < 4; ++i) q = __dp4a(__byte_perm(0x09040100u, 0x90402410u, w[i]), 0x01010101u, q);
    return (float)q * 0.25f * (s * s);
}

// Factors f of `n` rows (a multiple of 8, at most 32) at base + row * bytes, lane j's `row` that of row j
// (-1: none, f 0), eight rows in flight.  A row with an infinity or a NaN has f NaN.  (The loads are coherent
// ones, past L1: this kernel may start while the one before still writes rows, so to the read-only path they
// would not be read-only for as long as it runs.)
__device__ __forceinline__ float row_factors(const uint8_t* base, int64_t bytes, bool fp4, int row, int n) {
    const int lane = threadIdx.x & 31;
    float sum = 0.0f;
    for (int i = 0; i < n; i += 8) {
        float q[8];
        if (fp4) {
            uint2 c[8];
            uint32_t s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint8_t* p = base + max(0, __shfl_sync(FULL, row, i + j)) * bytes;
                c[j] = __ldcg(reinterpret_cast<const uint2*>(p) + lane);
                s[j] = __ldcg(p + TT_C / 2 + lane);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = lane_squares(c[j], s[j]);
        } else {
            uint4 u[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4* p = reinterpret_cast<const uint4*>(base + max(0, __shfl_sync(FULL, row, i + j)) * bytes) + lane;
                u[j][0] = __ldcg(p);
                u[j][1] = __ldcg(p + 32);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = lane_squares(u[j][0], u[j][1]);
        }
        // sums over the lanes: of two rows' parts a lane keeps one and sends the other; lane l ends with
        // row l / 4's
#pragma unroll
        for (int o = 16, m = 4; m > 0; o >>= 1, m >>= 1) {
            const bool upper = lane & o;
#pragma unroll
            for (int j = 0; j < m; ++j) q[j] = (upper ? q[j + m] : q[j]) + __shfl_xor_sync(FULL, upper ? q[j] : q[j + m], o);
        }
        q[0] += __shfl_xor_sync(FULL, q[0], 2);
        q[0] += __shfl_xor_sync(FULL, q[0], 1);
        const float t = __shfl_sync(FULL, q[0], 4 * (lane & 7));
        if ((lane & 24) == i) sum = t;
    }
    if (row < 0) return 0.0f;
    return sum < INFINITY ? (LOG2E / sqrtf((float)TT_C)) / sqrtf(sum / (float)TT_C + 1e-6f) : __int_as_float(0x7FC00000);
}

constexpr int TT_QROWS = 2;                      // query rows of a warp (images have multiples of 8)

// A warp: a few query rows; 32 entry slots of a node (dense: of a sequence); 32 slots of a group's window; 8 rows
// of a ring; or 8 drafts.
__global__ void __launch_bounds__(256) tree_prep_kernel(const PrepArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, T = a.r.T;
    const bool dense = a.r.n_visible;
    int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    // the long chains of loads first
    if (w < a.e_warps) {
        // entries: those the node selected, or those that any node of the sequence sees
        const int64_t eg = w / a.ew, b = dense ? eg : eg / T;
        const int s0 = (int)(w - eg * a.ew) * 32, s = s0 + lane;
        int live = 0;
        if (dense) {
            for (int i = lane; i < T; i += 32) live = max(live, tree_node(a.r, b * T + i).kq);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) live = max(live, __shfl_xor_sync(FULL, live, o));
        } else {
            live = tree_node(a.r, eg).kq;
        }
        if (s0 >= live) return;
        const int row = s < live ? (int)tree_entry_row(a.r, b, dense ? s : a.r.idx[eg * a.r.k + s], a.st, true) : -1;
        const uint32_t bits = __ballot_sync(FULL, row >= 0);
        if (lane == 0) a.l.eok[eg * (a.l.lde / 32) + s0 / 32] = bits;
        const float f = bits ? row_factors(a.kv, a.fp4 ? fp4_row_bytes(TT_C) : TT_C * 2, a.fp4, row, 32) : 0.0f;
        // (0 x NaN would reach the nodes that do not attend to the row: it keeps out of the products, and its
        // factor, NaN, is for those that do)
        a.l.erow[eg * a.l.lde + s] = f == f ? row : -1;
        a.l.ef[eg * a.l.lde + s] = f;
        return;
    }
    w -= a.e_warps;
    if (w < a.w_warps) {
        // the window: the ring's rows that any node sees, then the drafts: those of the node's path, or of all
        // nodes up to the group's last one
        const int v = (int)(w / a.ww), b = v / a.l.gps, n0 = (v - b * a.l.gps) * a.l.G, gv = min(a.l.G, T - n0);
        const int64_t bt0 = (int64_t)b * T + n0;
        const int s0 = (int)(w - (int64_t)v * a.ww) * 32, s = s0 + lane;
        // lane g: node g's position and entries
        const TreeNode node = tree_node(a.r, bt0 + min(lane, gv - 1));
        const int64_t t = lane < gv ? node.t : -1, len = node.len, W = a.r.window;
        int kq = node.kq;
        int64_t tmin = t >= 0 ? t : INT64_MAX;
#pragma unroll
        for (int o = TT_G / 2; o > 0; o >>= 1) {
            kq = max(kq, __shfl_xor_sync(FULL, kq, o));
            tmin = min(tmin, __shfl_xor_sync(FULL, tmin, o));
        }
        kq = __shfl_sync(FULL, kq, 0);
        tmin = __shfl_sync(FULL, tmin, 0);
        const bool any = W > 0 && tmin != INT64_MAX;
        const int64_t p0 = any ? max((int64_t)0, max(len - W + 1, tmin - W + 1)) : 0;
        const int nring = any ? (int)max((int64_t)0, min(len, tmin + 1) - p0) : 0;
        const int ndraft = !any ? 0 : (dense ? n0 + gv : (int)max((int64_t)0, min(W, tmin + 1 - max(len, p0))));
        const int slots = nring + ndraft;
        if (s0 == 0 && lane == 0) {
            const int kq32 = (kq + 31) / 32 * 32;
            a.l.info[v] = make_int4(kq32, kq32 + slots, nring, (int)(p0 - (len - W)));
        }
        if (s0 >= slots) return;
        const int d = s - nring;
        int64_t p = -1, row = -1;                // position of the slot, its row
        int j = -1;                              // draft node
        if (s < nring) {
            p = p0 + s;
            row = b * a.r.swa_cap + ((p - a.r.swa_pos0) % a.r.swa_cap + a.r.swa_cap) % a.r.swa_cap;
        } else if (d < ndraft) {
            if (dense) {
                j = d;
                p = a.r.pos[(int64_t)b * T + j];
                if (p < len || p - len >= T) j = -1;
            } else {
                int kind;
                p = max(len, p0) + d;
                const int64_t at = tree_window_row(a.r, tree_node(a.r, bt0), p, kind, a.st, true);
                if (at >= 0) j = (int)(at - (int64_t)b * T);
            }
            if (j >= 0) row = (int64_t)b * T + j;
        }
        uint32_t* mask = a.l.wmask + (v * (int64_t)(a.l.ldw / 32) + s0 / 32) * TT_G;
        bool wanted = false;
        for (int g = 0; g < gv; ++g) {
            const int64_t tg = __shfl_sync(FULL, t, g);
            bool on = row >= 0 && tg >= 0 && p <= tg && p > tg - W;
            if (on && j >= 0) on = a.r.path[(bt0 + g) * T + (p - len)] == j;
            const uint32_t bits = __ballot_sync(FULL, on);
            if (lane == 0) mask[g] = bits;
            wanted |= on;
        }
        a.l.wrow[v * (int64_t)a.l.ldw + s] = wanted ? (int32_t)row : -1;
        return;
    }
    w -= a.w_warps;
    if (w < a.r_warps) {
        const int64_t b = w / a.rw, W = a.r.window;
        const int j0 = (int)(w - b * a.rw) * 8, j = j0 + (lane & 7);
        const int64_t p = a.r.ctx_len[b] - W + j;
        const int row = p >= 0 && j < W ? (int)(((p - a.r.swa_pos0) % a.r.swa_cap + a.r.swa_cap) % a.r.swa_cap) : -1;
        const float f = row_factors(a.swa + b * a.r.swa_cap * (TT_C * 2), TT_C * 2, false, row, 8);
        if (lane < 8 && j < W) a.l.rf[b * W + j] = f;
        return;
    }
    w -= a.r_warps;
    if (w < a.d_warps) {
        const int64_t n = a.l.drafts, i = w * 8 + (lane & 7);
        const float f = row_factors(a.draft, TT_C * 2, false, i < n ? (int)i : -1, 8);
        if (lane < 8 && i < n) a.l.df[i] = f;
        return;
    }
    w -= a.d_warps;
    if (w >= a.q_warps) return;
    // query rows: all of a warp's are loaded before the first is used; the angles are a node's
    const int per = a.l.R8 / TT_QROWS, v = (int)(w / per), b = v / a.l.gps, n0 = (v - b * a.l.gps) * a.l.G, gv = min(a.l.G, T - n0);
    const int64_t bt0 = (int64_t)b * T + n0;
    const int row0 = (int)(w - (int64_t)v * per) * TT_QROWS;
    uint4 u[TT_QROWS][2];
    float ss[TT_QROWS];
#pragma unroll
    for (int k = 0; k < TT_QROWS; ++k) {
        u[k][0] = u[k][1] = make_uint4(0u, 0u, 0u, 0u);
        if (row0 + k < gv * a.l.H) {
            const uint4* p = reinterpret_cast<const uint4*>(a.q + (bt0 * a.l.H + row0 + k) * (int64_t)TT_C + 16 * lane);
            u[k][0] = p[0];
            u[k][1] = p[1];
        }
    }
#pragma unroll
    for (int k = 0; k < TT_QROWS; ++k) ss[k] = lane_squares(u[k][0], u[k][1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < TT_QROWS; ++k) ss[k] += __shfl_xor_sync(FULL, ss[k], o);
    int at = -1;                             // the node of the angles
    float cj[8], sj[8];
#pragma unroll
    for (int k = 0; k < TT_QROWS; ++k) {
        const int row = row0 + k, g = row / a.l.H;
        // the row times a power of two, which is exact, and the rest of its RMS factor for the logits (rounded
        // to bf16 with the whole factor, q^ moved every logit by 2^-8 / 3; now only its rotated dims are)
        const float rms = 1.0f / sqrtf(ss[k] / (float)TT_C + 1e-6f), r = __uint_as_float(__float_as_uint(rms) & 0x7F800000u);
        if (lane == 0) a.l.qm[v * (int64_t)a.l.R8 + row] = rms / r;
        const uint32_t c8[8] = {u[k][0].x, u[k][0].y, u[k][0].z, u[k][0].w, u[k][1].x, u[k][1].y, u[k][1].z, u[k][1].w};
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = __uint_as_float(c8[i] << 16) * r;
            x[2 * i + 1] = __uint_as_float(c8[i] & 0xFFFF0000u) * r;
        }
        if ((a.flags & CSA2_ROPE) && g < gv) {
            if (g != at) {
                // lane j has angle j; lanes 28 .. 31 rotate the pairs of dims 448 .. 511
                float c, s;
                ag_cos_sin(a.rope, a.r.pos[bt0 + g], lane, c, s);
                if (row == g * a.l.H) {
                    a.l.rope_cs[(bt0 + g) * 64 + lane] = c;
                    a.l.rope_cs[(bt0 + g) * 64 + 32 + lane] = s;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cj[i] = __shfl_sync(FULL, c, (8 * (lane - 28) + i) & 31);
                    sj[i] = __shfl_sync(FULL, s, (8 * (lane - 28) + i) & 31);
                }
                at = g;
            }
            if (lane >= 28) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = x[2 * i], x1 = x[2 * i + 1];
                    x[2 * i] = x0 * cj[i] - x1 * sj[i];
                    x[2 * i + 1] = x1 * cj[i] + x0 * sj[i];
                }
            }
        }
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        uint8_t* img = a.l.qimg + v * (int64_t)a.l.R8 * 1024 + (lane >> 2) * (int64_t)a.l.R8 * 128;      // chunk of 64 dims
        const uint32_t un = 2 * (lane & 3);
        *reinterpret_cast<uint4*>(img + sw128_offset(row, un)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(img + sw128_offset(row, un + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// ---------------------------------------------------------------- the main kernel

// The sixteen E2M1 codes of a scale block (eight a word, value 2k in the low nibble of byte k) times
// their E4M3 scale as bf16 pairs: the eight magnitudes times the scale (exact: 6 significant bits) as a
// table of low and one of high bytes, from which a code's 3 magnitude bits pick by byte permutes, its sign
// XORed in.  (Conversions of single codes run in the pipe that the softmax's exponentials need.)
__device__ __forceinline__ void fp4_16(uint32_t wa, uint32_t wb, uint32_t scale, uint4& va, uint4& vb) {
    const uint32_t s2 = __byte_perm(__float_as_uint(e4m3_to_f32(scale)), 0u, 0x3232);     // (bf16 scale, bf16 scale)
    const uint32_t t01 = bf16x2_mul(0x3F000000u, s2);                     // (0, 0.5) x scale
    const uint32_t t23 = bf16x2_mul(0x3FC03F80u, s2);                     // (1, 1.5)
    const uint32_t t45 = bf16x2_mul(0x40404000u, s2);                     // (2, 3)
    const uint32_t t67 = bf16x2_mul(0x40C04080u, s2);                     // (4, 6)
    const uint32_t lo0 = __byte_perm(t01, t23, 0x6420), hi0 = __byte_perm(t01, t23, 0x7531);
    const uint32_t lo1 = __byte_perm(t45, t67, 0x6420), hi1 = __byte_perm(t45, t67, 0x7531);
    const auto word = [&](uint32_t w) {
        const uint32_t m = w & 0x77777777u, mh = m >> 16, w4 = w << 4;
        uint32_t lo = __byte_perm(lo0, lo1, m), hi = __byte_perm(hi0, hi1, m);
        uint4 r;
        r.x = __byte_perm(lo, hi, 0x5140) ^ (__byte_perm(w4, w, 0x4000) & 0x80008000u);
        r.y = __byte_perm(lo, hi, 0x7362) ^ (__byte_perm(w4, w, 0x5010) & 0x80008000u);
        lo = __byte_perm(lo0, lo1, mh);
        hi = __byte_perm(hi0, hi1, mh);
        r.z = __byte_perm(lo, hi, 0x5140) ^ (__byte_perm(w4, w, 0x6020) & 0x80008000u);
        r.w = __byte_perm(lo, hi, 0x7362) ^ (__byte_perm(w4, w, 0x7030) & 0x80008000u);
        return r;
    };
    va = word(wa);
    vb = word(wb);
}

template <bool FP4, bool DENSE>
__global__ void __launch_bounds__(TT_THREADS, 1) __cluster_dims__(2, 1, 1)
    tree_tc_kernel(const TtArgs a, const __grid_constant__ TtMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sQ = smem + OFF_Q;
    uint8_t* sK = smem + OFF_K;
    uint8_t* sX = smem + OFF_X;
    uint8_t* sY = smem + OFF_Y;
    float* sF = reinterpret_cast<float*>(smem + OFF_F);
    float* sL = reinterpret_cast<float*>(smem + OFF_L);
    uint32_t* sMask = reinterpret_cast<uint32_t*>(smem + OFF_MASK);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* qfull = bars + 0;
    uint64_t* qempty = bars + 1;
    uint64_t* kfull = bars + 2;        // [2] a tile's rows are in shared memory
    uint64_t* sfull = bars + 4;        // [2] its half logits, its factors and masks
    uint64_t* pfull = bars + 6;        // [2] the P' of the slots that this CTA weighs
    uint64_t* yfull = bars + 8;        // the peer's P'
    uint64_t* yempty = bars + 9;       // the peer has taken this CTA's
    uint64_t* ofull = bars + 10;
    uint64_t* oempty = bars + 11;
    uint64_t* lred = bars + 12;
    uint64_t* done = bars + 13;        // [2] the last half logits, the last products
    uint64_t* kempty = bars + 18;      // [2][4] the products of a tile's 32-row groups are done
    uint64_t* xfull = bars + 26;       // [8] the peer's half logits for a softmax warp, its sums
    uint64_t* xempty = bars + 34;      // [8] the peer has read this warp's
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
    const int cluster = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        if (smem_u32(smem) & 1023u) csa2_flag(a.st, CSA2_DEVBIT_TIMEOUT);
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], TT_LOADERS);
            for (int j = 0; j < 4; ++j) mbar_init(&kempty[4 * i + j], 1);
            mbar_init(&sfull[i], 2);
            mbar_init(&pfull[i], 8);
        }
        mbar_init(yfull, 1);
        mbar_init(yempty, 1);
        mbar_init(ofull, 1);
        mbar_init(oempty, TT_OUT);
        mbar_init(lred, 8);
        mbar_init(&done[0], 1);
        mbar_init(&done[1], 1);
        for (int i = 0; i < 8; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 1);
        }
        fence_mbar_init();
        for (int i = 0; i < 3; ++i) prefetch_tmap(&maps.m[i]);
    }
    if (warp == 1) {
        tmem_alloc(sTmem, 512);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();                // the peer's barriers are initialised
    const uint32_t tmem = *sTmem;
    TtWalk walk;
    TtItem it;
    walk.start(a, cluster);

    if (warp == 0) {
        // ============================ query images ============================
        if (lane == 0) {
            int qi = 0, issued = -1;
            while (!a.stall && walk.next(a, it)) {
                if (qi > 0 && !mbar_wait(qempty, (qi - 1) & 1, a.budget, a.st)) break;
                const uint32_t bytes = (uint32_t)a.l.R8 * 128u;
                mbar_arrive_expect_tx(qfull, 4 * bytes);
                const uint8_t* src = a.l.qimg + ((int64_t)it.v * 2 + rank) * 4 * bytes;
                for (int c = 0; c < 4; ++c) bulk_g2s(sQ + c * TT_CHUNK, src + (int64_t)c * bytes, bytes, qfull);
                issued = qi++;
            }
            if (issued >= 0) mbar_wait(qfull, issued & 1, a.budget, a.st);
        }
    } else if (warp == 1) {
        // ============================ half logits ============================
        if (lane == 0) {
            constexpr uint32_t IDESC_QK = idesc_f16(TT_ROWS, TT_TILE, true);
            // descriptors of the operands' first bytes: an address further on adds to the low field
            const uint64_t dq = sdesc_sw128(smem_u32(sQ)), dk = sdesc_sw128(smem_u32(sK));
            int g = 0, qi = 0;
            bool ok = true;
            while (ok && walk.next(a, it)) {
                ok = mbar_wait(qfull, qi++ & 1, a.budget, a.st);
                for (int tt = 0; tt < it.nt && ok; ++tt, ++g) {
                    // (a tile's rows are there: the products of the tile two before, which read its P' from where
                    // the logits go, are done)
                    const int buf = g & 1;
                    ok = mbar_wait(&kfull[buf], (g >> 1) & 1, a.budget, a.st);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sc = tmem + 256 + 128 * buf, kb = (uint32_t)buf * (TT_TILE_BYTES >> 4);
#pragma unroll
                    for (uint32_t kk = 0; kk < 16; ++kk) {
                        const uint32_t o = ((kk >> 2) * TT_CHUNK + (kk & 3) * 32u) >> 4;
                        mma_ss(sc, dq + o, dk + (kb + o), IDESC_QK, kk != 0);
                    }
                    mma_commit(&sfull[buf]);
                    if (tt == it.nt - 1) mma_commit(qempty);
                }
            }
            // the MMAs must be complete before tensor memory is released
            mma_commit(&done[0]);
            mbar_wait(&done[0], 0, a.budget, a.st);
        }
    } else if (warp == 3) {
        // ============================ outputs ============================
        if (lane == 0) {
            constexpr uint32_t IDESC_PV = idesc_f16_major(TT_ROWS, TT_HALF, true, false, true);
            const uint64_t dv = sdesc_sw128_mn(smem_u32(sK), TT_CHUNK, 1024);
            const uint64_t dy = sdesc_plain(smem_u32(sY), TT_ROWS * 16, 128);
            const uint32_t y_bytes = (uint32_t)((a.l.G * a.l.H + 31) / 32) * 2 * (32 * 4 * 16);      // of the warps with rows
            int g = 0, qi = 0;
            bool ok = true;
            while (ok && walk.next(a, it)) {
                for (int tt = 0; tt < it.nt && ok; ++tt, ++g) {
                    const int buf = g & 1;
                    const uint32_t kb = (uint32_t)buf * (TT_TILE_BYTES >> 4), p = tmem + 256 + 128 * buf;
                    const auto products = [&](uint32_t ks0, bool first) {
#pragma unroll
                        for (uint32_t i = 0; i < 4; ++i) {
                            const uint32_t ks = ks0 + i;
                            mma_ts(tmem, p + (ks >> 1) * 32 + (ks & 1) * 8, dv + (kb + ks * (2048 >> 4)), IDESC_PV, !first || i > 0);
                            if (i & 1) mma_commit(&kempty[4 * buf + (ks >> 1)]);
                        }
                    };
                    mbar_arrive_expect_tx(yfull, y_bytes);
                    ok = mbar_wait(&pfull[buf], (g >> 1) & 1, a.budget, a.st) &&
                         (tt > 0 || qi == 0 || mbar_wait(oempty, (qi - 1) & 1, a.budget, a.st));
                    if (!ok) break;
                    tc_fence_after();
                    products(4 * rank, tt == 0);
                    // the peer's P' beside this CTA's (its slots' half logits are with the peer)
                    ok = mbar_wait(yfull, g & 1, a.budget, a.st);
                    if (!ok) break;
                    fence_proxy_async_smem();
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        tmem_cp_128x256b(p + 64 * peer + 32 * (i >> 1) + 8 * (i & 1), dy + i * (2 * TT_ROWS * 16 >> 4));
                    mma_commit_to(yempty, peer);
                    products(4 * peer, false);
                }
                if (!ok) break;
                mma_commit(ofull);
                ++qi;
            }
            mma_commit(&done[1]);
            mbar_wait(&done[1], 0, a.budget, a.st);
        }
    } else if (warp == 2) {
        // ============================ masks and factors ============================
        // lane 4 n + w: word w (32 slots) of node n
        const int n = lane >> 2, w = lane & 3;
        int g = 0;
        bool ok = true;
        while (ok && walk.next(a, it)) {
            const int64_t eg = DENSE ? it.b : (int64_t)it.b * a.r.T + it.n0;
            int seen = it.kq;
            if (DENSE && n < it.gv && a.r.k > 0)
                seen = a.r.pos[(int64_t)it.b * a.r.T + it.n0 + n] < 0
                           ? 0
                           : (int)max((int64_t)0, min((int64_t)a.r.k, a.r.n_visible[(int64_t)it.b * a.r.T + it.n0 + n]));
            for (int tt = 0; tt < it.nt && ok; ++tt, ++g) {
                const int s = (it.t0 + tt) * TT_TILE + 32 * w;
                uint32_t m = 0;
                if (n < it.gv && s < it.slots) {
                    if (s < it.kq) {
                        m = a.l.eok[eg * (a.l.lde / 32) + s / 32];
                        if (seen < s + 32) m &= seen > s ? (1u << (seen - s)) - 1u : 0u;
                    } else {
                        m = a.l.wmask[((int64_t)it.v * (a.l.ldw / 32) + (s - it.kq) / 32) * TT_G + n];
                    }
                }
                // lane l: the factors of slots 4 l .. 4 l + 3 (lists of entries are padded to multiples of 32)
                const int s4 = (it.t0 + tt) * TT_TILE + 4 * lane;
                float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (s4 < it.kq) {
                    f = *reinterpret_cast<const float4*>(a.l.ef + eg * a.l.lde + s4);
                } else {
                    float* fw = &f.x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = s4 + i - it.kq;
                        if (s4 + i < it.slots) fw[i] = window_factor(a, it, j, a.l.wrow[(int64_t)it.v * a.l.ldw + j]);
                    }
                }
                // (its products done, a tile's softmax has read its masks)
                const bool wt = g < 2 || mbar_wait(&kempty[4 * (g & 1) + 2 * peer + 1], ((g - 2) >> 1) & 1, a.budget, a.st);
                ok = __all_sync(FULL, wt);
                if (!ok) break;
                sMask[((g & 1) * TT_G + n) * 4 + w] = m;
                *reinterpret_cast<float4*>(sF + (g & 1) * TT_TILE + 4 * lane) = f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfull[g & 1]);
            }
        }
    } else if (warp >= 4 && warp < 12) {
        // ============================ softmax ============================
        const int quad = warp & 3, hh = (warp - 4) >> 2, w = 4 * hh + quad;
        const int r = quad * 32 + lane;                       // query row
        const bool live = quad * 32 < a.l.G * a.l.H;          // a warp without query rows only keeps step
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const int g_row = min(r / a.l.H, a.l.G - 1);
        // 32-slot groups of a tile: the one that this warp weighs, the one of its twin in the peer
        const int own = 2 * rank + hh, other = 2 * peer + hh;
        uint8_t* mine_x = sX + (hh * 4 * TT_ROWS + r) * 16;
        const uint32_t their_x = peer_addr(mine_x, peer), their_y = peer_addr(sY + (hh * 4 * TT_ROWS + r) * 16, peer);
        const uint32_t x_full = peer_addr(&xfull[w], peer), x_empty = peer_addr(&xempty[w], peer), y_full = peer_addr(yfull, peer);
        int g = 0, qi = 0;
        int nx = 0;                                           // exchanges by way of sX so far
        uint64_t lsum = two(0.0f, 0.0f);
        bool ok = true;
        uint64_t qm = 0;                                      // the row's factor times TT_FIX, twice
        const uint64_t fix_at = two(TT_FIX_AT, TT_FIX_AT), minus_at = two(-TT_FIX_AT, -TT_FIX_AT), unfix = two(1.0f / TT_FIX, 1.0f / TT_FIX);
        const auto weigh = [&]() {
            // (the peer has read the last exchange long before this tile's logits come)
            bool wt = (nx == 0 || !live || mbar_wait(&xempty[w], (nx - 1) & 1, a.budget, a.st)) &&
                      mbar_wait(&sfull[g & 1], (g >> 1) & 1, a.budget, a.st);
            ok = __all_sync(FULL, wt);
            if (!ok) return;
            tc_fence_after();
            const uint32_t s_col = lanes + 256 + 128 * (g & 1);
            if (live) {
                // the half logits of the peer's slots to the peer
                const float4* fac = reinterpret_cast<const float4*>(sF + (g & 1) * TT_TILE + 32 * other);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t sv[16], y[8];
                    tmem_ld16(s_col + 32 * other + 16 * i, sv);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 f = fac[4 * i + j];
                        const uint64_t s0 = two(__uint_as_float(sv[4 * j]), __uint_as_float(sv[4 * j + 1]));
                        const uint64_t s1 = two(__uint_as_float(sv[4 * j + 2]), __uint_as_float(sv[4 * j + 3]));
                        const float2 y0 = two_of(fma2(s0, mul2(two(f.x, f.y), qm), fix_at)), y1 = two_of(fma2(s1, mul2(two(f.z, f.w), qm), fix_at));
                        y[2 * j] = __byte_perm(__float_as_uint(y0.x), __float_as_uint(y0.y), 0x5410);
                        y[2 * j + 1] = __byte_perm(__float_as_uint(y1.x), __float_as_uint(y1.y), 0x5410);
                    }
                    peer_st4(their_x + 2 * i * TT_ROWS * 16, y[0], y[1], y[2], y[3], x_full);
                    peer_st4(their_x + (2 * i + 1) * TT_ROWS * 16, y[4], y[5], y[6], y[7], x_full);
                }
                // (a warp without rows must not: it could fall two phases behind its peer)
                if (lane == 0) mbar_arrive_expect_tx(&xfull[w], 32 * 4 * 16);
                wt = mbar_wait(&xfull[w], nx & 1, a.budget, a.st) && (g == 0 || mbar_wait(yempty, (g - 1) & 1, a.budget, a.st));
                ++nx;
            }
            ok = __all_sync(FULL, wt);
            if (!ok) return;
            if (live) {
                const float4* fac = reinterpret_cast<const float4*>(sF + (g & 1) * TT_TILE + 32 * own);
                const uint32_t m = sMask[((g & 1) * TT_G + g_row) * 4 + own];
                // p = 2^z, P' = p f in the place of the logits, here and at the peer; 16 slots at a time
                const auto tile_p = [&](auto all) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t sv[16], pk[8];
                        tmem_ld16(s_col + 32 * own + 16 * i, sv);
                        const uint4 o0 = *reinterpret_cast<const uint4*>(mine_x + 2 * i * TT_ROWS * 16);
                        const uint4 o1 = *reinterpret_cast<const uint4*>(mine_x + (2 * i + 1) * TT_ROWS * 16);
                        const uint32_t ov[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
                        const uint32_t mb = m >> (16 * i);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 f4 = fac[4 * i + (j >> 1)];
                            const uint64_t f = (j & 1) ? two(f4.z, f4.w) : two(f4.x, f4.y);
                            // (the 16 bits under the exponent of 2^23 are the peer's value plus TT_FIX_AT again; a
                            // NaN does not survive them, but its row's or query's factor makes one here too)
                            const uint64_t o = add2(two(__uint_as_float(__byte_perm(ov[j], 0x4B00u, 0x5410)),
                                                        __uint_as_float(__byte_perm(ov[j], 0x4B00u, 0x5432))), minus_at);
                            const float2 z = two_of(mul2(fma2(two(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), mul2(f, qm), o), unfix));
                            float p0 = ex2(z.x), p1 = ex2(z.y);
                            if (all) {
                                const uint64_t p = two(p0, p1);
                                lsum = add2(lsum, p);
                                const float2 pf = two_of(mul2(p, f));
                                pk[j] = pack_bf16(pf.x, pf.y);
                            } else {
                                // (a masked slot's factor may be NaN: its product must not count)
                                const bool m0 = (mb >> (2 * j)) & 1u, m1 = (mb >> (2 * j + 1)) & 1u;
                                p0 = m0 ? p0 : 0.0f;
                                p1 = m1 ? p1 : 0.0f;
                                lsum = add2(lsum, two(p0, p1));
                                const float2 ff = two_of(f);
                                pk[j] = pack_bf16(m0 ? p0 * ff.x : 0.0f, m1 ? p1 * ff.y : 0.0f);
                            }
                        }
                        tmem_st8(s_col + 32 * own + 8 * i, pk);
                        peer_st4(their_y + 2 * i * TT_ROWS * 16, pk[0], pk[1], pk[2], pk[3], y_full);
                        peer_st4(their_y + (2 * i + 1) * TT_ROWS * 16, pk[4], pk[5], pk[6], pk[7], y_full);
                    }
                };
                if (__all_sync(FULL, m == FULL)) tile_p(std::true_type{});
                else tile_p(std::false_type{});
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&pfull[g & 1]);
                if (live) peer_arrive(x_empty);
            }
        };
        while (ok && walk.next(a, it)) {
            const float m = r < it.gv * a.l.H ? TT_FIX * a.l.qm[it.v * (int64_t)a.l.R8 + r] : 0.0f;
            qm = two(m, m);
            for (int tt = 0; tt < it.nt && ok; ++tt, ++g) weigh();
            if (!ok) break;
            // the rows' sums: this warp's slots and its twin's; the last item's readers are done with sL
            const float2 ls = two_of(lsum);
            float sum = ls.x + ls.y;
            bool wt = true;
            if (live) {
                wt = mbar_wait(&xempty[w], (nx - 1) & 1, a.budget, a.st);
                ok = __all_sync(FULL, wt);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&xfull[w], 32 * 4);
                peer_st1(their_x, __float_as_uint(sum), x_full);
                wt = mbar_wait(&xfull[w], nx & 1, a.budget, a.st);
                if (wt) sum += *reinterpret_cast<const float*>(mine_x);
                ++nx;
            }
            wt = wt && (qi == 0 || mbar_wait(oempty, (qi - 1) & 1, a.budget, a.st));
            ok = __all_sync(FULL, wt);
            if (ok) sL[hh * TT_ROWS + r] = sum;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(lred);
                if (live) peer_arrive(x_empty);
            }
            ++qi;
            lsum = two(0.0f, 0.0f);
        }
        // (the peer's last arrival at this CTA's barriers)
        if (ok && live && g > 0) mbar_wait(yempty, (g - 1) & 1, a.budget, a.st);
    } else if (warp >= 12 && warp < 12 + TT_LOADERS) {
        // ============================ loaders ============================
        constexpr int ROWS = TT_TILE / TT_LOADERS;            // of a tile, a warp
        const int lw = warp - 12;
        const uint32_t row0 = ROWS * lw;                      // rows row0 .. row0 + ROWS - 1
        // Three steps, each a tile ahead of the one before, so that no load is waited for: the rows' list is
        // read (look_up), the rows are on their way (fetch), they go into the tile.
        int tt = 0;
        it.nt = 0;
        int row = -1, kind = 0;                               // looked up: lane j's row (-1: none) and source
        bool entry = false, more = true;
        const auto look_up = [&]() {
            if (tt >= it.nt) {
                more = more && walk.next(a, it);
                if (!more) return;
                tt = 0;
            }
            const int slot = (it.t0 + tt) * TT_TILE + row0 + (lane & (ROWS - 1)), j = slot - it.kq;
            entry = slot - (lane & (ROWS - 1)) < it.kq;
            kind = entry ? 0 : (j < it.ring ? 1 : 2);
            row = -1;
            if (entry) {
                row = a.l.erow[(DENSE ? it.b : (int64_t)it.b * a.r.T + it.n0) * a.l.lde + slot];
            } else if (slot < it.slots) {
                row = a.l.wrow[(int64_t)it.v * a.l.ldw + j];
                // (a row with a NaN keeps out of the products, as among the entries)
                const float f = window_factor(a, it, j, row);
                if (f != f) row = -1;
            }
            ++tt;
        };
        // FP4 rows through registers: 8 lanes a row, 4 rows an instruction, 16 code bytes and 2 scales a lane
        // (a slot without a row has scales of 0)
        constexpr int FP4_ROWS = ROWS / 4;
        uint4 d[FP4_ROWS];
        uint32_t sc[FP4_ROWS];
        uint64_t at = 0;              // bf16: the address of lane j's row, 0: none
        int box_row = -1, box_map = 0;    // bf16: the first row, where the rows follow one another
        bool fp4_rows = false;
        bool fetched = false;
        const auto fetch = [&]() {
            fetched = more;
            if (!more) return;
            fp4_rows = FP4 && entry;
            const uint8_t* src = nullptr;
            if (row >= 0)
                src = (kind == 0 ? a.kv : (kind == 1 ? a.swa : a.draft)) +
                      (int64_t)row * (fp4_rows ? fp4_row_bytes(TT_C) : (int64_t)(TT_C * 2));
            at = (uint64_t)(uintptr_t)src;
            box_map = kind;
            const int row_0 = __shfl_sync(FULL, row, 0), kind_0 = __shfl_sync(FULL, kind, 0);
            box_row = __all_sync(FULL, row_0 >= 0 && row == row_0 + (lane & (ROWS - 1)) && kind == kind_0) ? row_0 : -1;
            if (fp4_rows) {
#pragma unroll
                for (int i = 0; i < FP4_ROWS; ++i) {
                    const uint8_t* p = reinterpret_cast<const uint8_t*>((uintptr_t)__shfl_sync(FULL, at, 4 * i + (lane >> 3)));
                    const bool real = p;
                    if (!real) p = a.l.qimg;                  // (loads without conditions; the image has 8 KB)
                    d[i] = __ldcg(reinterpret_cast<const uint4*>(p + 128 * rank + 16 * (lane & 7)));
                    const uint32_t two = __ldcg(reinterpret_cast<const unsigned short*>(p + 256 + 16 * rank + 2 * (lane & 7)));
                    sc[i] = real ? two : 0u;
                }
            }
        };
        look_up();
        fetch();
        look_up();
        int g = 0;
        bool ok = true;
        for (; fetched; ++g) {
            const bool wt = g < 2 || mbar_wait(&kempty[4 * (g & 1) + row0 / 32], ((g - 2) >> 1) & 1, a.budget, a.st);
            ok = __all_sync(FULL, wt);
            if (!ok) break;
            uint8_t* tile = sK + (g & 1) * TT_TILE_BYTES;
            uint64_t* full = &kfull[g & 1];
            bool late = false;
            if (fp4_rows) {
                const int piece = lane & 7, c = piece >> 1;
                uint8_t* base = tile + c * TT_CHUNK;
#pragma unroll
                for (int i = 0; i < FP4_ROWS; ++i) {
                    uint8_t* at_row = base + ((row0 + 4 * i + (lane >> 3)) << 7);
                    const uint32_t swz = (4 * i + (lane >> 3)) & 7;
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        // units of 8 values, in an order that differs between the lanes of a row: no bank twice
                        const int blk = hb ^ (c >> 1), odd = c & 1;
                        const uint32_t w0 = blk ? d[i].z : d[i].x, w1 = blk ? d[i].w : d[i].y;
                        uint4 va, vb;
                        fp4_16(odd ? w1 : w0, odd ? w0 : w1, (blk ? sc[i] >> 8 : sc[i]) & 0xFFu, va, vb);
                        const uint32_t u = 4 * (piece & 1) + 2 * blk + odd;
                        *reinterpret_cast<uint4*>(at_row + ((u ^ swz) << 4)) = va;
                        *reinterpret_cast<uint4*>(at_row + (((u ^ 1) ^ swz) << 4)) = vb;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            } else if (box_row >= 0) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, ROWS * TT_HALF * 2);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tma_load_2d(tile + c * TT_CHUNK + row0 * 128, &maps.m[box_map], TT_HALF * rank + 64 * c, box_row, full);
                }
            } else {
                // a row an instruction, 16 bytes a lane
                uint8_t* base = tile + (lane >> 3) * TT_CHUNK;
#pragma unroll 8
                for (uint32_t i = 0; i < ROWS; ++i) {
                    const uint64_t p = __shfl_sync(FULL, at, i);
                    cp_async16_or_zero(base + sw128_offset(row0 + i, (uint32_t)(lane & 7)),
                                       reinterpret_cast<const uint8_t*>((uintptr_t)(p ? p : (uint64_t)(uintptr_t)a.l.qimg)) + 512 * rank + 16 * lane, p != 0);
                }
                cp_async_commit();
                late = true;
            }
            fetch();
            look_up();
            if (late) {
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            }
        }
        // tensor copies must land before the CTA exits
        for (int t = max(0, g - 2); t < g; ++t) mbar_wait(&kfull[t & 1], (t >> 1) & 1, a.budget, a.st);
    } else if (warp >= 12 + TT_LOADERS) {
        // ============================ outputs ============================
        const int quad = warp & 3, r = quad * 32 + lane, hq = r / a.l.H, h = r - hq * a.l.H;
        const bool live = quad * 32 < a.l.G * a.l.H;
        const int d0 = TT_HALF * rank;
        const uint32_t o_col = tmem + ((uint32_t)(quad * 32) << 16);
        int oq = 0;
        const float zs = a.sink && live ? a.sink[h] : -INFINITY;
        // (outputs and workspaces may begin at any multiple of 16 bytes)
        const bool sectors = ((uintptr_t)a.out & 31u) == 0, part_sectors = ((uintptr_t)a.part_o & 31u) == 0;
        while (walk.next(a, it)) {
            const bool valid = r < it.gv * a.l.H, part = it.pieces > 1;
            const int64_t bt = (int64_t)it.b * a.r.T + it.n0 + (valid ? hq : 0), orow = bt * a.l.H + h;
            const int64_t prow = part ? (int64_t)(it.part + it.piece) * (a.l.G * a.l.H) + r : 0;
            // (the sums are there before the last products)
            bool wt = mbar_wait(lred, oq & 1, a.budget, a.st);
            if (!__all_sync(FULL, wt)) break;
            const float L = sL[r] + sL[TT_ROWS + r];
            const float2 fin = part ? make_float2(1.0f, 0.0f) : finish_row(L, zs);
            if (valid && rank == 0) {
                if (part) a.part_l[prow] = L;
                else if (a.lse) a.lse[orow] = fin.y;
            }
            wt = mbar_wait(ofull, oq & 1, a.budget, a.st);
            if (!__all_sync(FULL, wt)) break;
            tc_fence_after();
            // (a piece without slots is left out of the sums)
            if (live && !(part && it.t0 * TT_TILE >= it.slots)) {
                const float* cs = a.l.rope_cs + bt * 64;
                const bool wide = part || a.out_f32, whole = part ? part_sectors : sectors;        // fp32 rows; whole sectors
                uint8_t* dst = part ? reinterpret_cast<uint8_t*>(a.part_o + prow * (int64_t)TT_C)
                                    : reinterpret_cast<uint8_t*>(a.out) + orow * (int64_t)(wide ? TT_C * 4 : TT_C * 2);
#pragma unroll 1
                for (int db = 0; db < TT_HALF / 32; ++db) {
                    const int d = d0 + 32 * db;
                    uint32_t o[32];
                    tmem_ld32(o_col + 32 * db, o);
                    tmem_wait_ld();
                    if (!part && (a.flags & CSA2_ROPE) && d >= TT_C - 64) {
                        const float* c = cs + (d - (TT_C - 64)) / 2;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float x0 = __uint_as_float(o[2 * j]), x1 = __uint_as_float(o[2 * j + 1]);
                            o[2 * j] = __float_as_uint(x0 * c[j] + x1 * c[32 + j]);
                            o[2 * j + 1] = __float_as_uint(x1 * c[j] - x0 * c[32 + j]);
                        }
                    }
                    const auto v = [&](int i) { return __uint_as_float(o[i]) * fin.x; };
                    if (!valid) continue;
                    if (wide) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v(k + i));
                            store_sector(dst + (d + k) * 4, w, whole);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v(k + 2 * i), v(k + 2 * i + 1));
                            store_sector(dst + (d + k) * 2, w, whole);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
            ++oq;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    if (warp == 1) tmem_dealloc(tmem, 512);
    cluster_sync_all();                // nothing of the peer's is on its way into this CTA
}

struct MergeArgs {
    const float* part_o;
    const float* part_l;
    const float* rope_cs;
    const float* sink;
    int64_t first, groups;        // of the groups that are dealt out, all
    int H, G, gps, T, pieces, share, tiles;
    unsigned flags;
    void* out;
    int out_f32;
    float* lse;
};

// The pieces of one query row, a warp each: outputs and sums add up.
__global__ void __launch_bounds__(256, 4) tree_merge_kernel(const MergeArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, rows = a.G * a.H;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= (a.groups - a.first) * rows) return;
    const int64_t o = i / rows, v = a.first + o, b = v / a.gps;
    const int r = (int)(i - o * rows), g = r / a.H, h = r - g * a.H, node = (int)(v % a.gps) * a.G + g;
    if (node >= a.T) return;
    const int64_t bt = b * a.T + node, g0 = o * a.tiles;
    const int n = (int)((g0 + a.tiles - 1) / a.share - g0 / a.share) + 1;
    if (n == 1) return;                          // (the main kernel has finished the group)
    float acc[16], L = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
    for (int s0 = 0; s0 < n; s0 += 2) {
        float l[2];
        float4 x[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t p = (o * a.pieces + s0 + s) * rows + r;
            l[s] = s0 + s < n ? a.part_l[p] : 0.0f;
            // (a piece without slots has left its output as it was)
            const float4* x0 = reinterpret_cast<const float4*>(a.part_o + p * TT_C) + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[s][j] = s0 + s < n ? __ldcs(x0 + 32 * j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            L += l[s];
            if (l[s] == 0.0f) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[4 * j] += x[s][j].x;
                acc[4 * j + 1] += x[s][j].y;
                acc[4 * j + 2] += x[s][j].z;
                acc[4 * j + 3] += x[s][j].w;
            }
        }
    }
    const float2 fin = finish_row(L, a.sink ? a.sink[h] : -INFINITY);
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] *= fin.x;
    if ((a.flags & CSA2_ROPE) && lane >= 16) {
        const float* cs = a.rope_cs + bt * 64 + 2 * (lane - 16);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float c = cs[j], s = cs[32 + j], x0 = acc[12 + 2 * j], x1 = acc[13 + 2 * j];
            acc[12 + 2 * j] = x0 * c + x1 * s;
            acc[13 + 2 * j] = x1 * c - x0 * s;
        }
    }
    const int64_t row = bt * a.H + h;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t e = row * TT_C + 128 * j + 4 * lane;
        if (a.out_f32)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + e) =
                make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        else
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + e) =
                make_uint2(pack_bf16(acc[4 * j], acc[4 * j + 1]), pack_bf16(acc[4 * j + 2], acc[4 * j + 3]));
    }
    if (a.lse && lane == 0) a.lse[row] = fin.y;
}

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct TtPlan {
    int G, R8, gps, lde, ldw, clusters, rounds, share, tiles, pieces;
    int64_t groups;
    size_t qm, erow, ef, eok, wrow, wmask, rf, df, info, rope, part_l, part_o, total;
};

TtPlan tt_plan(const csa2_ctx* ctx, int B, int T, int H, int k, int window, bool dense) {
    TtPlan p;
    // nodes that share their slots fill the 128 rows together
    p.G = dense ? std::max(1, std::min({TT_G, TT_ROWS / H, T})) : 1;
    p.R8 = (p.G * H + 7) / 8 * 8;
    p.gps = (T + p.G - 1) / p.G;
    p.groups = (int64_t)B * p.gps;
    const int near = window > 0 ? window + (dense ? T : 0) : 0;
    p.lde = (k + 31) / 32 * 32;
    p.ldw = (near + 31) / 32 * 32;
    // The groups go whole to the clusters, in rounds; the last, incomplete round whole as well, or dealt out
    // in even shares of tiles.  Shares cost a second start and output a cluster and the joining of the partial
    // outputs, measured at about six tiles' time.
    const int most = std::max(1, ctx->num_sms / 2);
    p.tiles = std::max(1, (p.lde + near + TT_TILE - 1) / TT_TILE);
    p.clusters = (int)std::min<int64_t>(most, p.groups);
    p.rounds = (int)(p.groups / most);
    const int64_t rest = p.groups - (int64_t)p.rounds * most;
    p.share = p.tiles;
    p.pieces = 1;
    const int64_t even = (rest * p.tiles + most - 1) / most;
    if (rest > 0 && even + 6 < p.tiles) {
        p.share = (int)even;
        p.clusters = p.rounds > 0 ? most : (int)((rest * p.tiles + even - 1) / even);
        p.pieces = (p.tiles + p.share - 2) / p.share + 1;     // of the shares that touch a group
    }
    const size_t eg = dense ? (size_t)B : (size_t)B * T;
    p.qm = up((size_t)p.groups * p.R8 * 1024, 256);
    p.erow = up(p.qm + (size_t)p.groups * p.R8 * 4, 256);
    p.ef = up(p.erow + eg * p.lde * 4, 256);
    p.eok = up(p.ef + eg * p.lde * 4, 256);
    p.wrow = up(p.eok + eg * (p.lde / 32) * 4, 256);
    p.wmask = up(p.wrow + (size_t)p.groups * p.ldw * 4, 256);
    p.rf = up(p.wmask + (size_t)p.groups * (p.ldw / 32) * TT_G * 4, 256);
    p.df = up(p.rf + (size_t)B * window * 4, 256);
    p.info = up(p.df + (size_t)B * T * 4, 256);
    p.rope = up(p.info + (size_t)p.groups * 16, 256);
    p.part_l = up(p.rope + (size_t)B * T * 64 * 4, 256);
    const size_t rows = p.pieces > 1 ? (size_t)rest * p.pieces * p.G * H : 0;
    p.part_o = up(p.part_l + rows * 4, 256);
    p.total = p.part_o + rows * TT_C * 4;
    return p;
}

template <bool FP4, bool DENSE>
csa2_status launch_tt(int clusters, const TtArgs& a, const TtMaps& m, cudaStream_t s) {
    auto kern = tree_tc_kernel<FP4, DENSE>;
    CSA2_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TT_SMEM));
    return launch_pdl(kern, dim3((unsigned)(2 * clusters)), dim3(TT_THREADS), TT_SMEM, s, a, m);
}

}  // namespace

bool tree_tc_applies(csa2_dtype q_dt, csa2_dtype kv_dt, csa2_dtype swa_dt, unsigned flags) {
    return q_dt == CSA2_BF16 && swa_dt == CSA2_BF16 && (kv_dt == CSA2_BF16 || kv_dt == CSA2_FP4_E4M3x16) &&
           (flags & (CSA2_QNORM | CSA2_KVNORM)) == (CSA2_QNORM | CSA2_KVNORM);
}

size_t tree_tc_ws_bytes(const csa2_ctx* ctx, int B, int T, int H, int k, int window, bool dense) {
    return tt_plan(ctx, B, T, H, k, window, dense).total;
}

csa2_status tree_tc_run(csa2_ctx* ctx, const TreeCall& c, void* ws, cudaStream_t s) {
    const bool dense = c.r.n_visible != nullptr, fp4 = c.kv_dt == CSA2_FP4_E4M3x16;
    const TtPlan p = tt_plan(ctx, c.B, c.r.T, c.H, c.r.k, c.r.window, dense);
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    PrepArgs pa = {};
    pa.l.qimg = base;
    pa.l.qm = reinterpret_cast<float*>(base + p.qm);
    pa.l.erow = reinterpret_cast<int32_t*>(base + p.erow);
    pa.l.ef = reinterpret_cast<float*>(base + p.ef);
    pa.l.eok = reinterpret_cast<uint32_t*>(base + p.eok);
    pa.l.wrow = reinterpret_cast<int32_t*>(base + p.wrow);
    pa.l.rf = reinterpret_cast<float*>(base + p.rf);
    pa.l.df = reinterpret_cast<float*>(base + p.df);
    pa.l.drafts = (int64_t)c.B * c.r.T;
    pa.l.wmask = reinterpret_cast<uint32_t*>(base + p.wmask);
    pa.l.info = reinterpret_cast<int4*>(base + p.info);
    pa.l.rope_cs = reinterpret_cast<float*>(base + p.rope);
    pa.l.lde = p.lde;
    pa.l.ldw = p.ldw;
    pa.l.H = c.H;
    pa.l.G = p.G;
    pa.l.R8 = p.R8;
    pa.l.gps = p.gps;
    pa.r = c.r;
    pa.q = reinterpret_cast<const __nv_bfloat16*>(c.q);
    pa.kv = reinterpret_cast<const uint8_t*>(c.kv);
    pa.swa = reinterpret_cast<const uint8_t*>(c.swa);
    pa.draft = reinterpret_cast<const uint8_t*>(c.draft);
    pa.fp4 = fp4;
    pa.ew = p.lde / 32;
    pa.ww = std::max(1, p.ldw / 32);
    pa.rw = (c.r.window + 7) / 8;
    pa.e_warps = (dense ? (int64_t)c.B : (int64_t)c.B * c.r.T) * pa.ew;
    pa.w_warps = p.groups * pa.ww;
    pa.r_warps = (int64_t)c.B * pa.rw;
    pa.d_warps = c.r.window > 0 ? (pa.l.drafts + 7) / 8 : 0;
    pa.q_warps = p.groups * (p.R8 / TT_QROWS);
    pa.rope = c.rope;
    pa.flags = c.flags;
    pa.st = ctx->status;
    TtMaps maps;
    // (a map that no slot refers to still needs an address: the query's)
    const int64_t map_rows[3] = {fp4 || c.r.k == 0 ? 0 : (c.r.table ? c.r.N : c.B * c.r.N), c.r.window > 0 ? c.B * c.r.swa_cap : 0,
                                 c.r.window > 0 ? (int64_t)c.B * c.r.T : 0};
    const void* map_at[3] = {c.kv, c.swa, c.draft};
    for (int i = 0; i < 3; ++i)
        if (!csa2_make_bf16_map(&maps.m[i], map_rows[i] > 0 ? map_at[i] : c.q, std::max<int64_t>(1, map_rows[i]), TT_C, 64, TT_TILE / TT_LOADERS))
            return CSA2_ERR_CUDA;
    const int64_t blocks = (pa.e_warps + pa.w_warps + pa.r_warps + pa.d_warps + pa.q_warps + 7) / 8;
    csa2_status st = launch_pdl(tree_prep_kernel, dim3((unsigned)blocks), dim3(256), 0, s, pa);
    if (st != CSA2_OK) return st;
    TtArgs a = {};
    a.l = pa.l;
    a.r = c.r;
    a.kv = pa.kv;
    a.swa = pa.swa;
    a.draft = pa.draft;
    a.sink = c.sink;
    a.groups = (int)p.groups;
    a.rounds = p.rounds;
    a.clusters = p.clusters;
    a.share = p.share;
    a.tiles = p.tiles;
    a.pieces = p.pieces;
    a.flags = c.flags;
    a.out = c.out;
    a.out_f32 = c.out_dt == CSA2_F32;
    a.lse = c.lse;
    a.part_l = reinterpret_cast<float*>(base + p.part_l);
    a.part_o = reinterpret_cast<float*>(base + p.part_o);
    a.st = ctx->status;
    a.budget = TT_BUDGET;
    if (ctx->stall_next) {
        a.stall = 1;
        // (long enough for every store between the CTAs to land before one of them gives up)
        if (ctx->stall_budget > 0) a.budget = std::max<long long>(ctx->stall_budget, 1 << 17);
        ctx->stall_next = 0;
    }
    if (fp4) st = dense ? launch_tt<true, true>(p.clusters, a, maps, s) : launch_tt<true, false>(p.clusters, a, maps, s);
    else st = dense ? launch_tt<false, true>(p.clusters, a, maps, s) : launch_tt<false, false>(p.clusters, a, maps, s);
    if (st != CSA2_OK) return st;
    if (p.pieces > 1) {
        const int64_t first = (int64_t)p.rounds * p.clusters;
        const MergeArgs m = {a.part_o, a.part_l, a.l.rope_cs, a.sink, first, p.groups, c.H, p.G, p.gps, c.r.T, p.pieces, p.share, p.tiles,
                             c.flags, c.out, a.out_f32, c.lse};
        const int64_t rows = (p.groups - first) * p.G * c.H;
        st = launch_pdl(tree_merge_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, m);
        if (st != CSA2_OK) return st;
    }
    return csa2_launch_status();
}
