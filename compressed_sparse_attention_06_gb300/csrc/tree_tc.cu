// Attention of drafted trees on the tcgen05 tensor cores (DSA-to-CSA/HCA page eqs. (18)-(19), (26),
// (27)): the same RMS-normalised row is key and value for all heads of a node and, in the dense
// form, for all nodes of a tree.
//
// A work item is a group of up to 128 query rows that read the same slots (a node's heads; dense:
// those of up to 8 nodes) and a range of tiles of 128 slots.  Two CTAs (a cluster) share an item,
// each with half of the 512 dims: the fp32 output of 128 rows x 512 dims alone is all of an SM's
// tensor memory, and 64 rows would leave half of every MMA unused (N = 64 costs what N = 128 does).
//   S[128 rows x 128 slots]  = Q^[128 x 256] . X[128 x 256]^T     this CTA's half of the logits
//   O[128 rows x 256 dims]  += P'[128 x 128] . X[128 x 256]       P' read from tensor memory
// The halves of the logits meet through distributed shared memory: each softmax warp scales its
// values by the slot's RMS factor, rounds them to fp16 (2^-12 of a half logit; q^'s own rounding to
// bf16 moves a logit by ten times that), and both CTAs add the same two fp16 numbers.  Both norms
// bound every logit by sqrt(512), so the softmax's offset is a constant (24): p is in (e^-47, 1].
//
// tree_prep_kernel runs first: q^ (normalised, rotated) as the swizzled image of the A operand, the
// RoPE table, and each group's list of row addresses, so that the loaders follow one address only.
//
// Warps (640 threads, one CTA an SM; the first four give most of their registers to the others):
//   0       query images (bulk copies)
//   1       issues the MMAs; owns tensor memory (O: columns 0-255, S / P': two buffers of 128)
//   4-11    softmax, two warps a lane quarter (64 slots each), and the output, a row a thread
//   12-19   loaders, 16 rows of the tile each: rows through registers into the swizzled tile (two
//           tiles deep), their squares summed on the way; FP4 rows are dequantised exactly
// Every wait is bounded; the CTAs meet at the cluster's barrier before either one exits.
#include <algorithm>

#include "fp4_tile.cuh"
#include "sm100_ptx.cuh"
#include "tree_tc.cuh"

namespace {

using namespace sm100;

constexpr unsigned FULL = 0xffffffffu;
constexpr int TT_C = 512, TT_HALF = 256;
constexpr int TT_ROWS = 128, TT_TILE = 128;
constexpr int TT_G = 8;                          // nodes of a group at most
constexpr int TT_THREADS = 640;
constexpr int TT_REGS_FEW = 64, TT_REGS_MANY = 104;      // registers of the first warpgroup and the other four
static_assert(TT_REGS_FEW + 4 * TT_REGS_MANY <= 5 * 96, "what the launch gives: 96 registers a thread");
constexpr int TT_CHUNK = TT_TILE * 128;          // 16 KB: 128 rows x 64 dims
constexpr int TT_TILE_BYTES = 4 * TT_CHUNK;
constexpr float TT_SHIFT = 24.0f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr long long TT_BUDGET = 1ll << 31;

constexpr int OFF_Q = 0;
constexpr int OFF_K = 65536;
constexpr int OFF_X = OFF_K + 2 * TT_TILE_BYTES;         // the peer's logits: [2 halves][8 units][128 rows] x 16 B
constexpr int OFF_SS = OFF_X + 32768;                    // [2][128] the peer's squares, then the RMS factors
constexpr int OFF_L = OFF_SS + 1024;                     // [2][128] sums of exponentials
constexpr int OFF_MASK = OFF_L + 1024;                   // [2][TT_G][8] x 16 bits
constexpr int OFF_BAR = OFF_MASK + 2 * TT_G * 16;
constexpr int N_BAR = 18 + 16 + 8 + 8;
constexpr int OFF_TMEM = OFF_BAR + N_BAR * 8;
constexpr int TT_SMEM = OFF_TMEM + 16;
static_assert(TT_SMEM <= 227 * 1024, "shared memory");

struct TtArgs {
    const uint8_t* qimg;          // [groups][2 halves][4 chunks][R8 rows x 128 B]
    const uint64_t* list;         // [groups][list_ld] addresses of the listed slots' rows (0: none)
    const uint16_t* mask;         // [groups][list_ld / 16][TT_G] who attends to them (dense)
    const int4* info;             // [groups] entries (a multiple of 16), slots
    const float* rope_cs;         // [B*T, 64] cos, sin of the 32 angles
    const uint8_t* kv;
    TreeRows r;
    const float* sink;
    int H, G, R8, gps;            // heads, nodes of a group, image rows, groups of a sequence
    int64_t list_ld, groups, items;
    int n_split, tps;
    unsigned flags;
    void* out;
    int out_f32;
    float* lse;
    float* part_o;                // [groups * n_split][G*H rows][512] (n_split > 1)
    float* part_l;                // [groups * n_split][G*H rows]
    unsigned* st;
    long long budget;
    int stall;
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
// An arrival at a barrier of the peer's that says "read": the values read are in registers, and
// nothing this thread wrote is behind it, so it carries no fence (a release at the cluster's scope
// waits for every access of the thread, microseconds a tile).
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Stores into the peer's shared memory that count their bytes at one of its barriers.
__device__ __forceinline__ void peer_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void peer_st(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

struct TtItem {
    int64_t v, b, bt0;            // group, sequence, first node
    int split, gv, kq16, slots;   // nodes, entry slots, all slots
    int t0, nt;                   // tiles t0 .. t0 + nt - 1
    int64_t prow;                 // its first row among the partials
};

__device__ __forceinline__ TtItem tt_item(const TtArgs& a, int64_t item) {
    TtItem r;
    r.v = item / a.n_split;
    r.split = (int)(item % a.n_split);
    r.b = r.v / a.gps;
    const int n0 = (int)(r.v % a.gps) * a.G;
    r.bt0 = r.b * a.r.T + n0;
    r.gv = min(a.G, a.r.T - n0);
    const int4 i = a.info[r.v];
    r.kq16 = i.x;
    r.slots = i.y;
    const int tiles = (i.y + TT_TILE - 1) / TT_TILE;
    r.t0 = r.split * a.tps;
    r.nt = max(0, min(tiles, r.t0 + a.tps) - r.t0);
    r.prow = item * (int64_t)(a.G * a.H);
    return r;
}

// ---------------------------------------------------------------- before the main kernel
struct PrepArgs {
    TreeRows r;
    const __nv_bfloat16* q;
    const uint8_t* kv;
    const uint8_t* swa;
    const uint8_t* draft;
    int64_t kv_row;               // bytes of a cache row
    int H, G, R8, gps;
    int64_t list_ld;
    RopeTable rope;
    unsigned flags;
    uint8_t* qimg;
    uint64_t* list;
    uint16_t* mask;
    int4* info;
    float* rope_cs;
    unsigned* st;
};

// Block (group, y): y < R8 / 8 normalises and rotates 8 query rows, a warp each; the last one
// lists the group's slots.
__global__ void __launch_bounds__(256) tree_prep_kernel(const PrepArgs a) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t v = blockIdx.x, b = v / a.gps;
    const int n0 = (int)(v % a.gps) * a.G, gv = min(a.G, a.r.T - n0);
    const int64_t bt0 = b * a.r.T + n0;
    if ((int)blockIdx.y < a.R8 / 8) {
        const int row = 8 * blockIdx.y + warp, g = row / a.H, h = row - g * a.H;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
        if (g < gv) {
            const int64_t t = a.r.pos[bt0 + g];
            const uint4* p = reinterpret_cast<const uint4*>(a.q + ((bt0 + g) * a.H + h) * (int64_t)TT_C + 16 * lane);
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 u = p[i];
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                    x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
            const float r = 1.0f / sqrtf(warp_sum(ss) / (float)TT_C + 1e-6f);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= r;
            if (a.flags & CSA2_ROPE) {
                // lane j has angle j; lanes 28 .. 31 rotate the pairs of dims 448 .. 511
                float c, s;
                rope_cos_sin(a.rope, t, lane, c, s);
                if (h == 0) {
                    a.rope_cs[(bt0 + g) * 64 + lane] = c;
                    a.rope_cs[(bt0 + g) * 64 + 32 + lane] = s;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = (8 * (lane - 28) + i) & 31;
                    const float cj = __shfl_sync(FULL, c, j), sj = __shfl_sync(FULL, s, j);
                    if (lane >= 28) {
                        const float x0 = x[2 * i], x1 = x[2 * i + 1];
                        x[2 * i] = x0 * cj - x1 * sj;
                        x[2 * i + 1] = x1 * cj + x0 * sj;
                    }
                }
            }
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        uint8_t* img = a.qimg + v * (int64_t)a.R8 * 1024 + (lane >> 2) * (int64_t)a.R8 * 128;      // chunk of 64 dims
        const uint32_t u = 2 * (lane & 3);
        *reinterpret_cast<uint4*>(img + sw128_offset(row, u)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(img + sw128_offset(row, u + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    uint64_t* list = a.list + v * a.list_ld;
    const auto window_addr = [&](int kind, int64_t row) {
        return (uint64_t)(uintptr_t)((kind == TREE_RING ? a.swa : a.draft) + row * (int64_t)(TT_C * 2));
    };
    if (!a.r.n_visible) {                        // one node: its entries, then its window
        const TreeNode n = tree_node(a.r, bt0);
        const int kq16 = (n.kq + 15) / 16 * 16;
        for (int s = threadIdx.x; s < kq16 + n.nw; s += blockDim.x) {
            uint64_t p = 0;
            if (s < kq16) {
                const int64_t row = s < n.kq ? tree_entry_row(a.r, b, a.r.idx[bt0 * a.r.k + s], a.st, true) : -1;
                if (row >= 0) p = (uint64_t)(uintptr_t)(a.kv + row * a.kv_row);
            } else {
                int kind;
                const int64_t row = tree_window_row(a.r, n, n.t - n.nw + 1 + (s - kq16), kind, a.st, true);
                if (row >= 0) p = window_addr(kind, row);
            }
            list[s] = p;
        }
        if (threadIdx.x == 0) a.info[v] = make_int4(kq16, kq16 + n.nw, 0, 0);
        return;
    }
    // dense: the entries any node sees need no list; then the ring's rows of any node's window, then
    // the drafts up to the group's last node, with the nodes that attend to each
    __shared__ int64_t t[TT_G];
    __shared__ int nv[TT_G];
    if (threadIdx.x < TT_G) {
        const int g = threadIdx.x;
        t[g] = g < gv ? a.r.pos[bt0 + g] : -1;
        nv[g] = t[g] >= 0 && a.r.k > 0 ? (int)max((int64_t)0, min((int64_t)a.r.k, a.r.n_visible[bt0 + g])) : 0;
    }
    __syncthreads();
    const int64_t len = a.r.ctx_len[b], W = a.r.window;
    int kq = 0;
    int64_t tmin = INT64_MAX;
    for (int g = 0; g < gv; ++g) {
        kq = max(kq, nv[g]);
        if (t[g] >= 0) tmin = min(tmin, t[g]);
    }
    const int kq16 = (kq + 15) / 16 * 16;
    const bool any = W > 0 && tmin != INT64_MAX;
    const int64_t p0 = max((int64_t)0, max(len - W + 1, any ? tmin - W + 1 : 0));
    const int nring = any ? (int)max((int64_t)0, len - p0) : 0, nw = any ? nring + n0 + gv : 0;
    uint16_t* mask = a.mask + v * (a.list_ld / 16) * TT_G;
    for (int s0 = 0; s0 < nw; s0 += blockDim.x) {
        const int s = s0 + threadIdx.x, j = s - nring;
        int64_t p = INT64_MIN, row = 0;          // position of the slot
        bool real = false;
        if (s < nring) {
            p = p0 + s;
            row = b * a.r.swa_cap + ((p - a.r.swa_pos0) % a.r.swa_cap + a.r.swa_cap) % a.r.swa_cap;
            real = true;
        } else if (s < nw) {
            p = a.r.pos[b * a.r.T + j];
            row = b * a.r.T + j;
            real = p >= len && p - len < a.r.T;
        }
        bool wanted = false;
        for (int g = 0; g < gv; ++g) {
            bool on = real && t[g] >= 0 && p <= t[g] && p > t[g] - W;
            if (on && s >= nring) on = a.r.path[(bt0 + g) * a.r.T + (p - len)] == j;
            const uint32_t bits = __ballot_sync(FULL, on);
            if ((lane & 15) == 0 && s < nw) mask[(s / 16) * TT_G + g] = (uint16_t)(bits >> (lane & 16));
            wanted |= on;
        }
        if (s < nw) list[s] = wanted ? window_addr(s < nring ? TREE_RING : TREE_DRAFT, row) : 0;
    }
    if (threadIdx.x == 0) a.info[v] = make_int4(kq16, kq16 + nw, 0, 0);
}

// ---------------------------------------------------------------- the main kernel

// 16 bytes of 32 E2M1 codes (value 2k in the low nibble of byte k) with their two scales, as bf16: unit u
// of 8 values in w[4 u .. 4 u + 3].  Exact (a code has 2 significant bits, a scale 4).
__device__ __forceinline__ void fp4_32(uint4 codes, uint32_t scales, uint32_t (&w)[16], float& ss) {
    const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float s = e4m3_to_f32((scales >> (8 * (u >> 1))) & 0xFFu);
        float v[8];
        e2m1x8_to_f32(cw[u], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] *= s;
            ss = fmaf(v[i], v[i], ss);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * u + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
}

template <bool FP4, bool DENSE>
__global__ void __launch_bounds__(TT_THREADS, 1) __cluster_dims__(2, 1, 1) tree_tc_kernel(const TtArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sQ = smem + OFF_Q;
    uint8_t* sK = smem + OFF_K;
    uint8_t* sX = smem + OFF_X;
    float* sSS = reinterpret_cast<float*>(smem + OFF_SS);
    float* sL = reinterpret_cast<float*>(smem + OFF_L);
    uint16_t* sMask = reinterpret_cast<uint16_t*>(smem + OFF_MASK);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* qfull = bars + 0;
    uint64_t* qempty = bars + 1;
    uint64_t* kfull = bars + 2;        // [2] a tile's rows are in shared memory
    uint64_t* kempty = bars + 4;       // [2] its products are done
    uint64_t* rfull = bars + 6;        // [2] its RMS factors and masks are there
    uint64_t* sfull = bars + 8;        // [2] its half logits
    uint64_t* pfull = bars + 10;       // [2] its P'
    uint64_t* ofull = bars + 12;
    uint64_t* oempty = bars + 13;
    uint64_t* lred = bars + 14;
    uint64_t* xdone = bars + 16;       // [2] the peer's softmax warps are done with a tile's factors
    uint64_t* ssfull = bars + 18;      // [2][8] the peer's squares of a loader warp's rows
    uint64_t* xfull = bars + 34;       // [8] the peer's logits of a softmax warp
    uint64_t* xempty = bars + 42;      // [8] the peer has read this warp's
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        if (smem_u32(smem) & 1023u) csa2_flag(a.st, CSA2_DEVBIT_TIMEOUT);
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], 8);
            mbar_init(&kempty[i], 1);
            mbar_init(&rfull[i], 8);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 8);
            mbar_init(&xdone[i], 8);
        }
        mbar_init(ofull, 1);
        mbar_init(oempty, 8);
        mbar_init(lred, 8);
        for (int i = 0; i < 16; ++i) mbar_init(&ssfull[i], 1);
        for (int i = 0; i < 8; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 1);
        }
        fence_mbar_init();
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

    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TT_REGS_FEW));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TT_REGS_MANY));
    if (warp < 4) {
        // ============================ query images ============================
        if (warp == 0 && lane == 0) {
            int qi = 0, issued = -1;
            for (int64_t item = first; item < a.items && !a.stall; item += step) {
                const TtItem it = tt_item(a, item);
                if (it.nt == 0) continue;
                if (qi > 0 && !mbar_wait(qempty, (qi - 1) & 1, a.budget, a.st)) break;
                const uint32_t bytes = (uint32_t)a.R8 * 128u;
                mbar_arrive_expect_tx(qfull, 4 * bytes);
                const uint8_t* src = a.qimg + (it.v * 2 + rank) * 4 * (int64_t)bytes;
                for (int c = 0; c < 4; ++c) bulk_g2s(sQ + c * TT_CHUNK, src + c * (int64_t)bytes, bytes, qfull);
                issued = qi++;
            }
            if (issued >= 0) mbar_wait(qfull, issued & 1, a.budget, a.st);
        }
        // ============================ MMA issuer ============================
        if (warp == 1 && lane == 0) {
            constexpr uint32_t IDESC_QK = idesc_f16(TT_ROWS, TT_TILE, true);
            constexpr uint32_t IDESC_PV = idesc_f16_major(TT_ROWS, TT_HALF, true, false, true);
            const uint32_t q_base = smem_u32(sQ), k_base = smem_u32(sK);
            int g = 0, qi = 0;
            bool ok = true;
            uint64_t* last = nullptr;
            uint32_t last_par = 0;
            // half logits of tile g (dims of this CTA)
            const auto qk = [&](int t) {
                if (!mbar_wait(&kfull[t & 1], (t >> 1) & 1, a.budget, a.st)) return false;
                tc_fence_after();
                const uint32_t kb = k_base + (t & 1) * TT_TILE_BYTES;
#pragma unroll
                for (int kk = 0; kk < 16; ++kk) {
                    const uint32_t o = (uint32_t)(kk >> 2) * TT_CHUNK + (uint32_t)(kk & 3) * 32u;
                    mma_ss(tmem + 256 + 128 * (t & 1), sdesc_sw128(q_base + o), sdesc_sw128(kb + o), IDESC_QK, kk != 0);
                }
                mma_commit(&sfull[t & 1]);
                last = &sfull[t & 1];
                last_par = (t >> 1) & 1;
                return true;
            };
            for (int64_t item = first; item < a.items && ok; item += step) {
                const TtItem it = tt_item(a, item);
                if (it.nt == 0) continue;
                ok = mbar_wait(qfull, qi & 1, a.budget, a.st);
                if (!ok) break;
                for (int tt = 0; tt < it.nt; ++tt, ++g) {
                    if (tt == 0) ok = qk(g);
                    if (ok && tt + 1 < it.nt) ok = qk(g + 1);
                    if (!ok) break;
                    if (tt + 1 >= it.nt) mma_commit(qempty);
                    if (!mbar_wait(&pfull[g & 1], (g >> 1) & 1, a.budget, a.st) ||
                        (tt == 0 && qi > 0 && !mbar_wait(oempty, (qi - 1) & 1, a.budget, a.st))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t kb = k_base + (g & 1) * TT_TILE_BYTES, p = tmem + 256 + 128 * (g & 1);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts(tmem, p + (ks >> 2) * 64 + (ks & 3) * 8, sdesc_sw128_mn(kb + ks * 2048, TT_CHUNK, 1024), IDESC_PV,
                               tt > 0 || ks > 0);
                    mma_commit(&kempty[g & 1]);
                    last = &kempty[g & 1];
                    last_par = (g >> 1) & 1;
                    if (tt == it.nt - 1) {
                        mma_commit(ofull);
                        last = ofull;
                        last_par = qi & 1;
                    }
                }
                if (ok) ++qi;
            }
            // the MMAs must be complete before tensor memory is released
            if (last) mbar_wait(last, last_par, a.budget, a.st);
        }
    } else if (warp < 12) {
        // ============================ softmax + output ============================
        const int quad = warp & 3, hh = (warp - 4) >> 2, w = 4 * hh + quad;
        const int r = quad * 32 + lane;                       // query row
        const bool live = quad * 32 < a.G * a.H;              // a warp without query rows only keeps step
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const float c1 = LOG2E / sqrtf((float)TT_C);
        const int g_row = min(r / a.H, a.G - 1);
        uint8_t* mine = sX + (hh * 8 * TT_ROWS + r) * 16;
        const uint32_t theirs = peer_addr(mine, peer);
        const uint32_t their_full = peer_addr(&xfull[w], peer), their_empty = peer_addr(&xempty[w], peer);
        const uint32_t their_done = peer_addr(xdone, peer);
        int g = 0, qi = 0;
        bool ok = true;
        for (int64_t item = first; item < a.items && ok; item += step) {
            const TtItem it = tt_item(a, item);
            const int rows = it.gv * a.H, hq = r / a.H;
            const int64_t bt = it.bt0 + hq;
            const int h = r - hq * a.H;
            if (it.nt == 0) {
                if (r < rows && rank == 0 && a.n_split > 1) {
                    if (hh == 0) a.part_l[it.prow + r] = 0.0f;
                } else if (r < rows && a.n_split == 1) {
                    const int64_t o = (bt * a.H + h) * (int64_t)TT_C + TT_HALF * rank + 128 * hh;
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) + o * (a.out_f32 ? 4 : 2));
                    for (int i = 0; i < (a.out_f32 ? 32 : 16); ++i) d[i] = z;
                    if (rank == 0 && hh == 0 && a.lse) a.lse[bt * a.H + h] = a.sink ? a.sink[h] : -INFINITY;
                }
                continue;
            }
            float lsum = 0.0f;
            for (int tt = 0; tt < it.nt; ++tt, ++g) {
                bool wt = mbar_wait(&sfull[g & 1], (g >> 1) & 1, a.budget, a.st) &&
                          mbar_wait(&rfull[g & 1], (g >> 1) & 1, a.budget, a.st) &&
                          (g == 0 || !live || mbar_wait(&xempty[w], (g - 1) & 1, a.budget, a.st));
                if (!__all_sync(FULL, wt)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float4* rinv = reinterpret_cast<const float4*>(sSS + (g & 1) * TT_TILE + 64 * hh);
                const uint32_t s_col = lanes + 256 + 128 * (g & 1) + 64 * hh;
                uint32_t y[32];                               // this CTA's half logits (log2), fp16 pairs
                if (live) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t sv[16];
                        tmem_ld16(s_col + 16 * i, sv);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f = rinv[4 * i + j];
                            y[8 * i + 2 * j] = pack_f16(__uint_as_float(sv[4 * j]) * (f.x * c1), __uint_as_float(sv[4 * j + 1]) * (f.y * c1));
                            y[8 * i + 2 * j + 1] =
                                pack_f16(__uint_as_float(sv[4 * j + 2]) * (f.z * c1), __uint_as_float(sv[4 * j + 3]) * (f.w * c1));
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        peer_st4(theirs + u * TT_ROWS * 16, y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3], their_full);
                }
                if (live) {
                    // (a warp without rows must not: it could fall two phases behind its peer)
                    if (lane == 0) mbar_arrive_expect_tx(&xfull[w], 32 * 8 * 16);
                    wt = mbar_wait(&xfull[w], g & 1, a.budget, a.st);
                }
                if (!__all_sync(FULL, wt)) {
                    ok = false;
                    break;
                }
                if (live) {
                    uint32_t m[2] = {FULL, FULL};             // the slots this row attends to
                    {
                        const uint2 mm = *reinterpret_cast<const uint2*>(sMask + ((g & 1) * TT_G + g_row) * 8 + 4 * hh);
                        m[0] = mm.x;
                        m[1] = mm.y;
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {             // 32 slots at a time
                        uint32_t pk[16];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint4 o = *reinterpret_cast<const uint4*>(mine + (4 * q + u) * TT_ROWS * 16);
                            const uint32_t ov[4] = {o.x, o.y, o.z, o.w};
                            const float4 f0 = rinv[2 * (4 * q + u)], f1 = rinv[2 * (4 * q + u) + 1];
                            const float fv[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                            const uint32_t mb = m[q] >> (8 * u);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 s0 = unpack_f16(y[16 * q + 4 * u + j]), s1 = unpack_f16(ov[j]);
                                float p0 = ex2(s0.x + s1.x - TT_SHIFT * LOG2E), p1 = ex2(s0.y + s1.y - TT_SHIFT * LOG2E);
                                p0 = (mb >> (2 * j)) & 1u ? p0 : 0.0f;
                                p1 = (mb >> (2 * j + 1)) & 1u ? p1 : 0.0f;
                                lsum += p0 + p1;
                                // (a masked slot's factor may be NaN: its product must not be formed)
                                pk[4 * u + j] = pack_bf16(p0 == 0.0f ? 0.0f : p0 * fv[2 * j], p1 == 0.0f ? 0.0f : p1 * fv[2 * j + 1]);
                            }
                        }
                        tmem_st16(s_col + 16 * q, pk);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&pfull[g & 1]);
                    if (live) peer_arrive(their_empty);
                    peer_arrive(their_done + 8 * (g & 1));
                }
            }
            if (!ok) break;
            // sums of the two halves of the slots; the last item's readers are done with sL
            bool wt = qi == 0 || mbar_wait(oempty, (qi - 1) & 1, a.budget, a.st);
            if (wt) sL[hh * TT_ROWS + r] = lsum;
            __syncwarp();
            if (lane == 0) mbar_arrive(lred);
            wt = wt && mbar_wait(lred, qi & 1, a.budget, a.st) && mbar_wait(ofull, qi & 1, a.budget, a.st);
            if (!__all_sync(FULL, wt)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (live) {
                const float L = sL[r] + sL[TT_ROWS + r];
                float sc = 1.0f;
                if (a.n_split == 1) {
                    const float zs = a.sink && r < rows ? a.sink[h] : -INFINITY;
                    float ls = zs;
                    sc = 0.0f;
                    if (L != 0.0f) {                          // (a NaN shows)
                        const float M = fmaxf(TT_SHIFT, zs), e = expf(TT_SHIFT - M);
                        const float den = L * e + (zs == -INFINITY ? 0.0f : expf(zs - M));
                        sc = e / den;
                        ls = M + logf(den);
                    }
                    if (rank == 0 && hh == 0 && r < rows && a.lse) a.lse[bt * a.H + h] = ls;
                } else if (rank == 0 && hh == 0 && r < rows) {
                    a.part_l[it.prow + r] = L;
                }
                const int d0 = TT_HALF * rank + 128 * hh;
                const bool rot = a.n_split == 1 && (a.flags & CSA2_ROPE) && d0 == 384;
                const float* cs = a.rope_cs + (r < rows ? bt : it.bt0) * 64;
#pragma unroll 1
                for (int db = 0; db < 4; ++db) {
                    uint32_t o[32];
                    tmem_ld32(lanes + 128 * hh + 32 * db, o);
                    tmem_wait_ld();
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * sc;
                    if (rot && db >= 2) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float c = cs[16 * (db - 2) + j], s = cs[32 + 16 * (db - 2) + j], x0 = v[2 * j], x1 = v[2 * j + 1];
                            v[2 * j] = x0 * c + x1 * s;
                            v[2 * j + 1] = x1 * c - x0 * s;
                        }
                    }
                    if (r < rows && (a.n_split > 1 || a.out_f32)) {
                        float* d = (a.n_split > 1 ? a.part_o + (it.prow + r) * (int64_t)TT_C
                                                  : reinterpret_cast<float*>(a.out) + (bt * a.H + h) * (int64_t)TT_C) + d0 + 32 * db;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4*>(d)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    } else if (r < rows) {
                        uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                                            (bt * a.H + h) * (int64_t)TT_C + d0 + 32 * db);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            d[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                              pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
            ++qi;
        }
    } else {
        // ============================ loaders ============================
        const int lw = warp - 12;                             // rows 16 lw .. 16 lw + 15 of the tile
        const uint32_t their_ss = peer_addr(sSS, peer), their_bar = peer_addr(ssfull, peer);
        int64_t item = first;
        TtItem it;
        int tt = 0;
        int nv = 0;                                           // lane g: entries node g sees (dense)
        // the next tile with rows, or item >= items
        const auto settle = [&]() {
            while (item < a.items) {
                if (tt == 0) {
                    it = tt_item(a, item);
                    if (DENSE && lane < it.gv) {
                        const bool used = a.r.pos[it.bt0 + lane] >= 0 && a.r.k > 0;
                        nv = used ? (int)max((int64_t)0, min((int64_t)a.r.k, a.r.n_visible[it.bt0 + lane])) : 0;
                    }
                }
                if (tt < it.nt) return;
                item += step;
                tt = 0;
            }
        };
        // The loads that the next tile's addresses and masks need are issued a tile ahead (look_up) and
        // used when its rows are fetched (resolve): lane j < 16 has row j, lanes 16 .. 31 repeat them.
        uint64_t ptr = 0;             // listed slot's address, or the page of a dense entry
        uint32_t bits = 0;            // listed dense slots: lane g has node g's mask
        int slot = 0;
        bool is_kv = false;
        const auto look_up = [&]() {
            const int s0 = (it.t0 + tt) * TT_TILE + 16 * lw;
            slot = s0 + (lane & 15);
            is_kv = s0 < it.kq16;
            ptr = 0;
            bits = 0;
            if (item >= a.items) return;
            if (DENSE && is_kv) {
                if (a.r.table) {
                    const int p = slot / a.r.page;
                    ptr = p < a.r.max_pages ? (uint64_t)(int64_t)a.r.table[it.b * a.r.max_pages + p] : ~0ull;
                }
                return;
            }
            const int64_t base = DENSE ? it.kq16 : 0;
            if (slot < it.slots) ptr = a.list[it.v * a.list_ld + (slot - base)];
            if (DENSE && s0 < it.slots && lane < it.gv)
                bits = a.mask[(it.v * (a.list_ld / 16) + (s0 - base) / 16) * TT_G + lane];
        };
        const auto resolve = [&](int nv_g, int gv) {
            if (DENSE && is_kv) {
                uint32_t mine = 0;
                bool seen = false;
                for (int g = 0; g < gv; ++g) {
                    const bool on = slot < __shfl_sync(FULL, nv_g, g);
                    const uint32_t m = __ballot_sync(FULL, on) & 0xFFFFu;
                    if (lane == g) mine = m;
                    seen |= on;
                }
                int64_t row = slot;                              // within the sequence, or the pool
                int64_t base = it.b * a.r.N;
                if (a.r.table) {
                    const int64_t t = (int64_t)ptr;
                    row = t >= 0 ? t * a.r.page + slot % a.r.page : -1;
                    base = 0;
                }
                const bool there = seen && row >= 0 && row < a.r.N;
                if (seen && !there) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
                ptr = there ? (uint64_t)(uintptr_t)(a.kv + (base + row) * (FP4 ? fp4_row_bytes(TT_C) : (int64_t)(TT_C * 2))) : 0;
                bits = mine & __ballot_sync(FULL, there);
            } else if (!DENSE) {
                bits = __ballot_sync(FULL, ptr != 0) & 0xFFFFu;
            }
        };
        settle();
        look_up();
        int g = 0;
        bool ok = true;
        float ss_prev = 0.0f;                                 // lane j < 16: this CTA's squares of row j, tile g - 1
        // RMS factors of tile t from both halves' squares
        const auto factors = [&](int t) {
            const bool wt = mbar_wait(&ssfull[8 * (t & 1) + lw], (t >> 1) & 1, a.budget, a.st);
            if (!__all_sync(FULL, wt)) return false;
            if (lane < 16) {
                float* p = sSS + (t & 1) * TT_TILE + 16 * lw + lane;
                const float s = ss_prev + *p;
                // a row with an infinity or a NaN makes the rows that attend to it NaN
                *p = s < INFINITY ? 1.0f / sqrtf(s / (float)TT_C + 1e-6f) : __int_as_float(0x7FC00000);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&rfull[t & 1]);
            return true;
        };
        while (item < a.items && ok) {
            // this tile's rows on their way
            uint4 d[16];
            uint32_t sc[4];
            resolve(nv, it.gv);
            const bool fp4_rows = FP4 && is_kv;
            const uint64_t my_ptr = ptr;
            const uint32_t my_bits = bits;
            if (fp4_rows) {
                // 8 lanes a row, 4 rows an instruction: 16 code bytes and 2 scales a lane
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t p = __shfl_sync(FULL, my_ptr, 4 * i + (lane >> 3));
                    d[i] = make_uint4(0u, 0u, 0u, 0u);
                    sc[i] = 0u;
                    if (p) {
                        const uint8_t* src = reinterpret_cast<const uint8_t*>((uintptr_t)p);
                        d[i] = *reinterpret_cast<const uint4*>(src + 128 * rank + 16 * (lane & 7));
                        sc[i] = *reinterpret_cast<const uint16_t*>(src + 256 + 16 * rank + 2 * (lane & 7));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t p = __shfl_sync(FULL, my_ptr, i);
                    d[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (p) d[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>((uintptr_t)p) + 512 * rank + 16 * lane);
                }
            }
            const int gv = it.gv;
            ++tt;
            settle();
            look_up();                                        // the next tile's addresses
            if (g > 0) ok = factors(g - 1);
            if (ok && g >= 2) {
                // (the peer's softmax reads the factors that this tile's squares will replace)
                const bool wt = mbar_wait(&kempty[g & 1], ((g - 2) >> 1) & 1, a.budget, a.st) &&
                                mbar_wait(&xdone[g & 1], ((g - 2) >> 1) & 1, a.budget, a.st);
                ok = __all_sync(FULL, wt);
            }
            if (!ok) break;
            uint8_t* tile = sK + (g & 1) * TT_TILE_BYTES;
            if (fp4_rows) {
                const int piece = lane & 7, c = piece >> 1;
                ss_prev = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t wv[16];
                    float q = 0.0f;
                    fp4_32(d[i], sc[i], wv, q);
                    // the squares of the row's 8 lanes; a scale of NaN empties the row's values
                    q += __shfl_xor_sync(FULL, q, 1);
                    q += __shfl_xor_sync(FULL, q, 2);
                    q += __shfl_xor_sync(FULL, q, 4);
                    if (!(q < INFINITY)) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) wv[k] = 0u;
                    }
                    // lane j < 16 takes row j = 4 i + j % 4 from the first of its 8 lanes
                    const float row_q = __shfl_sync(FULL, q, 8 * (lane & 3));
                    if ((lane >> 2) == i) ss_prev = row_q;
                    const uint32_t row = 16 * lw + 4 * i + (lane >> 3);
                    uint8_t* base = tile + c * TT_CHUNK;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // units in an order that differs between the lanes of a row: no bank twice
                        const int u = (k + c) & 3;
                        uint4 val = make_uint4(wv[0], wv[1], wv[2], wv[3]);
                        if (u == 1) val = make_uint4(wv[4], wv[5], wv[6], wv[7]);
                        if (u == 2) val = make_uint4(wv[8], wv[9], wv[10], wv[11]);
                        if (u == 3) val = make_uint4(wv[12], wv[13], wv[14], wv[15]);
                        *reinterpret_cast<uint4*>(base + sw128_offset(row, (uint32_t)(4 * (piece & 1) + u))) = val;
                    }
                }
            } else {
                // sums over the 32 lanes of 16 rows: of two rows' parts a lane keeps one and sends the
                // other, four times over, and ends with half of row lane / 2's sum
                const auto sq = [&](int i) {
                    const uint32_t wv[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
                    float q = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float lo = __uint_as_float(wv[k] << 16), hi = __uint_as_float(wv[k] & 0xFFFF0000u);
                        q = fmaf(lo, lo, q);
                        q = fmaf(hi, hi, q);
                    }
                    return q;
                };
                const auto join = [&](float x, float y, int o) {
                    const bool upper = lane & o;
                    return (upper ? y : x) + __shfl_xor_sync(FULL, upper ? x : y, o);
                };
                const auto four = [&](int i) {
                    return join(join(sq(i), sq(i + 8), 16), join(sq(i + 4), sq(i + 12), 16), 8);
                };
                const float half = join(join(four(0), four(2), 4), join(four(1), four(3), 4), 2);
                const float sum = half + __shfl_xor_sync(FULL, half, 1);
                const uint32_t bad = __ballot_sync(FULL, !(sum < INFINITY));      // bit 2 i: row i
                ss_prev = __shfl_sync(FULL, sum, (2 * lane) & 31);
                uint8_t* base = tile + (lane >> 3) * TT_CHUNK;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if ((bad >> (2 * i)) & 1u) d[i] = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(base + sw128_offset((uint32_t)(16 * lw + i), (uint32_t)(lane & 7))) = d[i];
                }
            }
            if (lane < (DENSE ? gv : 1)) sMask[((g & 1) * TT_G + lane) * 8 + lw] = (uint16_t)my_bits;
            if (lane < 16)
                peer_st(their_ss + ((g & 1) * TT_TILE + 16 * lw + lane) * 4, ss_prev, their_bar + (8 * (g & 1) + lw) * 8);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&kfull[g & 1]);
                mbar_arrive_expect_tx(&ssfull[8 * (g & 1) + lw], 16 * 4);
            }
            ++g;
        }
        if (ok && g > 0) factors(g - 1);
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
    int64_t groups;
    int H, G, gps, T, n_split;
    unsigned flags;
    void* out;
    int out_f32;
    float* lse;
};

// The splits of one query row, a warp each: all used the same offset, so outputs and sums add up.
__global__ void __launch_bounds__(256) tree_merge_kernel(const MergeArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, rows = a.G * a.H;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= a.groups * rows) return;
    const int64_t v = i / rows, b = v / a.gps;
    const int r = (int)(i - v * rows), g = r / a.H, h = r - g * a.H, node = (int)(v % a.gps) * a.G + g;
    if (node >= a.T) return;
    const int64_t bt = b * a.T + node;
    float acc[16], L = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
    for (int s0 = 0; s0 < a.n_split; s0 += 4) {
        float l[4];
        float4 x[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int64_t p = (v * a.n_split + s0 + s) * rows + r;
            l[s] = s0 + s < a.n_split ? a.part_l[p] : 0.0f;
            // (a split without slots has no output)
            const float4* o = reinterpret_cast<const float4*>(a.part_o + p * TT_C) + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[s][j] = l[s] != 0.0f ? __ldcs(o + 32 * j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            L += l[s];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[4 * j] += x[s][j].x;
                acc[4 * j + 1] += x[s][j].y;
                acc[4 * j + 2] += x[s][j].z;
                acc[4 * j + 3] += x[s][j].w;
            }
        }
    }
    const float zs = a.sink ? a.sink[h] : -INFINITY;
    float sc = 0.0f, ls = zs;
    if (L != 0.0f) {
        const float M = fmaxf(TT_SHIFT, zs), e = expf(TT_SHIFT - M);
        const float den = L * e + (zs == -INFINITY ? 0.0f : expf(zs - M));
        sc = e / den;
        ls = M + logf(den);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] *= sc;
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
        const int64_t o = row * TT_C + 128 * j + 4 * lane;
        if (a.out_f32)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + o) =
                make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        else
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + o) =
                make_uint2(pack_bf16(acc[4 * j], acc[4 * j + 1]), pack_bf16(acc[4 * j + 2], acc[4 * j + 3]));
    }
    if (a.lse && lane == 0) a.lse[row] = ls;
}

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct TtPlan {
    int G, R8, gps, n_split, tps;
    int64_t groups, list_ld;
    size_t qimg, list, mask, info, rope, part_l, part_o, total;
};

TtPlan tt_plan(const csa2_ctx* ctx, int B, int T, int H, int k, int window, bool dense) {
    TtPlan p;
    // nodes that share their slots fill the 128 rows together
    p.G = dense ? std::max(1, std::min({TT_G, TT_ROWS / H, T})) : 1;
    p.R8 = (p.G * H + 7) / 8 * 8;
    p.gps = (T + p.G - 1) / p.G;
    p.groups = (int64_t)B * p.gps;
    const int64_t k16 = (k + 15) / 16 * 16, near = window > 0 ? window + (dense ? T : 0) : 0;
    p.list_ld = ((dense ? 0 : k16) + near + 15) / 16 * 16;
    // Splits: every cluster walks its items one after another, each for its tiles and about four
    // tiles' time of filling and draining; with splits the partial outputs are written and read, half a
    // tile's time an item.
    const int64_t tiles = std::max<int64_t>(1, (k16 + near + TT_TILE - 1) / TT_TILE), clusters = std::max(1, ctx->num_sms / 2);
    double best = 1e300;
    p.n_split = 1;
    p.tps = (int)tiles;
    for (int64_t ns = 1; ns <= std::min<int64_t>(tiles, std::max<int64_t>(1, 4 * clusters / p.groups)); ++ns) {
        const int64_t tps = (tiles + ns - 1) / ns, n = (tiles + tps - 1) / tps;
        if (n != ns) continue;
        const double cost = (double)((p.groups * ns + clusters - 1) / clusters) * (tps + (ns > 1 ? 4.5 : 4.0)) + (ns > 1 ? 1.0 : 0.0);
        if (cost < best) {
            best = cost;
            p.n_split = (int)ns;
            p.tps = (int)tps;
        }
    }
    p.qimg = 0;
    p.list = up((size_t)p.groups * p.R8 * 1024, 256);
    p.mask = up(p.list + (size_t)p.groups * p.list_ld * 8, 256);
    p.info = up(p.mask + (dense ? (size_t)p.groups * (p.list_ld / 16) * TT_G * 2 : 0), 256);
    p.rope = up(p.info + (size_t)p.groups * 16, 256);
    p.part_l = up(p.rope + (size_t)B * T * 64 * 4, 256);
    const size_t rows = p.n_split > 1 ? (size_t)p.groups * p.n_split * p.G * H : 0;
    p.part_o = up(p.part_l + rows * 4, 256);
    p.total = p.part_o + rows * TT_C * 4;
    return p;
}

template <bool FP4, bool DENSE>
csa2_status launch_tt(const csa2_ctx* ctx, const TtArgs& a, cudaStream_t s) {
    auto kern = tree_tc_kernel<FP4, DENSE>;
    CSA2_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TT_SMEM));
    const int64_t clusters = std::min<int64_t>(a.items, std::max(1, ctx->num_sms / 2));
    return launch_pdl(kern, dim3((unsigned)(2 * clusters)), dim3(TT_THREADS), TT_SMEM, s, a);
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
    pa.r = c.r;
    pa.q = reinterpret_cast<const __nv_bfloat16*>(c.q);
    pa.kv = reinterpret_cast<const uint8_t*>(c.kv);
    pa.swa = reinterpret_cast<const uint8_t*>(c.swa);
    pa.draft = reinterpret_cast<const uint8_t*>(c.draft);
    pa.kv_row = fp4 ? fp4_row_bytes(TT_C) : TT_C * 2;
    pa.H = c.H;
    pa.G = p.G;
    pa.R8 = p.R8;
    pa.gps = p.gps;
    pa.list_ld = p.list_ld;
    pa.rope = c.rope;
    pa.flags = c.flags;
    pa.qimg = base + p.qimg;
    pa.list = reinterpret_cast<uint64_t*>(base + p.list);
    pa.mask = reinterpret_cast<uint16_t*>(base + p.mask);
    pa.info = reinterpret_cast<int4*>(base + p.info);
    pa.rope_cs = reinterpret_cast<float*>(base + p.rope);
    pa.st = ctx->status;
    csa2_status st = launch_pdl(tree_prep_kernel, dim3((unsigned)p.groups, (unsigned)(p.R8 / 8 + 1)), dim3(256), 0, s, pa);
    if (st != CSA2_OK) return st;
    TtArgs a = {};
    a.qimg = pa.qimg;
    a.list = pa.list;
    a.mask = pa.mask;
    a.info = pa.info;
    a.rope_cs = pa.rope_cs;
    a.kv = pa.kv;
    a.r = c.r;
    a.sink = c.sink;
    a.H = c.H;
    a.G = p.G;
    a.R8 = p.R8;
    a.gps = p.gps;
    a.list_ld = p.list_ld;
    a.groups = p.groups;
    a.items = p.groups * p.n_split;
    a.n_split = p.n_split;
    a.tps = p.tps;
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
    if (fp4) st = dense ? launch_tt<true, true>(ctx, a, s) : launch_tt<true, false>(ctx, a, s);
    else st = dense ? launch_tt<false, true>(ctx, a, s) : launch_tt<false, false>(ctx, a, s);
    if (st != CSA2_OK) return st;
    if (p.n_split > 1) {
        const MergeArgs m = {a.part_o, a.part_l, a.rope_cs, a.sink, p.groups, c.H, p.G, p.gps, c.r.T, p.n_split, c.flags,
                             c.out, a.out_f32, c.lse};
        const int64_t rows = p.groups * p.G * c.H;
        st = launch_pdl(tree_merge_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, m);
        if (st != CSA2_OK) return st;
    }
    return csa2_launch_status();
}
