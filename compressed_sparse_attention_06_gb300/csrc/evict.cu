// Eviction from a cache: which entries stay (csa2_evict_select) and their rows moved
// together (csa2_cache_gather).
//
// Selection: the newest `recent` of a row's n entries stay, and the best of the others by
// (accumulated weight descending, entry ascending).  The threshold is found by radix
// selection on the order-preserving 32-bit key of the weight (digits of 11, 11 and 10
// bits), ties at the threshold go to the lowest entries, and the kept entries are written
// in ascending order.  Nothing depends on thread timing.
//
// One thread-block cluster per row: each CTA owns a contiguous stretch of the entries and
// counts its digits in shared memory; the cluster adds the counts through distributed
// shared memory, so a row needs one launch and no workspace.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "attn_grad.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int EV_THREADS = 1024;
constexpr int EV_BINS = 2048;
constexpr int EV_CLUSTER_MAX = 16;      // where the device runs such clusters (more than 8 is not portable)
constexpr int EV_PER_CTA = 8192;        // entries of a row that are worth another CTA
constexpr unsigned FULL = 0xffffffffu;

// Key of a weight: larger weight, larger key; NaN (of any sign) above +inf.
__device__ __forceinline__ uint32_t evict_key(float x) { return isnan(x) ? 0xFFFFFFFFu : order_key(x); }

struct EvictArgs {
    const float* acc;
    int64_t ld;
    const int64_t* n_entries;
    int keep, recent;
    int32_t* out;
    unsigned* st;
};

struct EvictShared {
    uint32_t hist[EV_BINS];      // this CTA's counts (read by the cluster)
    uint32_t sum[EV_BINS];       // the cluster's counts
    uint32_t warp_tot[2][32];
    uint32_t cnt_gt, cnt_eq;     // this CTA's entries above / at the threshold (read by the cluster)
    uint32_t digit, rest;
};

// Exclusive scan over the block of two counts at once.
__device__ __forceinline__ void block_scan2(EvictShared& sh, uint32_t a, uint32_t b, uint32_t& pa, uint32_t& pb,
                                            uint32_t& ta, uint32_t& tb) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += ua;
            ib += ub;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sh.warp_tot[0][w] = ia;
        sh.warp_tot[1][w] = ib;
    }
    __syncthreads();
    uint32_t ba = 0, bb = 0;
    ta = tb = 0;
#pragma unroll 8
    for (int i = 0; i < EV_THREADS / 32; ++i) {
        const uint32_t xa = sh.warp_tot[0][i], xb = sh.warp_tot[1][i];
        if (i < w) {
            ba += xa;
            bb += xb;
        }
        ta += xa;
        tb += xb;
    }
    pa = ba + ia - a;
    pb = bb + ib - b;
}

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(EvictArgs a) {
    __shared__ EvictShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), nc = (int)cl.num_blocks();
    const int64_t b = blockIdx.x / nc;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int64_t n = a.n_entries[b];
    if (n > a.ld) {
        if (rank == 0 && tid == 0) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
        n = a.ld;
    }
    if (n < 0) n = 0;
    const float* acc = a.acc + b * a.ld;
    int32_t* out = a.out + b * (int64_t)a.keep;
    const int64_t kept = min(n, (int64_t)a.keep);
    for (int64_t i = kept + (int64_t)rank * EV_THREADS + tid; i < a.keep; i += (int64_t)nc * EV_THREADS) out[i] = -1;
    if (n <= a.keep) {
        for (int64_t i = (int64_t)rank * EV_THREADS + tid; i < n; i += (int64_t)nc * EV_THREADS) out[i] = (int32_t)i;
        return;                                    // the whole cluster takes this branch
    }
    // the newest entries stay without a contest: old entries 0 .. m-1 compete for `want` places
    const int64_t m = n - a.recent;
    const uint32_t want = (uint32_t)(a.keep - a.recent);
    for (int64_t i = (int64_t)rank * EV_THREADS + tid; i < a.recent; i += (int64_t)nc * EV_THREADS)
        out[want + i] = (int32_t)(m + i);
    if (want == 0) return;
    const int64_t per = (m + nc - 1) / nc;
    const int64_t e0 = min(m, (int64_t)rank * per), e1 = min(m, e0 + per);
    uint32_t prefix = 0, mask = 0, rest = want;    // the threshold's digits so far; places left within them
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < EV_BINS; i += EV_THREADS) sh.hist[i] = 0;
        __syncthreads();
        // eight loads in flight a thread; lanes with lane 0's digit count together (weights that
        // were never touched are all 0)
        for (int64_t base = e0; base < e1; base += 8 * EV_THREADS) {
            uint32_t key[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t e = base + j * EV_THREADS + tid;
                key[j] = e < e1 ? evict_key(acc[e]) : 0u;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = base + j * EV_THREADS + tid < e1 && (key[j] & mask) == prefix;
                const uint32_t d = (key[j] >> shift) & ((1u << bits) - 1), d0 = __shfl_sync(FULL, d, 0);
                const unsigned same = __ballot_sync(FULL, in && d == d0);
                if (in && d != d0)
                    atomicAdd(&sh.hist[d], 1u);
                else if (same && lane == 0)
                    atomicAdd(&sh.hist[d0], (uint32_t)__popc(same));
            }
        }
        cl.sync();
        // the cluster's counts: two bins a thread, highest digit first
        uint32_t c0 = 0, c1 = 0;
        const int b0 = (1 << bits) - 1 - 2 * tid, b1 = b0 - 1;
        if (b1 >= 0) {
            for (int r = 0; r < nc; ++r) {
                const uint32_t* h = cl.map_shared_rank(sh.hist, r);
                c0 += h[b0];
                c1 += h[b1];
            }
        }
        uint32_t p, q, tp, tq;
        block_scan2(sh, c0 + c1, 0u, p, q, tp, tq);
        if (p < rest && rest <= p + c0 + c1 && b1 >= 0) {
            const bool first = rest <= p + c0;
            sh.digit = (uint32_t)(first ? b0 : b1);
            sh.rest = rest - p - (first ? 0u : c0);
        }
        cl.sync();                                 // every CTA is done with the counts
        prefix |= sh.digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        rest = sh.rest;
        __syncthreads();
    }
    // kept: keys above the threshold, and the first `rest` of those at it, in entry order.  Warp w
    // owns a stretch of the CTA's entries: it counts both kinds, then writes its own.
    const int64_t per_w = ((e1 - e0 + EV_THREADS - 1) / EV_THREADS) * 32;
    const int64_t w0 = min(e1, e0 + wid * per_w), w1 = min(e1, w0 + per_w);
    uint32_t gt = 0, eq = 0;
    for (int64_t base = w0; base < w1; base += 8 * 32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t e = base + j * 32 + lane;
            const uint32_t k = e < w1 ? evict_key(acc[e]) : 0u;
            gt += e < w1 && k > prefix;
            eq += e < w1 && k == prefix;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        gt += __shfl_xor_sync(FULL, gt, o);
        eq += __shfl_xor_sync(FULL, eq, o);
    }
    uint32_t pg, pe, tg, te;
    block_scan2(sh, lane == 0 ? gt : 0u, lane == 0 ? eq : 0u, pg, pe, tg, te);
    pg = __shfl_sync(FULL, pg, 0);                 // lane 0's prefixes: the warps before this one
    pe = __shfl_sync(FULL, pe, 0);
    if (tid == 0) {
        sh.cnt_gt = tg;
        sh.cnt_eq = te;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {               // and the CTAs before this one
        pg += *cl.map_shared_rank(&sh.cnt_gt, r);
        pe += *cl.map_shared_rank(&sh.cnt_eq, r);
    }
    const unsigned below = (1u << lane) - 1u;
    for (int64_t base = w0; base < w1; base += 8 * 32) {
        uint32_t key[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t e = base + j * 32 + lane;
            key[j] = e < w1 ? evict_key(acc[e]) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t e = base + j * 32 + lane;
            const bool g = e < w1 && key[j] > prefix, q = e < w1 && key[j] == prefix;
            const unsigned mg = __ballot_sync(FULL, g), mq = __ballot_sync(FULL, q);
            const uint32_t eqb = pe + __popc(mq & below);
            // kept before this entry: all above the threshold, and of those at it at most `rest`
            if (g || (q && eqb < rest)) out[pg + __popc(mg & below) + min(rest, eqb)] = (int32_t)e;
            pg += __popc(mg);
            pe += __popc(mq);
        }
    }
    cl.sync();                                     // no CTA leaves while another reads its counts
}

// Rows dst[b, i] = src[b, idx[b, i]] in pieces of V; -1 leaves dst's row as it is.  A block
// moves `rows_b` rows: their ids go to shared memory, then each thread has up to eight pieces
// in flight, adjacent threads adjacent pieces, so both sides are read and written in full
// lines where rows are long and the destination always is.
constexpr int GA_THREADS = 256, GA_PIECES = 8, GA_ROWS = 2048;

template <typename V>
__global__ void __launch_bounds__(GA_THREADS) cache_gather_kernel(const V* src, uint32_t pieces, int64_t N,
                                                                  const int32_t* idx, int64_t rows, uint32_t rows_b,
                                                                  int keep, V* dst, unsigned* st) {
    __shared__ int64_t from[GA_ROWS];              // first piece of the source row, -1 = leave
    const int64_t r0 = (int64_t)blockIdx.x * rows_b;
    const uint32_t nr = (uint32_t)min((int64_t)rows_b, rows - r0), total = nr * pieces;
    for (uint32_t r = threadIdx.x; r < nr; r += GA_THREADS) {
        const int64_t row = r0 + r;
        const int32_t id = idx[row];
        if (id >= N) csa2_flag(st, CSA2_DEVBIT_RANGE);
        from[r] = id >= 0 && id < N ? ((row / keep) * N + id) * (int64_t)pieces : -1;
    }
    __syncthreads();
    V* out = dst + r0 * pieces;
    for (uint32_t u0 = threadIdx.x; u0 < total; u0 += GA_THREADS * GA_PIECES) {
        V v[GA_PIECES];
        bool live[GA_PIECES];
#pragma unroll
        for (int j = 0; j < GA_PIECES; ++j) {
            const uint32_t u = u0 + j * GA_THREADS;
            const uint32_t r = u / pieces;
            const int64_t f = u < total ? from[r] : -1;
            live[j] = f >= 0;
            if (live[j]) v[j] = __ldcs(src + f + (u - r * pieces));
        }
#pragma unroll
        for (int j = 0; j < GA_PIECES; ++j)
            if (live[j]) __stcs(out + u0 + j * GA_THREADS, v[j]);
    }
}

// Whether clusters of 16 CTAs of the selection run on the device (asked once per device).
bool evict_cluster16(int device) {
    static std::atomic<int> known[64];             // 0 = not asked, 1 = no, 2 = yes
    std::atomic<int>& k = known[device & 63];
    int v = k.load(std::memory_order_relaxed);
    if (v == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(EV_THREADS);
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 16;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        const bool ok = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                            cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, evict_select_kernel, &cfg) == cudaSuccess && n > 0;
        (void)cudaGetLastError();
        v = ok ? 2 : 1;
        k.store(v, std::memory_order_relaxed);
    }
    return v == 2;
}

}  // namespace

extern "C" csa2_status csa2_evict_select(csa2_ctx* ctx, const float* acc, int B, int64_t ld, const int64_t* n_entries,
                                         int keep, int recent, int32_t* out_idx, void* stream) {
    if (!ctx || B < 0 || ld < 0 || ld > 0x7FFFFFFF || keep < 1 || recent < 0 || recent > keep) return CSA2_ERR_INVALID_ARG;
    if (B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0) return CSA2_OK;
    if (!n_entries || !out_idx || (ld > 0 && !acc)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(acc, 4) || !aligned(n_entries, 8) || !aligned(out_idx, 4)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    int nc = 1;
    while (nc < 8 && (int64_t)nc * EV_PER_CTA < ld) nc *= 2;
    if (nc == 8 && (int64_t)nc * EV_PER_CTA < ld && evict_cluster16(ctx->device)) nc = EV_CLUSTER_MAX;
    const EvictArgs a = {acc, ld, n_entries, keep, recent, out_idx, ctx->status};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * nc));
    cfg.blockDim = dim3(EV_THREADS);
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nc;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a) != cudaSuccess) return CSA2_ERR_CUDA;
    return csa2_launch_status();
}

extern "C" csa2_status csa2_cache_gather(csa2_ctx* ctx, const void* src, int64_t row_bytes, int B, int64_t N,
                                         const int32_t* idx, int keep, void* dst, void* stream) {
    if (!ctx || B < 0 || N < 0 || keep < 0 || row_bytes < 4 || row_bytes > (1 << 20)) return CSA2_ERR_INVALID_ARG;
    if (row_bytes % 4) return CSA2_ERR_UNSUPPORTED;
    if (B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0 || keep == 0) return CSA2_OK;
    if (!src || !idx || !dst || !aligned(src, 4) || !aligned(dst, 4) || !aligned(idx, 4)) return CSA2_ERR_INVALID_ARG;
    // moving rows within one buffer would overwrite rows before they are read
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(src), d0 = reinterpret_cast<uintptr_t>(dst);
    const uintptr_t s1 = s0 + (size_t)B * N * row_bytes, d1 = d0 + (size_t)B * keep * row_bytes;
    if (s0 < d1 && d0 < s1) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    const int64_t rows = (int64_t)B * keep;
    const bool wide = row_bytes % 16 == 0 && aligned(src, 16) && aligned(dst, 16);
    const int64_t pieces = row_bytes / (wide ? 16 : 4);
    const int64_t rows_b = std::min<int64_t>(GA_ROWS, std::max<int64_t>(1, GA_THREADS * GA_PIECES / pieces));
    const int64_t blocks = (rows + rows_b - 1) / rows_b;
    if (blocks > 0x7FFFFFFF) return CSA2_ERR_UNSUPPORTED;
    if (wide)
        cache_gather_kernel<uint4><<<(unsigned)blocks, GA_THREADS, 0, s>>>(
            reinterpret_cast<const uint4*>(src), (uint32_t)pieces, N, idx, rows, (uint32_t)rows_b, keep,
            reinterpret_cast<uint4*>(dst), ctx->status);
    else
        cache_gather_kernel<uint32_t><<<(unsigned)blocks, GA_THREADS, 0, s>>>(
            reinterpret_cast<const uint32_t*>(src), (uint32_t)pieces, N, idx, rows, (uint32_t)rows_b, keep,
            reinterpret_cast<uint32_t*>(dst), ctx->status);
    return csa2_launch_status();
}
