// Eviction from a cache: which entries stay (csa2_evict_select) and their rows moved
// together (csa2_cache_gather).
//
// Selection: the newest `recent` of a row's n entries stay, and the best of the others by
// (accumulated weight descending, entry ascending).  The threshold is found by radix
// selection on the order-preserving 32-bit key of the weight (digits of 11, 11 and 10
// bits), ties at the threshold go to the lowest entries, and the kept entries are written
// in ascending order.  Nothing depends on thread timing.
//
// Rows of up to 65,536 entries: a thread-block cluster per row, 8,192 entries a CTA in
// registers, read once; the CTAs' digit counts meet through distributed shared memory.  One
// launch, bound by its chain of barriers.  Longer rows: five launches over all SMs (three
// digits, counting, writing), each a pass over the weights, which mostly come from L2; a
// cluster per row would leave most SMs idle there (eight 1M rows on clusters of 8: 206 us; of
// 16, which are slower still: 282 us).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "attn_grad.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int EV_THREADS = 1024;
constexpr int EV_BINS = 2048;
constexpr int EV_KEYS = 8;              // keys a thread holds
constexpr int EV_CTA = EV_THREADS * EV_KEYS;
constexpr int EV_CLUSTER = 8;
constexpr int64_t EV_SHORT = (int64_t)EV_CTA * EV_CLUSTER;   // the longest row of the one-launch path
constexpr int EL_THREADS = 512;
constexpr int EL_CHUNK = 16384;         // least entries a block of the long path takes, and their step
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
    uint32_t* hist;                     // long path: [B][3][EV_BINS]
    uint32_t* cnt;                      // long path: [B][chunks][2] entries above / at the threshold
    int chunks, chunk;                  // chunks of a row, entries of a chunk
};

// A row's entries: n (clamped to ld), of which the last `recent` stay without a contest when
// there are more than keep.
struct Row {
    int64_t n, m;                       // m: old entries 0 .. m-1 compete for `want` places
    uint32_t want;
    bool all;                           // every entry stays
};

__device__ __forceinline__ Row row_of(const EvictArgs& a, int64_t b, bool flag) {
    Row r;
    r.n = a.n_entries[b];
    if (r.n > a.ld) {
        if (flag) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
        r.n = a.ld;
    }
    if (r.n < 0) r.n = 0;
    r.all = r.n <= a.keep;
    r.m = r.all ? 0 : r.n - a.recent;
    r.want = r.all ? 0u : (uint32_t)(a.keep - a.recent);
    return r;
}

// What needs no contest: a whole short row, the newest entries, the padding; thread t of nt.
__device__ __forceinline__ void write_sure(const EvictArgs& a, const Row& r, int32_t* out, int64_t t, int64_t nt) {
    if (r.all) {
        for (int64_t i = t; i < a.keep; i += nt) out[i] = i < r.n ? (int32_t)i : -1;
    } else {
        for (int64_t i = t; i < a.recent; i += nt) out[r.want + i] = (int32_t)(r.m + i);
    }
}

// Exclusive scan over the block of two counts at once (tot: [2][32] shared words).
__device__ __forceinline__ void block_scan2(uint32_t (*tot)[32], uint32_t a, uint32_t b, uint32_t& pa, uint32_t& pb,
                                            uint32_t& ta, uint32_t& tb) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    uint32_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ua = __shfl_up_sync(FULL, ia, o), ub = __shfl_up_sync(FULL, ib, o);
        if (lane >= o) {
            ia += ua;
            ib += ub;
        }
    }
    __syncthreads();
    if (lane == 31) {
        tot[0][w] = ia;
        tot[1][w] = ib;
    }
    __syncthreads();
    uint32_t xa = lane < nw ? tot[0][lane] : 0u, xb = lane < nw ? tot[1][lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ua = __shfl_up_sync(FULL, xa, o), ub = __shfl_up_sync(FULL, xb, o);
        if (lane >= o) {
            xa += ua;
            xb += ub;
        }
    }
    ta = __shfl_sync(FULL, xa, 31);
    tb = __shfl_sync(FULL, xb, 31);
    const uint32_t ba = __shfl_sync(FULL, xa, w > 0 ? w - 1 : 0), bb = __shfl_sync(FULL, xb, w > 0 ? w - 1 : 0);
    pa = (w > 0 ? ba : 0u) + ia - a;
    pb = (w > 0 ? bb : 0u) + ib - b;
}

// Keys of 16 entries, `step` apart from `e` on; past `end` the last one's (end > 0; the caller
// masks them).  Loads without a condition, so that all are in flight together.
__device__ __forceinline__ void load_keys(const float* __restrict__ acc, int64_t e, int step, int64_t end, uint32_t (&key)[16]) {
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = __ldg(acc + min(e + j * step, end - 1));
#pragma unroll
    for (int j = 0; j < 16; ++j) key[j] = evict_key(x[j]);
}

__device__ __forceinline__ int digit_shift(int pass) { return pass == 0 ? 21 : (pass == 1 ? 10 : 0); }
__device__ __forceinline__ int digit_bits(int pass) { return pass == 2 ? 10 : 11; }

// Counts a warp's key in shared memory; lanes with lane 0's digit count together (weights that
// were never touched are all 0).
__device__ __forceinline__ void count_digit(uint32_t* hist, bool in, uint32_t d) {
    const uint32_t d0 = __shfl_sync(FULL, d, 0);
    const unsigned same = __ballot_sync(FULL, in && d == d0);
    if (in && d != d0)
        atomicAdd(&hist[d], 1u);
    else if (same && (threadIdx.x & 31) == 0)
        atomicAdd(&hist[d0], (uint32_t)__popc(same));
}

// Writes a warp's kept entries among base + 32 j + lane in entry order: keys above the
// threshold T, and of those at it the ones with fewer than `rest` of their kind before them.
// pg / pe: entries above / at the threshold before these, updated.
__device__ __forceinline__ void emit(int32_t* out, int64_t e, bool in, uint32_t key, uint32_t T, uint32_t rest, uint32_t& pg,
                                     uint32_t& pe) {
    const unsigned below = (1u << (threadIdx.x & 31)) - 1u;
    const bool g = in && key > T, q = in && key == T;
    const unsigned mg = __ballot_sync(FULL, g), mq = __ballot_sync(FULL, q);
    const uint32_t eqb = pe + __popc(mq & below);
    if (g || (q && eqb < rest)) out[pg + __popc(mg & below) + min(rest, eqb)] = (int32_t)e;
    pg += __popc(mg);
    pe += __popc(mq);
}

struct EvictShared {
    uint32_t hist[2][EV_BINS];          // this CTA's counts (read by the cluster), two passes in turn
    uint32_t warp_tot[2][32];
    uint32_t cnt[2];                    // this CTA's entries above / at the threshold (read by the cluster)
    uint32_t digit, rest;
};

// Rows of at most EV_SHORT entries; a cluster per row, warp w of a CTA holds 256 adjacent entries.
__global__ void __launch_bounds__(EV_THREADS) evict_short_kernel(EvictArgs a) {
    __shared__ EvictShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), nc = (int)cl.num_blocks();
    const int64_t b = blockIdx.x / nc;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const Row r = row_of(a, b, rank == 0 && tid == 0);
    int32_t* out = a.out + b * (int64_t)a.keep;
    write_sure(a, r, out, (int64_t)rank * EV_THREADS + tid, (int64_t)nc * EV_THREADS);
    if (r.want == 0) return;                       // the whole cluster takes this branch
    const float* acc = a.acc + b * a.ld;
    const int64_t w0 = (int64_t)rank * EV_CTA + wid * (32 * EV_KEYS);
    uint32_t key[EV_KEYS];
#pragma unroll
    for (int j = 0; j < EV_KEYS; ++j) {
        const int64_t e = w0 + 32 * j + lane;
        key[j] = e < r.m ? evict_key(acc[e]) : 0u;
    }
    for (int i = tid; i < 2 * EV_BINS; i += EV_THREADS) sh.hist[0][i] = 0;
    __syncthreads();
    uint32_t prefix = 0, mask = 0, rest = r.want;  // the threshold's digits so far; places left within them
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = digit_shift(pass), bits = digit_bits(pass);
        uint32_t* hist = sh.hist[pass & 1];
#pragma unroll
        for (int j = 0; j < EV_KEYS; ++j)
            if (w0 + 32 * j < r.m)
                count_digit(hist, w0 + 32 * j + lane < r.m && (key[j] & mask) == prefix, (key[j] >> shift) & ((1u << bits) - 1));
        cl.sync();
        // the cluster's counts: two bins a thread, highest digit first
        uint32_t c0 = 0, c1 = 0;
        const int b0 = (1 << bits) - 1 - 2 * tid;
        if (b0 >= 1) {
            uint2 x[EV_CLUSTER];
#pragma unroll
            for (int k = 0; k < EV_CLUSTER; ++k)
                x[k] = k < nc ? *reinterpret_cast<const uint2*>(cl.map_shared_rank(hist, k) + b0 - 1) : make_uint2(0u, 0u);
#pragma unroll
            for (int k = 0; k < EV_CLUSTER; ++k) {
                c0 += x[k].y;
                c1 += x[k].x;
            }
        }
        uint32_t p, q, tp, tq;
        block_scan2(sh.warp_tot, c0 + c1, 0u, p, q, tp, tq);
        if (p < rest && rest <= p + c0 + c1) {
            const bool first = rest <= p + c0;
            sh.digit = (uint32_t)(first ? b0 : b0 - 1);
            sh.rest = rest - p - (first ? 0u : c0);
        }
        // (the buffer of the pass before this one is free: every CTA has passed this pass's barrier)
        if (pass == 1)
            for (int i = tid; i < EV_BINS; i += EV_THREADS) sh.hist[0][i] = 0;
        __syncthreads();
        prefix |= sh.digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        rest = sh.rest;
        __syncthreads();
    }
    // kept: keys above the threshold, and the first `rest` of those at it, in entry order
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < EV_KEYS; ++j) {
        const bool in = w0 + 32 * j + lane < r.m;
        gt += __popc(__ballot_sync(FULL, in && key[j] > prefix));
        eq += __popc(__ballot_sync(FULL, in && key[j] == prefix));
    }
    uint32_t pg, pe, tg, te;
    block_scan2(sh.warp_tot, lane == 0 ? gt : 0u, lane == 0 ? eq : 0u, pg, pe, tg, te);
    pg = __shfl_sync(FULL, pg, 0);                 // lane 0's prefixes: the warps before this one
    pe = __shfl_sync(FULL, pe, 0);
    if (tid == 0) {
        sh.cnt[0] = tg;
        sh.cnt[1] = te;
    }
    cl.sync();
    for (int k = 0; k < rank; ++k) {               // and the CTAs before this one
        const uint32_t* c = cl.map_shared_rank(sh.cnt, k);
        pg += c[0];
        pe += c[1];
    }
#pragma unroll
    for (int j = 0; j < EV_KEYS; ++j) emit(out, w0 + 32 * j + lane, w0 + 32 * j + lane < r.m, key[j], prefix, rest, pg, pe);
    cl.sync();                                     // no CTA leaves while another reads its counts
}

// The threshold's digits after `passes` passes, from the row's counts (each block works them out
// again: 2,048 counts a digit).
__device__ __forceinline__ void long_prefix(const uint32_t* hist, int passes, uint32_t want, uint32_t (*tot)[32],
                                            uint32_t* found, uint32_t& prefix, uint32_t& mask, uint32_t& rest) {
    prefix = mask = 0;
    rest = want;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = digit_shift(pass), bits = digit_bits(pass);
        const int per = (1 << bits) / EL_THREADS;             // 4 or 2 bins a thread, highest digit first
        const int top = (1 << bits) - 1 - per * (int)threadIdx.x;
        uint32_t c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = i < per ? hist[pass * EV_BINS + top - i] : 0u;
            sum += c[i];
        }
        uint32_t p, q, tp, tq;
        block_scan2(tot, sum, 0u, p, q, tp, tq);
        if (p < rest && rest <= p + sum) {
            uint32_t left = rest - p;
            int d = 0;
            while (left > c[d]) left -= c[d++];
            found[0] = (uint32_t)(top - d);
            found[1] = left;
        }
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= ((1u << bits) - 1) << shift;
        rest = found[1];
        __syncthreads();
    }
}

// Long rows, digit `pass`: a block counts one chunk's entries that match the digits so far.
__global__ void __launch_bounds__(EL_THREADS) evict_long_count_kernel(EvictArgs a, int pass) {
    __shared__ uint32_t hist[EV_BINS], tot[2][32], found[2];
    pdl_wait();
    pdl_trigger();
    const int64_t b = blockIdx.y;
    const Row r = row_of(a, b, pass == 0 && blockIdx.x == 0 && threadIdx.x == 0);
    if (pass == 0)
        write_sure(a, r, a.out + b * (int64_t)a.keep, (int64_t)blockIdx.x * EL_THREADS + threadIdx.x,
                   (int64_t)gridDim.x * EL_THREADS);
    const int64_t e0 = (int64_t)blockIdx.x * a.chunk, e1 = min(r.m, e0 + a.chunk);
    if (r.want == 0 || e0 >= e1) return;
    uint32_t* rows = a.hist + b * 3 * EV_BINS;
    uint32_t prefix, mask, rest;
    for (int i = threadIdx.x; i < EV_BINS; i += EL_THREADS) hist[i] = 0;
    long_prefix(rows, pass, r.want, tot, found, prefix, mask, rest);
    __syncthreads();
    const int shift = digit_shift(pass), bits = digit_bits(pass);
    const float* acc = a.acc + b * a.ld;
    for (int64_t base = e0; base < e1; base += 16 * EL_THREADS) {
        uint32_t key[16];
        load_keys(acc, base + threadIdx.x, EL_THREADS, e1, key);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            count_digit(hist, base + j * EL_THREADS + threadIdx.x < e1 && (key[j] & mask) == prefix,
                        (key[j] >> shift) & ((1u << bits) - 1));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (1 << bits); i += EL_THREADS)
        if (hist[i]) atomicAdd(&rows[pass * EV_BINS + i], hist[i]);
}

// Long rows: entries of each chunk above and at the threshold (EMIT = false), then the kept ones
// of each chunk behind those of the chunks before it (EMIT = true).  Warp w owns a sixteenth of
// the chunk.
template <bool EMIT>
__global__ void __launch_bounds__(EL_THREADS) evict_long_write_kernel(EvictArgs a) {
    __shared__ uint32_t tot[2][32], found[2];
    pdl_wait();
    pdl_trigger();
    const int64_t b = blockIdx.y;
    const Row r = row_of(a, b, false);
    const int64_t e0 = (int64_t)blockIdx.x * a.chunk, e1 = min(r.m, e0 + a.chunk);
    if (r.want == 0 || e0 >= e1) return;
    uint32_t T, mask, rest;
    long_prefix(a.hist + b * 3 * EV_BINS, 3, r.want, tot, found, T, mask, rest);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int per_w = a.chunk / (EL_THREADS / 32);
    const int64_t w0 = min(e1, e0 + wid * per_w), w1 = min(e1, w0 + per_w);
    const float* acc = a.acc + b * a.ld;
    uint32_t gt = 0, eq = 0;
    for (int64_t base = w0; base < w1; base += 16 * 32) {
        uint32_t key[16];
        load_keys(acc, base + lane, 32, w1, key);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const bool in = base + j * 32 + lane < w1;
            gt += in && key[j] > T;
            eq += in && key[j] == T;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        gt += __shfl_xor_sync(FULL, gt, o);
        eq += __shfl_xor_sync(FULL, eq, o);
    }
    uint32_t pg, pe, tg, te;
    block_scan2(tot, lane == 0 ? gt : 0u, lane == 0 ? eq : 0u, pg, pe, tg, te);
    uint32_t* cnt = a.cnt + b * a.chunks * 2;
    if (!EMIT) {
        if (threadIdx.x == 0) {
            cnt[2 * blockIdx.x] = tg;
            cnt[2 * blockIdx.x + 1] = te;
        }
        return;
    }
    pg = __shfl_sync(FULL, pg, 0);
    pe = __shfl_sync(FULL, pe, 0);
    uint32_t g0 = 0, q0 = 0;                       // the chunks before this one
    for (int i = lane; i < (int)blockIdx.x; i += 32) {
        g0 += cnt[2 * i];
        q0 += cnt[2 * i + 1];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        g0 += __shfl_xor_sync(FULL, g0, o);
        q0 += __shfl_xor_sync(FULL, q0, o);
    }
    pg += g0;
    pe += q0;
    int32_t* out = a.out + b * (int64_t)a.keep;
    for (int64_t base = w0; base < w1; base += 16 * 32) {
        uint32_t key[16];
        load_keys(acc, base + lane, 32, w1, key);
#pragma unroll
        for (int j = 0; j < 16; ++j) emit(out, base + j * 32 + lane, base + j * 32 + lane < w1, key[j], T, rest, pg, pe);
    }
}

size_t long_hist_bytes(int B) { return (size_t)B * 3 * EV_BINS * 4; }

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
        if (id < -1 || id >= N) csa2_flag(st, CSA2_DEVBIT_RANGE);
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

}  // namespace

extern "C" size_t csa2_evict_select_workspace_bytes(int B, int64_t ld) {
    if (B <= 0 || ld <= EV_SHORT) return 0;
    return long_hist_bytes(B) + (size_t)B * ((ld + EL_CHUNK - 1) / EL_CHUNK) * 2 * 4;
}

extern "C" csa2_status csa2_evict_select(csa2_ctx* ctx, const float* acc, int B, int64_t ld, const int64_t* n_entries,
                                         int keep, int recent, int32_t* out_idx, void* ws, size_t ws_bytes, void* stream) {
    if (!ctx || B < 0 || ld < 0 || ld > 0x7FFFFFFF || keep < 1 || recent < 0 || recent > keep) return CSA2_ERR_INVALID_ARG;
    if (B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0) return CSA2_OK;
    if (!n_entries || !out_idx || (ld > 0 && !acc)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(acc, 4) || !aligned(n_entries, 8) || !aligned(out_idx, 4) || !aligned(ws, 16)) return CSA2_ERR_INVALID_ARG;
    const size_t need = csa2_evict_select_workspace_bytes(B, ld);
    if (need > 0 && (!ws || ws_bytes < need)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    EvictArgs a = {acc, ld, n_entries, keep, recent, out_idx, ctx->status, nullptr, nullptr, 0, 0};
    if (need > 0) {
        a.hist = reinterpret_cast<uint32_t*>(ws);
        a.cnt = a.hist + (size_t)B * 3 * EV_BINS;
        // one wave of blocks, two an SM, if the rows give them work (eight 1M rows in chunks of 16,384,
        // 1.7 waves: 140 us)
        const int64_t even = ((int64_t)B * ld + 2 * ctx->num_sms - 1) / (2 * ctx->num_sms);
        const int64_t chunk = std::min<int64_t>(std::max<int64_t>(1, (even + EL_CHUNK - 1) / EL_CHUNK), 1 << 16) * EL_CHUNK;
        a.chunk = (int)chunk;
        a.chunks = (int)((ld + chunk - 1) / chunk);
        CSA2_CHECK_CUDA(cudaMemsetAsync(a.hist, 0, long_hist_bytes(B), s));
        const dim3 grid((unsigned)a.chunks, (unsigned)B), block(EL_THREADS);
        csa2_status r = CSA2_OK;
        for (int pass = 0; pass < 3 && r == CSA2_OK; ++pass) r = launch_pdl(evict_long_count_kernel, grid, block, 0, s, a, pass);
        if (r == CSA2_OK) r = launch_pdl(evict_long_write_kernel<false>, grid, block, 0, s, a);
        if (r == CSA2_OK) r = launch_pdl(evict_long_write_kernel<true>, grid, block, 0, s, a);
        return r != CSA2_OK ? r : csa2_launch_status();
    }
    int nc = 1;
    while ((int64_t)nc * EV_CTA < ld) nc *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * nc));
    cfg.blockDim = dim3(EV_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nc;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_short_kernel, a) != cudaSuccess) return CSA2_ERR_CUDA;
    return csa2_launch_status();
}

extern "C" csa2_status csa2_cache_gather(csa2_ctx* ctx, const void* src, int64_t row_bytes, int B, int64_t N,
                                         const int32_t* idx, int keep, void* dst, void* stream) {
    if (!ctx || B < 0 || N < 0 || keep < 0 || row_bytes < 4 || row_bytes > (1 << 20)) return CSA2_ERR_INVALID_ARG;
    if (row_bytes % 4) return CSA2_ERR_UNSUPPORTED;
    if (B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0 || keep == 0) return CSA2_OK;
    if ((N > 0 && !src) || !idx || !dst || !aligned(src, 4) || !aligned(dst, 4) || !aligned(idx, 4)) return CSA2_ERR_INVALID_ARG;
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
