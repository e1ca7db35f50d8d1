// Caches in pages: sequences that share pages (fork, free), pages made writable (reserve, copy on
// write), a pool whose used pages are moved to its front (compact), whole pages copied, and rows
// written to and read from pages through the table.
//
// The only state is refs, the number of places that hold a page, so there is no free list to go
// out of step: a call that needs free pages finds the lowest ones by a pass over refs.  That pass
// and what follows from it are one thread-block cluster of 8 CTAs whose phases meet at cluster
// barriers (a launch of its own per phase would cost more than the phase for any pool that fits a
// GPU), or one CTA where the state is small; the ranks come from counts in order of (sequence, page)
// and of page id, so results do not depend on timing.  A call is short, and a step makes several: each
// kernel's launch overlaps the end of the one before (64 continuations of 8 prompts, 7 kernels: 101 us,
// 110 without).
#include <algorithm>

#include "attn_grad.cuh"
#include "csa2_internal.cuh"

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int PG_CTAS = 8;               // CTAs of the cluster at most (gridDim.x of them)
constexpr int PG_THREADS = 1024;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_SEQS = 65536 / PG_CTAS; // sequences of a CTA at most
// One CTA takes a small state in less time than the cluster's barriers cost (reserve of 16 pages of a pool
// of 25 in cold caches: 10.9 us, in a cluster 12.7; of 4,160 pages of 12,000: 26.6 and 13 us).
constexpr int PG_SMALL_PAGES = 2048, PG_SMALL_SEQS = 256;

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// v to *p of CTA `rank` of the cluster
__device__ __forceinline__ void put_remote(const uint32_t* p, uint32_t rank, uint32_t v) {
    uint32_t a, r;
    a = (uint32_t)__cvta_generic_to_shared(p);
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(r), "r"(v) : "memory");
}

// Exclusive prefix of v over the block's threads and the block's total.  `tmp`: PG_WARPS + 1 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t* tmp, uint32_t v, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                     // tmp may still be read from the call before
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const uint32_t own = lane < PG_WARPS ? tmp[lane] : 0u;
        uint32_t t = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(FULL, t, o);
            if (lane >= o) t += y;
        }
        tmp[lane] = t - own;
        if (lane == 31) tmp[PG_WARPS] = t;
    }
    __syncthreads();
    total = tmp[PG_WARPS];
    return tmp[warp] + x - v;
}
static_assert(PG_WARPS == 32, "one warp scans the warps' totals");

__global__ void __launch_bounds__(256) pages_fork_kernel(int32_t* refs, int64_t n_pages, const int32_t* table, int B, int P,
                                                         const int32_t* parent, int64_t total, int32_t* out, unsigned* st) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t b = i / P;
        const int32_t p = parent[b];
        if (p >= B) csa2_flag(st, CSA2_DEVBIT_RANGE);
        int32_t t = p >= 0 && p < B ? table[(int64_t)p * P + (i - b * P)] : -1;
        if (t < -1 || t >= n_pages) {
            csa2_flag(st, CSA2_DEVBIT_RANGE);
            t = -1;
        }
        out[i] = t;
        if (t >= 0) atomicAdd(refs + t, 1);
    }
}

__global__ void __launch_bounds__(256) pages_free_kernel(int32_t* refs, int64_t n_pages, int32_t* table, int P, int64_t total,
                                                         int page, const int64_t* keep, unsigned* st) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t b = i / P;
        const int64_t k = keep ? keep[b] : 0;
        if (k < 0 || (i - b * P) * (int64_t)page < k) continue;
        const int32_t t = table[i];
        if (t == -1) continue;
        table[i] = -1;
        if (t < 0 || t >= n_pages) {
            csa2_flag(st, CSA2_DEVBIT_RANGE);
        } else if (atomicSub(refs + t, 1) <= 0) {    // more places than uses: the count stays at 0
            atomicAdd(refs + t, 1);
            csa2_flag(st, CSA2_DEVBIT_RANGE);
        }
    }
}

struct ReserveArgs {
    int32_t* refs;
    int64_t n_pages;
    int32_t* table;
    int B, P, page;
    const int64_t* first;
    const int64_t* count;
    int64_t* granted;
    int32_t* copies;
    int32_t* free_ids;                   // [n_pages] the free pages, lowest first
    uint32_t* want;                      // [B, W] bit j: page j0 + 32 w + j is to be replaced
    uint32_t* base;                      // [B, W] replaced pages of this CTA's sequences before the word
    int W;
    unsigned* st;
};

// Pages [j0, j1) that a sequence's entries lie on (none: j0 == j1), limit = the first entry that
// cannot be written for lack of table.
struct PageRange {
    int j0, j1;
    int64_t first, end;
};
__device__ __forceinline__ PageRange page_range(const ReserveArgs& a, int64_t b, bool flag) {
    PageRange r = {0, 0, a.first[b], 0};
    const int64_t n = a.count[b], cap = (int64_t)a.P * a.page;
    if (r.first < 0 || n <= 0) {
        r.first = r.end = 0;
        return r;
    }
    r.end = r.first >= cap ? r.first : (n > cap - r.first ? cap : r.first + n);
    if (flag && (r.first >= cap || n > cap - r.first)) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
    if (r.end > r.first) {
        r.j0 = (int)(r.first / a.page);
        r.j1 = (int)((r.end + a.page - 1) / a.page);
    }
    return r;
}

struct ReserveSmem {
    uint32_t words[PG_SEQS + 1];         // words of 32 pages before each of the CTA's sequences
    int32_t fail[PG_SEQS];               // the first page a sequence does not get
    uint32_t tmp[PG_WARPS + 1];
    uint32_t wants[PG_CTAS], frees[PG_CTAS];
};

// The sequence (of the CTA's) that flattened word i belongs to.
__device__ __forceinline__ int word_seq(const uint32_t* words, int n, uint32_t i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (words[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(PG_THREADS) pages_reserve_kernel(const ReserveArgs a) {
    extern __shared__ uint8_t raw[];
    ReserveSmem& s = *reinterpret_cast<ReserveSmem*>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cta_rank();
    pdl_wait();
    pdl_trigger();
    cluster_sync();                      // every CTA runs: its shared memory may be written
    // the sequences of this CTA, and the words of their pages
    const int nc = gridDim.x;
    const int per = (a.B + nc - 1) / nc;
    const int b0 = min(a.B, (int)rank * per), nb = min(a.B, b0 + per) - b0;
    uint32_t n_words = 0;
    for (int i0 = 0; i0 < nb; i0 += PG_THREADS) {
        const int i = i0 + threadIdx.x;
        uint32_t w = 0, total;
        if (i < nb) {
            const PageRange r = page_range(a, b0 + i, true);
            w = ((uint32_t)(r.j1 - r.j0) + 31u) / 32u;
            s.fail[i] = 0x7FFFFFFF;
        }
        const uint32_t before = block_scan(s.tmp, w, total);
        if (i < nb) s.words[i] = n_words + before;
        n_words += total;
    }
    __syncthreads();
    // which pages are to be replaced: a warp a word
    uint32_t wants = 0;
    for (uint32_t i0 = 0; i0 < n_words; i0 += PG_WARPS) {
        const uint32_t i = i0 + warp;
        uint32_t mask = 0, total;
        int64_t at = 0;
        if (i < n_words) {
            const int q = word_seq(s.words, nb, i);
            const int64_t b = b0 + q;
            const PageRange r = page_range(a, b, false);
            const uint32_t w = i - s.words[q];
            const int64_t j = r.j0 + 32 * (int64_t)w + lane;      // (past 32 bits behind the longest rows)
            at = b * a.W + w;
            bool want = false;
            if (j < r.j1) {
                const int32_t t = a.table[b * a.P + j];
                want = t == -1;
                if (!want) {
                    const int32_t uses = t >= 0 && t < a.n_pages ? a.refs[t] : 0;
                    want = uses > 1;
                    if (uses < 1) {      // no page of the pool, or one that is free
                        csa2_flag(a.st, CSA2_DEVBIT_RANGE);
                        atomicMin(&s.fail[q], (int)j);
                    }
                }
            }
            mask = __ballot_sync(FULL, want);
        }
        const uint32_t before = block_scan(s.tmp, lane == 0 ? __popc(mask) : 0u, total);
        if (i < n_words && lane == 0) {
            a.want[at] = mask;
            a.base[at] = wants + before;
        }
        wants += total;
    }
    // the free pages of this CTA's share of the pool, 4 a thread at a time
    const int64_t share = ((a.n_pages + nc - 1) / nc + 3) / 4 * 4;
    const int64_t p0 = min(a.n_pages, rank * share), p1 = min(a.n_pages, p0 + share);
    uint32_t mine = 0, frees;
    for (int64_t p = p0 + threadIdx.x; p < p1; p += PG_THREADS) mine += a.refs[p] == 0;
    block_scan(s.tmp, mine, frees);
    if (threadIdx.x < nc) {
        put_remote(&s.wants[rank], threadIdx.x, wants);
        put_remote(&s.frees[rank], threadIdx.x, frees);
    }
    cluster_sync();
    uint32_t all_wants = 0, all_frees = 0, want0 = 0, free0 = 0;
    for (int i = 0; i < nc; ++i) {
        if (i < (int)rank) {
            want0 += s.wants[i];
            free0 += s.frees[i];
        }
        all_wants += s.wants[i];
        all_frees += s.frees[i];
    }
    // their ids, as many as are wanted
    for (int64_t q = p0; q < p1 && free0 < all_wants; q += 4 * PG_THREADS) {
        const int64_t p = q + 4 * (int64_t)threadIdx.x;
        bool f[4];
        uint32_t n = 0, total;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = p + j < p1 && a.refs[p + j] == 0;
            n += f[j];
        }
        uint32_t at = free0 + block_scan(s.tmp, n, total);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (f[j] && at < all_wants) a.free_ids[at++] = (int32_t)(p + j);
        free0 += total;
    }
    __threadfence();
    cluster_sync();                      // every id is listed, every count of uses has been read
    for (uint32_t i = warp; i < n_words; i += PG_WARPS) {
        const int q = word_seq(s.words, nb, i);
        const int64_t b = b0 + q;
        const PageRange r = page_range(a, b, false);
        const uint32_t w = i - s.words[q];
        const int64_t j = r.j0 + 32 * (int64_t)w + lane;
        const uint32_t mask = a.want[b * a.W + w];
        int2 copy = make_int2(-1, -1);
        if ((mask >> lane) & 1u) {
            const uint32_t k = want0 + a.base[b * a.W + w] + __popc(mask & ((1u << lane) - 1u));
            if (k < all_frees) {
                const int32_t old = a.table[b * a.P + j], id = a.free_ids[k];
                a.table[b * a.P + j] = id;
                a.refs[id] = 1;
                if (old >= 0) {
                    atomicSub(a.refs + old, 1);
                    if (j == r.j0 && r.first % a.page != 0) copy = make_int2(old, id);
                }
            } else {
                atomicMin(&s.fail[q], (int)j);
            }
        }
        if (w == 0 && lane == 0) {
            a.copies[2 * b] = copy.x;
            a.copies[2 * b + 1] = copy.y;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += PG_THREADS) {
        const PageRange r = page_range(a, b0 + i, false);
        const int64_t end = min(r.end, (int64_t)s.fail[i] * a.page);
        a.granted[b0 + i] = max((int64_t)0, end - r.first);
        if (r.j0 == r.j1) a.copies[2 * (b0 + i)] = a.copies[2 * (b0 + i) + 1] = -1;
    }
}

struct CompactArgs {
    int32_t* refs;
    int64_t n_pages;
    int32_t* moves;                      // [n_pages / 2, 2]
    int64_t* n_used;
    int32_t* to;                         // [n_pages] where a page at or behind the used ones goes
    int64_t* cut;                        // the number of used pages, for the tables' kernel
    int32_t* table;                      // the tables, [entries]
    int64_t entries;
    bool inside;                         // this kernel sees to them, else one behind it
    unsigned* st;
};

// This thread's part of the places that tables hold, of `step` threads.
__device__ __forceinline__ uint32_t count_places(const int32_t* table, int64_t entries, int64_t n_pages, int64_t i, int64_t step) {
    const auto is = [&](int32_t t) { return (uint32_t)(t >= 0 && t < n_pages); };
    uint32_t n = 0;
    int64_t done = 0;
    if (((uintptr_t)table & 15u) == 0) {
        const int4* quads = reinterpret_cast<const int4*>(table);
        done = entries / 4 * 4;
#pragma unroll 4
        for (int64_t q = i; q < entries / 4; q += step) {
            const int4 t = quads[q];
            n += is(t.x) + is(t.y) + is(t.z) + is(t.w);
        }
    }
    for (int64_t e = done + i; e < entries; e += step) n += is(table[e]);
    return n;
}

// A table's entry after the moves.
__device__ __forceinline__ void remap(int32_t* entry, int64_t n_pages, int64_t cut, const int32_t* to, unsigned* st) {
    const int32_t t = *entry;
    if (t >= -1 && t < cut) return;
    const int32_t d = t >= 0 && t < n_pages ? __ldcg(to + t) : -2;
    if (d >= 0) *entry = d;
    else csa2_flag(st, CSA2_DEVBIT_RANGE);           // a page that is none, or one without uses
}

__global__ void __launch_bounds__(PG_THREADS) pages_compact_kernel(const CompactArgs a) {
    __shared__ uint32_t tmp[PG_WARPS + 1], used[PG_CTAS], spare[PG_CTAS], from[PG_CTAS], into[PG_CTAS];
    const int nc = gridDim.x;
    const uint32_t rank = cta_rank();
    pdl_wait();
    pdl_trigger();
    cluster_sync();                      // every CTA runs: its shared memory may be written
    const int64_t share = ((a.n_pages + nc - 1) / nc + 3) / 4 * 4;
    const int64_t p0 = min(a.n_pages, rank * share), p1 = min(a.n_pages, p0 + share);
    const int64_t step = (int64_t)nc * PG_THREADS, half = a.n_pages / 2, i0 = (int64_t)rank * PG_THREADS + threadIdx.x;
    uint32_t n = 0, total, uses = 0, rest;
    for (int64_t p = p0 + threadIdx.x; p < p1; p += PG_THREADS) {
        const int32_t r = a.refs[p];
        n += r > 0;
        uses += (uint32_t)max(r, 0);
    }
    uses -= count_places(a.table, a.entries, a.n_pages, i0, step);
    block_scan(tmp, n, total);
    block_scan(tmp, uses, rest);
    if (threadIdx.x < nc) {
        put_remote(&used[rank], threadIdx.x, total);
        put_remote(&spare[rank], threadIdx.x, rest);
    }
    cluster_sync();
    int64_t cut = 0;
    uint32_t missing = 0;                // uses less places, modulo 2^32
    for (int i = 0; i < nc; ++i) {
        cut += used[i];
        missing += spare[i];
    }
    if (missing != 0) {
        // a table that holds pages is not among these: they would move away under it, so none does
        for (int64_t i = i0; i < half; i += step) a.moves[2 * i] = a.moves[2 * i + 1] = -1;
        if (rank == 0 && threadIdx.x == 0) {
            csa2_flag(a.st, CSA2_DEVBIT_RANGE);
            *a.cut = a.n_pages;
            if (a.n_used) *a.n_used = a.n_pages;
        }
        return;
    }
    // sources (used, at or behind the cut) and holes (free, before it) of this share
    uint32_t ns = 0, nh = 0, ts, th;
    for (int64_t p = p0 + threadIdx.x; p < p1; p += PG_THREADS) {
        const bool u = a.refs[p] > 0;
        ns += u && p >= cut;
        nh += !u && p < cut;
    }
    block_scan(tmp, ns, ts);
    block_scan(tmp, nh, th);
    if (threadIdx.x < nc) {
        put_remote(&from[rank], threadIdx.x, ts);
        put_remote(&into[rank], threadIdx.x, th);
    }
    cluster_sync();
    int64_t n_moves = 0;
    uint32_t s0 = 0, h0 = 0;
    for (int i = 0; i < nc; ++i) {
        if (i < (int)rank) {
            s0 += from[i];
            h0 += into[i];
        }
        n_moves += from[i];
    }
    for (int64_t q = p0; q < p1; q += 4 * PG_THREADS) {
        const int64_t p = q + 4 * (int64_t)threadIdx.x;
        bool src[4], hole[4];
        ns = nh = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = p + j < p1, u = in && a.refs[p + j] > 0;
            src[j] = u && p + j >= cut;
            hole[j] = in && !u && p + j < cut;
            ns += src[j];
            nh += hole[j];
            if (in && !u && p + j >= cut) a.to[p + j] = -1;
        }
        uint32_t s = s0 + block_scan(tmp, ns, ts), h = h0 + block_scan(tmp, nh, th);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (src[j]) a.moves[2 * (int64_t)s++] = (int32_t)(p + j);
            if (hole[j]) a.moves[2 * (int64_t)h++ + 1] = (int32_t)(p + j);
        }
        s0 += ts;
        h0 += th;
    }
    __threadfence();
    cluster_sync();
    for (int64_t i = i0; i < half; i += step) {
        if (i < n_moves) {
            const int32_t src = a.moves[2 * i], dst = a.moves[2 * i + 1];
            a.to[src] = dst;
            a.refs[dst] = a.refs[src];
            a.refs[src] = 0;
        } else {
            a.moves[2 * i] = a.moves[2 * i + 1] = -1;
        }
    }
    if (rank == 0 && threadIdx.x == 0) {
        *a.cut = cut;
        if (a.n_used) *a.n_used = cut;
    }
    if (!a.inside) return;
    __threadfence();
    cluster_sync();                      // every page's way is written
    for (int64_t i = i0; i < a.entries; i += step) remap(a.table + i, a.n_pages, cut, a.to, a.st);
}

__global__ void __launch_bounds__(256) pages_remap_kernel(int32_t* table, int64_t total, int64_t n_pages, const int32_t* to,
                                                          const int64_t* cut_p, unsigned* st) {
    pdl_wait();
    pdl_trigger();
    const int64_t cut = *cut_p;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x)
        remap(table + i, n_pages, cut, to, st);
}

constexpr int PC_THREADS = 256, PC_PIECES = 8;

// Whole pages in pieces of V: a block takes pairs_b pairs (pages of fewer than PC_BLOCK pieces) or PC_BLOCK
// pieces of one, eight in flight a thread.  The pairs that move nothing are the last ones of a compaction
// and cost their lookup.  Bound by device memory: 10,000 of 40,000 pages of 18 KB moved in 59 us, 6.3 TB/s
// read and written.
constexpr int PC_BLOCK = 4 * PC_THREADS * PC_PIECES, PC_PAIRS = 512;

template <typename V>
__global__ void __launch_bounds__(PC_THREADS) page_copy_kernel(V* pool, int64_t n_pages, int64_t pieces, const int32_t* pairs,
                                                               int64_t n, int pairs_b, int64_t chunks, unsigned* st) {
    __shared__ int64_t from[PC_PAIRS], to[PC_PAIRS];     // first pieces of the block's pages, -1 = nothing to move
    const int64_t groups = (n + pairs_b - 1) / pairs_b;
    pdl_wait();
    pdl_trigger();
    for (int64_t i = blockIdx.x; i < groups * chunks; i += gridDim.x) {
        const int64_t g = chunks == 1 ? i : i / chunks, p0 = g * pairs_b;
        const int np = (int)min((int64_t)pairs_b, n - p0);
        bool any = false;
        for (int p = threadIdx.x; p < np; p += PC_THREADS) {
            const int32_t src = pairs[2 * (p0 + p)], dst = pairs[2 * (p0 + p) + 1];
            bool move = src != -1 && dst != -1;
            if (move && (src < 0 || src >= n_pages || dst < 0 || dst >= n_pages)) {
                csa2_flag(st, CSA2_DEVBIT_RANGE);
                move = false;
            }
            from[p] = move ? src * pieces : -1;
            to[p] = dst * pieces;
            any |= move;
        }
        if (!__syncthreads_or(any)) continue;
        const int64_t c0 = (i - g * chunks) * PC_BLOCK;
        const uint32_t total = (uint32_t)min((int64_t)np * pieces - c0, (int64_t)PC_BLOCK);
        for (uint32_t u0 = threadIdx.x; u0 < total; u0 += PC_THREADS * PC_PIECES) {
            V v[PC_PIECES];
            int64_t d[PC_PIECES];
#pragma unroll
            for (int j = 0; j < PC_PIECES; ++j) {
                const uint32_t u = u0 + j * PC_THREADS, p = chunks == 1 ? u / (uint32_t)pieces : 0;
                d[j] = -1;
                if (u >= total || from[p] < 0) continue;
                const int64_t k = c0 + u - p * pieces;
                d[j] = to[p] + k;
                v[j] = __ldcs(pool + from[p] + k);
            }
#pragma unroll
            for (int j = 0; j < PC_PIECES; ++j)
                if (d[j] >= 0) __stcs(pool + d[j], v[j]);
        }
        __syncthreads();                         // the tables are filled again
    }
}

struct RowsArgs {
    int64_t n_pages;
    int P, page;
    const int32_t* table;
    const int64_t* first;                // write: entry first[b] + i, i < count[b]
    const int64_t* count;
    const int32_t* idx;                  // read: entry idx[b, i]
    int n;                               // rows of a sequence
    int64_t rows;
    uint32_t pieces, rows_b;
    unsigned* st;
};

// Rows between a dense block [B, n, row] and the pages, in pieces of V: a block takes rows_b rows,
// looks their places up into shared memory, then each thread has eight pieces in flight, adjacent
// threads adjacent pieces.  Bound by device memory: 99,948 rows of 1 KB read in 33 us, 6.2 TB/s read and
// written.
template <typename V, bool WRITE>
__global__ void __launch_bounds__(PC_THREADS) page_rows_kernel(V* pool, V* dense, const RowsArgs a) {
    __shared__ int64_t at[PC_THREADS * PC_PIECES];   // first piece of the row in the pool, -1 = none
    const int64_t r0 = (int64_t)blockIdx.x * a.rows_b;
    const uint32_t nr = (uint32_t)min((int64_t)a.rows_b, a.rows - r0), total = nr * a.pieces;
    pdl_wait();
    pdl_trigger();
    for (uint32_t r = threadIdx.x; r < nr; r += PC_THREADS) {
        const int64_t row = r0 + r, b = row / a.n;
        int64_t e = -1;
        bool want;
        if (WRITE) {
            const int64_t i = row - b * a.n, f = a.first[b];
            want = f >= 0 && i < a.count[b];
            e = f + i;
        } else {
            e = a.idx[row];
            want = e != -1;
        }
        int64_t place = -1;
        if (want) {
            const int64_t p = e >= 0 ? e / a.page : a.P;
            if (p < a.P) {
                const int32_t t = a.table[b * a.P + p];
                if (t >= 0 && t < a.n_pages) place = ((int64_t)t * a.page + (e - p * a.page)) * a.pieces;
            }
            if (place < 0) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
        }
        at[r] = place;
    }
    __syncthreads();
    V* d = dense + r0 * a.pieces;
    for (uint32_t u0 = threadIdx.x; u0 < total; u0 += PC_THREADS * PC_PIECES) {
        V v[PC_PIECES];
        int64_t f[PC_PIECES];
#pragma unroll
        for (int j = 0; j < PC_PIECES; ++j) {
            const uint32_t u = u0 + j * PC_THREADS, r = u / a.pieces;
            f[j] = u < total ? at[r] : -1;
            if (f[j] >= 0) {
                f[j] += u - r * a.pieces;
                v[j] = WRITE ? __ldcs(d + u) : __ldcs(pool + f[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < PC_PIECES; ++j)
            if (f[j] >= 0) {
                if (WRITE) __stcs(pool + f[j], v[j]);
                else __stcs(d + u0 + j * PC_THREADS, v[j]);
            }
    }
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

unsigned flat_grid(const csa2_ctx* ctx, int64_t total) {
    return (unsigned)std::min<int64_t>((total + 255) / 256, 8ll * std::max(1, ctx->num_sms));
}

// The state kernels' launch: one CTA for a small state, else the cluster.
void cluster_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, int64_t n_pages, int B, size_t smem, cudaStream_t s) {
    const unsigned nc = n_pages <= PG_SMALL_PAGES && B <= PG_SMALL_SEQS ? 1 : PG_CTAS;
    cfg = {};
    cfg.gridDim = dim3(nc);
    cfg.blockDim = dim3(PG_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = nc;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
}

// Arguments every call of the page state shares.
csa2_status state_ok(const csa2_ctx* ctx, const void* refs, int64_t n_pages, const void* table, int B, int P) {
    if (!ctx || n_pages < 0 || B < 0 || P < 0) return CSA2_ERR_INVALID_ARG;
    if (n_pages > 0x7FFFFFFF || B > 65535) return CSA2_ERR_UNSUPPORTED;
    if ((n_pages > 0 && !refs) || (B > 0 && P > 0 && !table) || !aligned(refs, 4) || !aligned(table, 4)) return CSA2_ERR_INVALID_ARG;
    return CSA2_OK;
}

csa2_status rows_call(csa2_ctx* ctx, bool write, void* pool, int64_t n_pages, int page, int64_t row_bytes, const int32_t* table,
                      int B, int P, void* dense, int n, const int64_t* first, const int64_t* count, const int32_t* idx,
                      void* stream) {
    if (!ctx || n_pages < 0 || B < 0 || P < 0 || n < 0 || page < 1 || page > 65536 || row_bytes < 4 || row_bytes > (1 << 20))
        return CSA2_ERR_INVALID_ARG;
    if (row_bytes % 4 || n_pages > 0x7FFFFFFF || n_pages * page >= (1ll << 40) || B > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B == 0 || n == 0) return CSA2_OK;
    if ((n_pages > 0 && !pool) || (P > 0 && !table) || !dense || (write ? !first || !count : !idx)) return CSA2_ERR_INVALID_ARG;
    if (!aligned(pool, 4) || !aligned(table, 4) || !aligned(dense, 4) || !aligned(first, 8) || !aligned(count, 8) || !aligned(idx, 4))
        return CSA2_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)B * n;
    if (overlap(pool, (size_t)n_pages * page * row_bytes, dense, (size_t)rows * row_bytes)) return CSA2_ERR_INVALID_ARG;
    const bool wide = row_bytes % 16 == 0 && aligned(pool, 16) && aligned(dense, 16);
    const int64_t pieces = row_bytes / (wide ? 16 : 4);
    const int64_t rows_b = std::min<int64_t>(PC_THREADS * PC_PIECES, std::max<int64_t>(1, PC_THREADS * PC_PIECES / pieces));
    const int64_t blocks = (rows + rows_b - 1) / rows_b;
    if (blocks > 0x7FFFFFFF) return CSA2_ERR_UNSUPPORTED;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    const RowsArgs a = {n_pages, P, page, table, first, count, idx, n, rows, (uint32_t)pieces, (uint32_t)rows_b, ctx->status};
    cudaStream_t s = as_stream(stream);
    const unsigned g = (unsigned)blocks;
    csa2_status r;
    if (wide) {
        uint4 *p = reinterpret_cast<uint4*>(pool), *d = reinterpret_cast<uint4*>(dense);
        r = launch_pdl(write ? page_rows_kernel<uint4, true> : page_rows_kernel<uint4, false>, dim3(g), dim3(PC_THREADS), 0, s, p, d, a);
    } else {
        uint32_t *p = reinterpret_cast<uint32_t*>(pool), *d = reinterpret_cast<uint32_t*>(dense);
        r = launch_pdl(write ? page_rows_kernel<uint32_t, true> : page_rows_kernel<uint32_t, false>, dim3(g), dim3(PC_THREADS), 0, s, p, d,
                       a);
    }
    return r != CSA2_OK ? r : csa2_launch_status();
}

int reserve_words(int P) { return P / 32 + 1; }      // a range of P pages at most, from any page on

}  // namespace

extern "C" csa2_status csa2_pages_fork(csa2_ctx* ctx, int32_t* refs, int64_t n_pages, const int32_t* table, int B, int max_pages,
                                       const int32_t* parent, int B_out, int32_t* table_out, void* stream) {
    const csa2_status r = state_ok(ctx, refs, n_pages, table, B, max_pages);
    if (r != CSA2_OK) return r;
    if (B_out < 0) return CSA2_ERR_INVALID_ARG;
    if (B_out > 65535) return CSA2_ERR_UNSUPPORTED;
    if (B_out == 0 || max_pages == 0) return CSA2_OK;
    if (!parent || !table_out || !aligned(parent, 4) || !aligned(table_out, 4)) return CSA2_ERR_INVALID_ARG;
    const int64_t total = (int64_t)B_out * max_pages;
    if (overlap(table, (size_t)B * max_pages * 4, table_out, (size_t)total * 4)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    const csa2_status l = launch_pdl(pages_fork_kernel, dim3(flat_grid(ctx, total)), dim3(256), 0, as_stream(stream), refs, n_pages, table,
                                     B, max_pages, parent, total, table_out, ctx->status);
    return l != CSA2_OK ? l : csa2_launch_status();
}

extern "C" csa2_status csa2_pages_free(csa2_ctx* ctx, int32_t* refs, int64_t n_pages, int32_t* table, int B, int max_pages,
                                       int page, const int64_t* keep, void* stream) {
    const csa2_status r = state_ok(ctx, refs, n_pages, table, B, max_pages);
    if (r != CSA2_OK) return r;
    if (page < 1 || page > 65536 || !aligned(keep, 8)) return CSA2_ERR_INVALID_ARG;
    const int64_t total = (int64_t)B * max_pages;
    if (total == 0) return CSA2_OK;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    const csa2_status l = launch_pdl(pages_free_kernel, dim3(flat_grid(ctx, total)), dim3(256), 0, as_stream(stream), refs, n_pages, table,
                                     max_pages, total, page, keep, ctx->status);
    return l != CSA2_OK ? l : csa2_launch_status();
}

extern "C" size_t csa2_pages_reserve_workspace_bytes(int64_t n_pages, int B, int max_pages) {
    if (n_pages < 0 || B <= 0 || max_pages < 0) return 0;
    return ((size_t)n_pages + 2 * (size_t)B * reserve_words(max_pages)) * 4;
}

extern "C" csa2_status csa2_pages_reserve(csa2_ctx* ctx, int32_t* refs, int64_t n_pages, int32_t* table, int B, int max_pages,
                                          int page, const int64_t* first, const int64_t* count, int64_t* granted,
                                          int32_t* copies, void* ws, size_t ws_bytes, void* stream) {
    const csa2_status r = state_ok(ctx, refs, n_pages, table, B, max_pages);
    if (r != CSA2_OK) return r;
    if (page < 1 || page > 65536) return CSA2_ERR_INVALID_ARG;
    if (B == 0) return CSA2_OK;
    if (!first || !count || !granted || !copies || !ws || ws_bytes < csa2_pages_reserve_workspace_bytes(n_pages, B, max_pages) ||
        !aligned(first, 8) || !aligned(count, 8) || !aligned(granted, 8) || !aligned(copies, 4) || !aligned(ws, 16))
        return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    ReserveArgs a = {refs, n_pages, table, B, max_pages, page, first, count, granted, copies,
                     reinterpret_cast<int32_t*>(ws), nullptr, nullptr, reserve_words(max_pages), ctx->status};
    a.want = reinterpret_cast<uint32_t*>(ws) + n_pages;
    a.base = a.want + (size_t)B * a.W;
    CSA2_CHECK_CUDA(cudaFuncSetAttribute(pages_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ReserveSmem)));
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    cluster_config(cfg, at, n_pages, B, sizeof(ReserveSmem), as_stream(stream));
    if (cudaLaunchKernelEx(&cfg, pages_reserve_kernel, a) != cudaSuccess) return CSA2_ERR_CUDA;
    return csa2_launch_status();
}

extern "C" size_t csa2_pages_compact_workspace_bytes(int64_t n_pages) {
    return n_pages > 0 ? (size_t)n_pages * 4 + 16 : 0;
}

extern "C" csa2_status csa2_pages_compact(csa2_ctx* ctx, int32_t* refs, int64_t n_pages, int32_t* table, int B, int max_pages,
                                          int32_t* moves, int64_t* n_used, void* ws, size_t ws_bytes, void* stream) {
    const csa2_status r = state_ok(ctx, refs, n_pages, table, B, max_pages);
    if (r != CSA2_OK) return r;
    if (!aligned(n_used, 8)) return CSA2_ERR_INVALID_ARG;
    if (n_pages == 0) {
        DeviceGuard dev(ctx);
        if (!dev.ok) return CSA2_ERR_CUDA;
        if (n_used) CSA2_CHECK_CUDA(cudaMemsetAsync(n_used, 0, 8, as_stream(stream)));
        return CSA2_OK;
    }
    if ((n_pages > 1 && !moves) || !ws || ws_bytes < csa2_pages_compact_workspace_bytes(n_pages) || !aligned(moves, 4) ||
        !aligned(ws, 16))
        return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    int64_t* cut = reinterpret_cast<int64_t*>(ws);
    int32_t* to = reinterpret_cast<int32_t*>(ws) + 4;
    const int64_t total = (int64_t)B * max_pages;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    cluster_config(cfg, at, n_pages, 0, 0, s);
    // a small table is seen to by the same kernel (a launch less: 300 pages and two pools 47 us a step, not 51)
    const bool inside = total <= 4ll * cfg.gridDim.x * PG_THREADS;
    const CompactArgs a = {refs, n_pages, moves, n_used, to, cut, table, total, inside, ctx->status};
    if (cudaLaunchKernelEx(&cfg, pages_compact_kernel, a) != cudaSuccess) return CSA2_ERR_CUDA;
    if (inside) return csa2_launch_status();
    const csa2_status l = launch_pdl(pages_remap_kernel, dim3(flat_grid(ctx, total)), dim3(256), 0, s, table, total, n_pages,
                                     (const int32_t*)to, (const int64_t*)cut, ctx->status);
    return l != CSA2_OK ? l : csa2_launch_status();
}

extern "C" csa2_status csa2_page_copy(csa2_ctx* ctx, void* pool, int64_t n_pages, int64_t page_bytes, const int32_t* pairs,
                                      int64_t n, void* stream) {
    if (!ctx || n_pages < 0 || n < 0 || page_bytes < 4 || page_bytes > (1ll << 36)) return CSA2_ERR_INVALID_ARG;
    if (page_bytes % 4 || n_pages > 0x7FFFFFFF || n > 0x7FFFFFFF) return CSA2_ERR_UNSUPPORTED;
    if (n == 0 || n_pages == 0) return CSA2_OK;
    if (!pool || !pairs || !aligned(pool, 4) || !aligned(pairs, 4)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    const bool wide = page_bytes % 16 == 0 && aligned(pool, 16);
    const int64_t pieces = page_bytes / (wide ? 16 : 4), chunks = (pieces + PC_BLOCK - 1) / PC_BLOCK;
    // few pairs: a block each, so that they move at once
    const int64_t fit = std::min<int64_t>(PC_PAIRS, std::max<int64_t>(1, PC_BLOCK / pieces));
    const int pairs_b = (int)std::max<int64_t>(1, std::min(fit, n / (4 * std::max(1, ctx->num_sms))));
    const unsigned grid = (unsigned)std::min<int64_t>((n + pairs_b - 1) / pairs_b * chunks, 8ll * std::max(1, ctx->num_sms));
    cudaStream_t s = as_stream(stream);
    const csa2_status l = wide ? launch_pdl(page_copy_kernel<uint4>, dim3(grid), dim3(PC_THREADS), 0, s, reinterpret_cast<uint4*>(pool),
                                            n_pages, pieces, pairs, n, pairs_b, chunks, ctx->status)
                               : launch_pdl(page_copy_kernel<uint32_t>, dim3(grid), dim3(PC_THREADS), 0, s,
                                            reinterpret_cast<uint32_t*>(pool), n_pages, pieces, pairs, n, pairs_b, chunks, ctx->status);
    return l != CSA2_OK ? l : csa2_launch_status();
}

extern "C" csa2_status csa2_page_write(csa2_ctx* ctx, void* pool, int64_t n_pages, int page, int64_t row_bytes,
                                       const int32_t* table, int B, int max_pages, const void* rows, int n, const int64_t* first,
                                       const int64_t* count, void* stream) {
    return rows_call(ctx, true, pool, n_pages, page, row_bytes, table, B, max_pages, const_cast<void*>(rows), n, first, count,
                     nullptr, stream);
}

extern "C" csa2_status csa2_page_read(csa2_ctx* ctx, const void* pool, int64_t n_pages, int page, int64_t row_bytes,
                                      const int32_t* table, int B, int max_pages, const int32_t* idx, int keep, void* dst,
                                      void* stream) {
    return rows_call(ctx, false, const_cast<void*>(pool), n_pages, page, row_bytes, table, B, max_pages, dst, keep, nullptr, nullptr,
                     idx, stream);
}
