// Backward pass of the shared-KV MQA (csa2_sparse_attn_bwd, csa2_dense_attn_bwd).
//
// With qn = RMS(q), q^ = RoPE_t(qn), k^_j = r_j x_j (r_j the row's RMS factor) and the
// forward's lse, per query and head:
//     p_j  = exp(q^.k^_j / sqrt(c) - lse)             (recomputed, nothing else is kept)
//     do'  = RoPE_t(dout),  D = dout . out
//     dS_j = p_j (do'.k^_j - D) / sqrt(c)
//     dq^  = sum_j dS_j k^_j,   dq = rq (RoPE_-t dq^ - qn mean(qn . RoPE_-t dq^))
//     row gradient: G_j = r_j sum over queries and heads of (dS_j q^ + p_j do'),
//     dx_j = G_j - k^_j mean(k^_j . G_j)
//     dsink = - sum over queries of exp(sink - lse) D
// The row gradients are a scatter: every (query, slot) adds 512 values to its row.  They
// are summed without atomics, in query order, so a call's results are the same bits every
// time: a plan gives every (query, slot) its place in a list sorted by row and query (a
// counting sort over groups of queries), the main kernels write each contribution there,
// and one pass sums every row's stretch of the list, applies the row's norm and stores.
//
// Queries run in chunks of as many as the workspace holds; with more than one chunk the
// rows' sums are carried in fp32 in the workspace.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attn_bwd_tc.cuh"
#include "attn_grad.cuh"

namespace {

constexpr int MAX_GROUPS = 304;          // query groups of the scatter plan: a block of 1,024 threads each,
                                         // two on an SM
constexpr int64_t MAX_COUNTERS = 1 << 24;

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ---------------------------------------------------------------- scatter plan

// rank[q][s] = how many (query, slot) pairs of the group before this one (in query order)
// lie in the same row.  A block walks its group's queries in order: the barrier between
// two queries orders their counter updates (an atomic's round trip a query, so many groups: 30 us
// for 2,048 queries, 71 us for 8,192).  Slots of one query in the same row (the same
// index twice) hold the same contribution, so their order does not matter.
__global__ void __launch_bounds__(1024, 2) bwd_rank_kernel(SlotArgs a, int64_t bq0, int nb, int group_q, int n_slots,
                                                          int64_t rows, uint32_t* cnt, int32_t* rank) {
    const int g = blockIdx.x, t = threadIdx.x;
    uint32_t* c = cnt + (int64_t)g * rows;
    const int q0 = g * group_q, q1 = min(nb, q0 + group_q);
    // the first 1,024 slots' rows of the next query are looked up while this one counts
    int64_t next = q0 < q1 && t < n_slots ? slot_row(a, bq0 + q0, t, true) : -1;
    for (int q = q0; q < q1; ++q) {
        int64_t row = next;
        if (q + 1 < q1 && t < n_slots) next = slot_row(a, bq0 + q + 1, t, true);
        for (int s = t; s < n_slots; s += 1024) {
            if (s != t) row = slot_row(a, bq0 + q, s, true);
            rank[(int64_t)q * n_slots + s] = row >= 0 ? (int32_t)atomicAdd(&c[row], 1u) : -1;
        }
        __syncthreads();
    }
}

// Block-wide exclusive scan of one value per thread; returns the prefix, total in *tot.
__device__ __forceinline__ uint32_t block_excl_scan(uint32_t v, uint32_t* warp_tot, uint32_t* tot) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_tot[w] = incl;
    __syncthreads();
    if (w == 0) {
        uint32_t t = lane < nw ? warp_tot[lane] : 0u, ti = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, ti, o);
            if (lane >= o) ti += u;
        }
        warp_tot[lane] = ti - t;
        if (lane == 31) *tot = ti;
    }
    __syncthreads();
    return warp_tot[w] + incl - v;
}

// Counts -> places: base[g][row] (in place of cnt) = first place of group g's stretch of
// the row, relative to the row's block of BWD_SCAN_ROWS rows; loc / tot: the row's own start
// (relative) and length; blk[b] = the block's length (scanned by bwd_scan_kernel).  Small
// blocks: the walk over the groups is a chain of strided loads, so it wants many of them.
__global__ void __launch_bounds__(BWD_SCAN_ROWS) bwd_place_kernel(uint32_t* cnt, int groups, int64_t rows,
                                                                  uint32_t* loc, uint32_t* tot, uint32_t* blk) {
    __shared__ uint32_t wt[32], total;
    const int64_t row = (int64_t)blockIdx.x * BWD_SCAN_ROWS + threadIdx.x;
    uint32_t n = 0;
    if (row < rows) {
#pragma unroll 16
        for (int g = 0; g < groups; ++g) n += cnt[(int64_t)g * rows + row];
    }
    const uint32_t start = block_excl_scan(n, wt, &total);
    if (row < rows) {
        uint32_t at = start;
        int g = 0;
        for (; g + 16 <= groups; g += 16) {
            uint32_t here[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) here[i] = cnt[(int64_t)(g + i) * rows + row];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                cnt[(int64_t)(g + i) * rows + row] = at;
                at += here[i];
            }
        }
        for (; g < groups; ++g) {
            const uint32_t here = cnt[(int64_t)g * rows + row];
            cnt[(int64_t)g * rows + row] = at;
            at += here;
        }
        loc[row] = start;
        tot[row] = n;
    }
    if (threadIdx.x == 0) blk[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) bwd_scan_kernel(uint32_t* blk, int64_t n) {
    __shared__ uint32_t wt[32], total;
    uint32_t carry = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t v = i < n ? blk[i] : 0u;
        const uint32_t p = block_excl_scan(v, wt, &total);
        if (i < n) blk[i] = carry + p;
        carry += total;
        __syncthreads();
    }
}

__device__ __forceinline__ int64_t pair_place(const BwdChunk& c, int q, int slot, int64_t row) {
    const int32_t r = c.rank[(int64_t)q * c.n_slots + slot];
    return (int64_t)c.blk[row / BWD_SCAN_ROWS] + c.base[(int64_t)(q / c.group_q) * c.rows + row] + r;
}

// ---------------------------------------------------------------- preparation

// RMS factor of every row (cache rows, then window rows); a warp per row.
__global__ void __launch_bounds__(256) bwd_rinv_kernel(const void* kv, int kv_dt, int64_t n_kv, const void* swa,
                                                       int swa_dt, int64_t rows, unsigned flags, float* rinv) {
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    float r = 1.0f;
    if (flags & CSA2_KVNORM) {
        float v[16];
        if (row < n_kv)
            ag_load_row16(kv, kv_dt, row, lane, v);
        else
            ag_load_row16(swa, swa_dt, row - n_kv, lane, v);
        r = ag_rms_factor(warp_sum(ag_sumsq16(v)));
    }
    if (lane == 0) rinv[row] = r;
}

// dsink[h] = - sum over queries of exp(sink_h - lse) D, added in a fixed order: block (x, y)
// sums stretch y of the queries for the heads 32 x .. (a lane a head, a warp every eighth query,
// then the warps), and the stretches' sums go to `part` [y][H], or to dsink if there is only one.
__global__ void __launch_bounds__(256) bwd_sink_kernel(const float* sink, const float* lse, const float* D, int64_t n_bq,
                                                       int H, int64_t per, float* part) {
    __shared__ float red[8][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.x * 32 + lane;
    const int64_t i1 = min(n_bq, ((int64_t)blockIdx.y + 1) * per);
    const float zs = sink && h < H ? sink[h] : -INFINITY;
    float s = 0.0f;
    if (zs != -INFINITY) {
#pragma unroll 4
        for (int64_t i = blockIdx.y * per + w; i < i1; i += 8) {
            const float l = lse[i * H + h];
            if (l != -INFINITY) s = fmaf(-expf(zs - l), D[i * H + h], s);
        }
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && h < H) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += red[i][lane];
        part[(int64_t)blockIdx.y * H + h] = s;
    }
}

__global__ void __launch_bounds__(128) bwd_sink_sum_kernel(const float* part, int n, int H, float* dsink) {
    const int h = threadIdx.x;
    if (h >= H) return;
    float s = 0.0f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) s += part[(int64_t)i * H + h];
    dsink[h] = s;
}

// q^ and do' of every (query, head) of the chunk in fp32 and D = dout . out (CUDA-core path); a
// warp per row.
template <typename TQ, typename TO>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const TQ* q, const TO* dout, const TO* out, const int64_t* q_pos,
                                                       int64_t bq0, int64_t n_rows, int H, AgRope rope,
                                                       unsigned flags, float* qh, float* dh, float* D) {
    __shared__ float cs[8][32], sn[8][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + w;
    if (r >= n_rows) return;
    ag_cos_sin(rope, q_pos[bq0 + r / H], lane, cs[w][lane], sn[w][lane]);
    __syncwarp();
    const int64_t src = (bq0 * H + r) * AG_C + 16 * lane, dst = r * AG_C + 16 * lane;
    float v[16];
    ag_load16<TQ>(q + src, v);
    if (flags & CSA2_QNORM) {
        const float f = ag_rms_factor(warp_sum(ag_sumsq16(v)));
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= f;
    }
    if (flags & CSA2_ROPE) ag_rope16(v, lane, cs[w], sn[w], 1.0f);
    ag_store16<float>(qh + dst, v);
    ag_load16<TO>(dout + src, v);
    float o[16], dot = 0.0f;
    ag_load16<TO>(out + src, o);
#pragma unroll
    for (int i = 0; i < 16; ++i) dot = fmaf(v[i], o[i], dot);
    dot = warp_sum(dot);
    if (lane == 0) D[bq0 * H + r] = dot;
    if (flags & CSA2_ROPE) ag_rope16(v, lane, cs[w], sn[w], 1.0f);
    ag_store16<float>(dh + dst, v);
}

// ---------------------------------------------------------------- CUDA-core path (fp32)

constexpr int SB_HG = 16;                // heads per CTA of the query pass
constexpr int SB_KC = 32;                // key rows per staged chunk

// dq of one head row by a warp, lane l holding channels l + 32 i: dq^ back through RoPE and the
// query's RMSNorm (on q^ and dq^: a rotation keeps their product).  A query that attends to
// nothing has no gradient, whatever its values.
template <typename TQ>
__device__ __forceinline__ void finish_dq(const BwdChunk& c, int64_t bq, int h, int lane, const float (&qv)[16],
                                          float (&acc)[16], const float* cs, const float* sn, TQ* dq) {
    const int64_t o = (bq * c.H + h) * AG_C;
    const TQ* qraw = reinterpret_cast<const TQ*>(c.q) + o;
    if (c.flags & CSA2_QNORM) {
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = to_f32<TQ>(qraw[lane + 32 * i]);
            ss = fmaf(x, x, ss);
            dot = fmaf(qv[i], acc[i], dot);
        }
        const float f = ag_rms_factor(warp_sum(ss));
        dot = warp_sum(dot) / (float)AG_C;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = f * (acc[i] - qv[i] * dot);
    }
    if (c.flags & CSA2_ROPE) rope_lanes(acc, lane, cs, sn, -1.0f);
    const bool none = c.lse[bq * c.H + h] == -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) dq[o + lane + 32 * i] = from_f32<TQ>(none ? 0.0f : acc[i]);
}

// Query pass: p and dS of every slot (kept for the row pass) and dq; a CTA per (16 heads,
// query, range of slots), a warp per two heads, key rows staged 32 at a time in fp32.  With few
// queries the slots are split over CTAs (p needs no other slot, the lse is given) and
// bwd_simt_dq_kernel adds the ranges' dq^.  Bound by shared memory's port, which the loads of a
// row (32 a warp, shared by its two heads) and the sums' shuffles go through: 20 cycles a (head,
// slot) against 12 of the FMAs; with one head a warp and a sum of its own for each row it was 42.
template <typename TQ>
__global__ void __launch_bounds__(256, 1) bwd_simt_q_kernel(BwdChunk c, const float* qh, const float* dh, float2* pds,
                                                            float* dqh, int per, TQ* dq) {
    extern __shared__ float smem[];
    float* xs = smem;                                        // [32][512] normalised rows
    int* ok = reinterpret_cast<int*>(xs + SB_KC * AG_C);     // [32]
    float* cs = reinterpret_cast<float*>(ok + SB_KC);        // [32]
    float* sn = cs + 32;
    const int q = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h0 = blockIdx.x * SB_HG + 2 * w;
    const int64_t bq = c.bq0 + q;
    if (threadIdx.x < 32) ag_cos_sin(c.rope, c.slots.q_pos[bq], lane, cs[lane], sn[lane]);
    float qv[2][16], dv[2][16], acc[2][16], lse[2], D[2];
    const int64_t hr = (int64_t)q * c.H + h0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const bool live = h0 + e < c.H;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            qv[e][i] = live ? qh[(hr + e) * AG_C + lane + 32 * i] : 0.0f;
            dv[e][i] = live ? dh[(hr + e) * AG_C + lane + 32 * i] : 0.0f;
            acc[e][i] = 0.0f;
        }
        lse[e] = live ? c.lse[bq * c.H + h0 + e] : -INFINITY;
        D[e] = live ? c.D[bq * c.H + h0 + e] : 0.0f;
    }
    const float isc = 1.0f / sqrtf((float)AG_C);
    const int s_end = min(c.n_slots, ((int)blockIdx.z + 1) * per);
    for (int s0 = blockIdx.z * per; s0 < s_end; s0 += SB_KC) {
        __syncthreads();
        {
            // rows w, w + 8, w + 16, w + 24 of the chunk: all looked up, then all loaded
            int64_t mine = -1;
            float fm = 0.0f;
            const int sr = s0 + w + 8 * lane;
            if (lane < SB_KC / 8 && sr < c.n_slots) mine = slot_row(c.slots, bq, sr, false);
            if (mine >= 0) fm = c.rinv[mine];
            float v[SB_KC / 8][16];
#pragma unroll
            for (int j = 0; j < SB_KC / 8; ++j) {
                const int64_t row = __shfl_sync(0xffffffffu, mine, j);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[j][i] = 0.0f;
                if (row >= 0) {
                    if (row < c.slots.n_kv)
                        ag_load_row16(c.kv, c.kv_dt, row, lane, v[j]);
                    else
                        ag_load_row16(c.swa, c.swa_dt, row - c.slots.n_kv, lane, v[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < SB_KC / 8; ++j) {
                const float f = __shfl_sync(0xffffffffu, fm, j);
                const bool there = __shfl_sync(0xffffffffu, mine, j) >= 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[j][i] *= f;
                ag_store16<float>(xs + (w + 8 * j) * AG_C + 16 * lane, v[j]);
                if (lane == 0) ok[w + 8 * j] = there;
            }
        }
        __syncthreads();
        if (h0 >= c.H) continue;
        float z[2] = {0.0f, 0.0f}, dp[2] = {0.0f, 0.0f};
#pragma unroll 1
        for (int j0 = 0; j0 < SB_KC; j0 += 8) {
            float a[2][8], b[2][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) a[e][j] = b[e][j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = xs[(j0 + j) * AG_C + lane + 32 * i];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[e][j] = fmaf(qv[e][i], x, a[e][j]);
                        b[e][j] = fmaf(dv[e][i], x, b[e][j]);
                    }
                }
            }
            const bool mine = (lane & 24) == j0;             // slots j0 .. j0 + 7 belong to these lanes
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float sa = ag_sums_of_8(a[e], lane), sb = ag_sums_of_8(b[e], lane);
                if (mine) {
                    z[e] = sa * isc;
                    dp[e] = sb;
                }
            }
        }
        float ds[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float p = 0.0f;
            ds[e] = 0.0f;
            if (ok[lane] && lse[e] != -INFINITY) {
                p = expf(z[e] - lse[e]);
                ds[e] = p * (dp[e] - D[e]) * isc;
            }
            if (h0 + e < c.H && s0 + lane < c.n_slots) pds[(hr + e) * c.n_slots + s0 + lane] = make_float2(p, ds[e]);
        }
#pragma unroll 4
        for (int j = 0; j < SB_KC; ++j) {
            const float d0 = __shfl_sync(0xffffffffu, ds[0], j), d1 = __shfl_sync(0xffffffffu, ds[1], j);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = xs[j * AG_C + lane + 32 * i];
                acc[0][i] = fmaf(d0, x, acc[0][i]);
                acc[1][i] = fmaf(d1, x, acc[1][i]);
            }
        }
    }
    __syncthreads();                                         // (cs, sn; every warp is past its rows)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (h0 + e >= c.H) break;
        if (gridDim.z == 1) {
            finish_dq<TQ>(c, bq, h0 + e, lane, qv[e], acc[e], cs, sn, dq);
            continue;
        }
        float* o = dqh + ((hr + e) * gridDim.z + blockIdx.z) * AG_C;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[lane + 32 * i] = acc[e][i];
    }
}

// dq from the slot ranges' dq^; a warp per (query, head).
template <typename TQ>
__global__ void __launch_bounds__(256) bwd_simt_dq_kernel(BwdChunk c, const float* qh, const float* dqh, int n_split, TQ* dq) {
    __shared__ float cs[8][32], sn[8][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t hr = (int64_t)blockIdx.x * 8 + w;
    if (hr >= (int64_t)c.nb * c.H) return;
    const int64_t bq = c.bq0 + hr / c.H;
    ag_cos_sin(c.rope, c.slots.q_pos[bq], lane, cs[w][lane], sn[w][lane]);
    __syncwarp();
    float qv[16], acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        qv[i] = qh[hr * AG_C + lane + 32 * i];
        acc[i] = 0.0f;
    }
#pragma unroll 4
    for (int k = 0; k < n_split; ++k)                 // unrolled: 64 loads in flight, not 16
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] += dqh[(hr * n_split + k) * AG_C + lane + 32 * i];
    finish_dq<TQ>(c, bq, (int)(hr % c.H), lane, qv, acc, cs[w], sn[w], dq);
}

// Row pass: the contribution r_j sum_h (dS_hj q^_h + p_hj do'_h) of every (query, slot);
// a CTA per (32 slots, query), two channels a thread.
__global__ void __launch_bounds__(256) bwd_simt_row_kernel(BwdChunk c, const float* qh, const float* dh,
                                                           const float2* pds) {
    __shared__ __align__(16) float2 sp[32][34];       // (rows of whole float4)
    __shared__ int64_t at[32];                        // places, -1 = no contribution
    __shared__ float fac[32];
    const int q = blockIdx.y, s0 = blockIdx.x * 32, t = threadIdx.x;
    const int64_t bq = c.bq0 + q;
    if (t < 32) {
        const int64_t row = s0 + t < c.n_slots ? slot_row(c.slots, bq, s0 + t, false) : -1;
        at[t] = row >= 0 ? pair_place(c, q, s0 + t, row) : -1;
        fac[t] = row >= 0 ? c.rinv[row] : 0.0f;
    }
    __syncthreads();
    float acc0[32], acc1[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) acc0[j] = acc1[j] = 0.0f;
    for (int h0 = 0; h0 < c.H; h0 += 32) {
        __syncthreads();
        for (int i = t; i < 32 * 32; i += 256) {
            const int h = h0 + (i >> 5), s = s0 + (i & 31);
            sp[i >> 5][i & 31] = h < c.H && s < c.n_slots ? pds[((int64_t)q * c.H + h) * c.n_slots + s] : make_float2(0.0f, 0.0f);
        }
        __syncthreads();
        const int hn = min(32, c.H - h0);
        // four heads' values are loaded during the four before (a head past the end: the last one's
        // again, times weights of 0)
        const int64_t o = ((int64_t)q * c.H + h0) * AG_C + 2 * t;
        float2 qn[4], dn[4];
        auto load = [&](int h) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = o + (int64_t)min(h + e, hn - 1) * AG_C;
                qn[e] = *reinterpret_cast<const float2*>(qh + at);
                dn[e] = *reinterpret_cast<const float2*>(dh + at);
            }
        };
        load(0);
        for (int h = 0; h < hn; h += 4) {
            float2 qv[4], dv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                qv[e] = qn[e];
                dv[e] = dn[e];
            }
            if (h + 4 < hn) load(h + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float4 pd = *reinterpret_cast<const float4*>(&sp[h + e][j]);
                    acc0[j] = fmaf(pd.y, qv[e].x, fmaf(pd.x, dv[e].x, acc0[j]));
                    acc1[j] = fmaf(pd.y, qv[e].y, fmaf(pd.x, dv[e].y, acc1[j]));
                    acc0[j + 1] = fmaf(pd.w, qv[e].x, fmaf(pd.z, dv[e].x, acc0[j + 1]));
                    acc1[j + 1] = fmaf(pd.w, qv[e].y, fmaf(pd.z, dv[e].y, acc1[j + 1]));
                }
        }
    }
    float2* part = reinterpret_cast<float2*>(c.part);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (at[j] < 0) continue;
        part[at[j] * (AG_C / 2) + t] = make_float2(acc0[j] * fac[j], acc1[j] * fac[j]);
    }
}

// ---------------------------------------------------------------- row sums

template <typename TP>
__device__ __forceinline__ float4 part4(const TP* p);
template <>
__device__ __forceinline__ float4 part4<float>(const float* p) {
    return __ldcs(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 part4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

__device__ __forceinline__ void store4(void* base, int dt, int64_t off, float4 v) {
    if (dt == CSA2_F32) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + off) = v;
    } else {
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(base) + off) =
            make_uint2(ag_pack_bf16x2(v.x, v.y), ag_pack_bf16x2(v.z, v.w));
    }
}

__device__ __forceinline__ float4 load4_any(const void* base, int dt, int64_t off) {
    if (dt == CSA2_F32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + off);
    const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(base) + off);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

struct RowSumArgs {
    const void* part;
    int passes;               // entries per place (head passes of the tensor-core path)
    const uint32_t *loc, *tot, *blk;
    int64_t rows, n_kv;
    const void *kv, *swa;
    int kv_dt, swa_dt;
    const float* rinv;
    unsigned flags;
    float* acc;               // [rows, 512] sums carried between chunks, or NULL (one chunk)
    int first, last;
    void *dkv, *dswa;         // NULL: not wanted
};

// Sum of a row's contributions in list order, then (last chunk) the row's norm; a CTA of
// 128 threads per row, four channels a thread.  Bound by device memory: the list of 2,048
// queries of 640 slots is 1.34 GB in bf16, 194 us.
template <typename TP>
__global__ void __launch_bounds__(128) bwd_rowsum_kernel(RowSumArgs a) {
    __shared__ float red[4];
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x, ch = 4 * t;
    void* dst = row < a.n_kv ? a.dkv : a.dswa;
    if (!dst) return;
    float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.acc && !a.first) g = *reinterpret_cast<const float4*>(a.acc + row * AG_C + ch);
    const int64_t n = (int64_t)a.tot[row] * a.passes;
    if (n > 0) {
        const TP* p = reinterpret_cast<const TP*>(a.part) +
                      ((int64_t)a.blk[row / BWD_SCAN_ROWS] + a.loc[row]) * a.passes * AG_C + ch;
        int64_t i = 0;
        for (; i + 8 <= n; i += 8) {
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = part4<TP>(p + (i + j) * AG_C);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g.x += v[j].x;
                g.y += v[j].y;
                g.z += v[j].z;
                g.w += v[j].w;
            }
        }
        for (; i < n; ++i) {
            const float4 v = part4<TP>(p + i * AG_C);
            g.x += v.x;
            g.y += v.y;
            g.z += v.z;
            g.w += v.w;
        }
    }
    if (!a.last) {
        *reinterpret_cast<float4*>(a.acc + row * AG_C + ch) = g;
        return;
    }
    const int64_t off = (row < a.n_kv ? row : row - a.n_kv) * AG_C + ch;
    const int dt = row < a.n_kv ? a.kv_dt : a.swa_dt;
    // A row without contributions has no gradient, whatever its values (one that no slot points to may
    // hold anything).  Of the chunks before, only the sum is known: 0 if there was none, and where the
    // contributions cancel to 0 the norm makes 0 of it as well.
    const bool any = n > 0 || (a.acc && __syncthreads_or(g.x != 0.0f || g.y != 0.0f || g.z != 0.0f || g.w != 0.0f));
    if ((a.flags & CSA2_KVNORM) && any) {
        const float f = a.rinv[row];
        const float4 x = load4_any(row < a.n_kv ? a.kv : a.swa, dt, off);
        const float4 k = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
        float d = warp_sum(fmaf(k.x, g.x, fmaf(k.y, g.y, fmaf(k.z, g.z, k.w * g.w))));
        if ((t & 31) == 0) red[t >> 5] = d;
        __syncthreads();
        d = (red[0] + red[1] + red[2] + red[3]) / (float)AG_C;
        g.x = fmaf(-k.x, d, g.x);
        g.y = fmaf(-k.y, d, g.y);
        g.z = fmaf(-k.z, d, g.z);
        g.w = fmaf(-k.w, d, g.w);
    }
    store4(dst, dt, off, g);
}

constexpr size_t SB_SMEM = (size_t)SB_KC * AG_C * 4 + SB_KC * 4 + 64 * 4;

// Raises a kernel's dynamic shared memory once per device (bit `device` of `done`).
template <typename K>
csa2_status raise_smem(K kern, size_t bytes, int device, std::atomic<uint64_t>& done) {
    const uint64_t bit = 1ull << (device & 63);
    if (done.load(std::memory_order_relaxed) & bit) return CSA2_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return CSA2_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_relaxed);
    return CSA2_OK;
}

// ---------------------------------------------------------------- workspace

struct BwdSizes {
    int64_t n_bq;
    int H, n_slots;
    int64_t rows;             // cache and window rows
    bool tc;                  // tensor-core path
    int num_sms;
};

struct BwdLayout {
    size_t D, sink, rinv, cnt, loc, tot, blk, rank, qh, dh, pds, img, slots, dqh, part, acc, total;
    int groups, group_q, n_pass;
    int n_split, tps;         // CUDA cores: slot ranges of a query, slots of one
};

// Stretches of queries that dsink is summed in: 32 queries are four a warp.
int64_t sink_stretches(int64_t n_bq) { return std::max<int64_t>(1, std::min<int64_t>(64, n_bq / 32)); }

// Slot ranges (of `per` slots) of the CUDA-core query pass: with few (query, 16 heads) groups, as
// many as give every SM two CTAs.
void simt_splits(int num_sms, int64_t groups, int n_slots, int* n_split, int* per) {
    const int chunks = std::max(1, (n_slots + SB_KC - 1) / SB_KC);
    const int want = (int)std::min<int64_t>(chunks, std::max<int64_t>(1, 2LL * num_sms / std::max<int64_t>(1, groups)));
    const int cps = (chunks + want - 1) / want;
    *per = cps * SB_KC;
    *n_split = (chunks + cps - 1) / cps;
}

// Workspace of chunks of nb queries.
BwdLayout bwd_layout(const BwdSizes& z, int64_t nb) {
    BwdLayout L;
    // counting walks a group's queries one by one (about 1 us each), placing walks the groups 16
    // at a time: the two walks are about as long with sqrt(16 nb) groups
    const int64_t even = (int64_t)std::ceil(std::sqrt(16.0 * (double)nb));
    const int64_t g = std::min<int64_t>({nb, even, MAX_GROUPS, std::max<int64_t>(1, MAX_COUNTERS / std::max<int64_t>(1, z.rows))});
    L.group_q = (int)((nb + g - 1) / g);
    L.groups = (int)((nb + L.group_q - 1) / L.group_q);
    L.n_pass = z.tc ? (z.H + 63) / 64 : 1;
    L.n_split = L.tps = 0;
    if (!z.tc)
        simt_splits(z.num_sms, nb * ((z.H + SB_HG - 1) / SB_HG), z.n_slots, &L.n_split, &L.tps);
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at = align_up(at + bytes, 256);
        return o;
    };
    const size_t row_f32 = (size_t)AG_C * 4, heads = (size_t)nb * z.H, pairs = (size_t)nb * z.n_slots;
    L.D = take((size_t)z.n_bq * z.H * 4);
    L.sink = take((size_t)sink_stretches(z.n_bq) * z.H * 4);
    L.rinv = take((size_t)z.rows * 4);
    L.cnt = take((size_t)L.groups * z.rows * 4);
    L.loc = take((size_t)z.rows * 4);
    L.tot = take((size_t)z.rows * 4);
    L.blk = take((size_t)((z.rows + BWD_SCAN_ROWS - 1) / BWD_SCAN_ROWS) * 4);
    L.rank = take(pairs * 4);
    L.qh = take(z.tc ? 0 : heads * row_f32);
    L.dh = take(z.tc ? 0 : heads * row_f32);
    L.pds = take(z.tc ? 0 : heads * z.n_slots * 8);
    L.img = take(z.tc ? (size_t)nb * L.n_pass * bwd_tc_image_bytes() : 0);
    L.slots = take(z.tc ? bwd_tc_slots_bytes(nb, z.n_slots) : 0);
    L.dqh = take(z.tc ? bwd_tc_dq_bytes(z.num_sms, nb * L.n_pass, z.n_slots)
                      : (L.n_split > 1 ? heads * L.n_split * row_f32 : 0));
    L.part = take(z.tc ? pairs * L.n_pass * AG_C * 2 : pairs * row_f32);
    L.acc = take(nb < z.n_bq ? (size_t)z.rows * row_f32 : 0);
    L.total = at;
    return L;
}

constexpr size_t WS_TARGET = (size_t)16 << 30;   // the recommended workspace stays below this

// The buffers begin at a 256-byte boundary (the list of contributions is stored 32 bytes at a time);
// a workspace may begin at any 16-byte one, so the size asked for has room for the way to it.
constexpr size_t WS_ALIGN = 256, WS_SLACK = WS_ALIGN - 16;

// The most queries a chunk can have in `bytes` of workspace (0: not one fits).
int64_t chunk_for(const BwdSizes& z, size_t bytes) {
    // fewer queries may split their keys further, so sizes are not monotonic where splits set
    // in; what fits is looked for from above, halving
    int64_t nb = std::min<int64_t>(z.n_bq, 65535);
    if (z.n_slots > 0) nb = std::min<int64_t>(nb, 0x7FFFFFFFll / z.n_slots);   // places fit an int
    while (nb > 0 && bwd_layout(z, nb).total > bytes) nb = nb > 1 ? (nb + 1) / 2 : 0;
    return nb;
}

struct BwdCall {
    const void *q, *kv, *swa, *out, *dout;
    csa2_dtype q_dt, kv_dt, swa_dt, out_dt;
    int64_t N, swa_cap, swa_pos0;
    const int32_t* idx;
    const int64_t *nv, *q_pos;
    int k, window, B, Q, H;
    const float *sink, *lse;
    float rope_base;
    unsigned flags;
    void *dq, *dkv, *dswa;
    float* dsink;
};

csa2_status zero_bytes(void* p, size_t bytes, cudaStream_t s) {
    if (!p || bytes == 0) return CSA2_OK;
    return cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

size_t dt_bytes(csa2_dtype d) { return d == CSA2_F32 ? 4 : 2; }

template <typename TQ, typename TO>
csa2_status simt_chunk(const csa2_ctx* ctx, const BwdCall& a, const BwdChunk& c, float* qh, float* dh, float2* pds,
                       float* dqh, int n_split, int per, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const csa2_status r = raise_smem(bwd_simt_q_kernel<TQ>, SB_SMEM, ctx->device, done);
    if (r != CSA2_OK) return r;
    const int64_t n_rows = (int64_t)c.nb * a.H;
    bwd_prep_kernel<TQ, TO><<<(unsigned)((n_rows + 7) / 8), 256, 0, s>>>(
        reinterpret_cast<const TQ*>(a.q), reinterpret_cast<const TO*>(a.dout), reinterpret_cast<const TO*>(a.out), a.q_pos,
        c.bq0, n_rows, a.H, c.rope, a.flags, qh, dh, const_cast<float*>(c.D));
    bwd_simt_q_kernel<TQ><<<dim3((unsigned)((a.H + SB_HG - 1) / SB_HG), (unsigned)c.nb, (unsigned)n_split), 256, SB_SMEM,
                           s>>>(c, qh, dh, pds, dqh, per, reinterpret_cast<TQ*>(a.dq));
    if (n_split > 1)
        bwd_simt_dq_kernel<TQ><<<(unsigned)((n_rows + 7) / 8), 256, 0, s>>>(c, qh, dqh, n_split, reinterpret_cast<TQ*>(a.dq));
    if (c.n_slots > 0)
        bwd_simt_row_kernel<<<dim3((unsigned)((c.n_slots + 31) / 32), (unsigned)c.nb), 256, 0, s>>>(c, qh, dh, pds);
    return csa2_launch_status();
}

csa2_status bwd_run(csa2_ctx* ctx, const BwdCall& a, void* ws, size_t ws_bytes, cudaStream_t s) {
    const int64_t n_bq = (int64_t)a.B * a.Q;
    const int n_slots = a.k + a.window;
    const int64_t n_kv = a.k > 0 ? (int64_t)a.B * a.N : 0, n_sw = a.window > 0 ? (int64_t)a.B * a.swa_cap : 0;
    const int64_t rows = n_kv + n_sw;
    const BwdSizes z = {n_bq, a.H, n_slots, rows,
                        bwd_tc_applies(a.q_dt, a.kv_dt, a.k, a.swa_dt, a.window, a.out_dt, a.flags), ctx->num_sms};
    const size_t skip = align_up(reinterpret_cast<uintptr_t>(ws), WS_ALIGN) - reinterpret_cast<uintptr_t>(ws);
    // (the chunks go by the size alone, so the results do not depend on where the workspace begins)
    const int64_t nb_max = ws_bytes > WS_SLACK ? chunk_for(z, ws_bytes - WS_SLACK) : 0;
    if (nb_max < 1) return CSA2_ERR_INVALID_ARG;
    const BwdLayout L = bwd_layout(z, nb_max);
    uint8_t* base = reinterpret_cast<uint8_t*>(ws) + skip;
    float* D = reinterpret_cast<float*>(base + L.D);
    float* rinv = reinterpret_cast<float*>(base + L.rinv);
    if (rows > 0)
        bwd_rinv_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a.kv, a.kv_dt, n_kv, a.swa, a.swa_dt, rows, a.flags,
                                                                  rinv);
    BwdChunk c;
    c.slots = {a.idx, a.nv, a.q_pos, a.N, a.swa_cap, a.swa_pos0, a.k, a.window, a.Q, n_kv, ctx->status};
    c.q = a.q;
    c.q_dt = a.q_dt;
    c.kv = a.kv;
    c.kv_dt = a.kv_dt;
    c.swa = a.swa;
    c.swa_dt = a.swa_dt;
    c.lse = a.lse;
    c.D = D;
    c.rinv = rinv;
    c.H = a.H;
    c.n_slots = n_slots;
    c.flags = a.flags;
    c.rope = make_ag_rope(a.rope_base);
    uint32_t* cnt = reinterpret_cast<uint32_t*>(base + L.cnt);
    uint32_t* loc = reinterpret_cast<uint32_t*>(base + L.loc);
    uint32_t* tot = reinterpret_cast<uint32_t*>(base + L.tot);
    uint32_t* blk = reinterpret_cast<uint32_t*>(base + L.blk);
    int32_t* rank = reinterpret_cast<int32_t*>(base + L.rank);
    c.rank = rank;
    c.base = cnt;
    c.blk = blk;
    c.rows = rows;
    c.group_q = L.group_q;
    c.part = base + L.part;
    c.dq = a.dq;
    const int64_t n_blk = (rows + BWD_SCAN_ROWS - 1) / BWD_SCAN_ROWS;
    for (int64_t bq0 = 0; bq0 < n_bq; bq0 += nb_max) {
        c.bq0 = bq0;
        c.nb = (int)std::min<int64_t>(nb_max, n_bq - bq0);
        // (without rows too: an index into a cache of none is flagged here)
        if (n_slots > 0) {
            const csa2_status zr = zero_bytes(cnt, (size_t)L.groups * rows * 4, s);
            if (zr != CSA2_OK) return zr;
            bwd_rank_kernel<<<(unsigned)L.groups, 1024, 0, s>>>(c.slots, bq0, c.nb, L.group_q, n_slots, rows, cnt, rank);
        }
        if (rows > 0) {
            bwd_place_kernel<<<(unsigned)n_blk, BWD_SCAN_ROWS, 0, s>>>(cnt, L.groups, rows, loc, tot, blk);
            bwd_scan(blk, n_blk, s);
        }
        float* qh = reinterpret_cast<float*>(base + L.qh);
        float* dh = reinterpret_cast<float*>(base + L.dh);
        float2* pds = reinterpret_cast<float2*>(base + L.pds);
        float* dqh = reinterpret_cast<float*>(base + L.dqh);
        csa2_status r;
        if (z.tc) {
            BwdTcArgs t;
            t.c = c;
            t.dqh = reinterpret_cast<float*>(base + L.dqh);
            t.n_pass = L.n_pass;
            r = bwd_tc_chunk(ctx, t, a.dout, a.out, D, base + L.img, base + L.slots, s);
        } else if (a.q_dt == CSA2_F32)
            r = a.out_dt == CSA2_F32 ? simt_chunk<float, float>(ctx, a, c, qh, dh, pds, dqh, L.n_split, L.tps, s)
                                     : simt_chunk<float, __nv_bfloat16>(ctx, a, c, qh, dh, pds, dqh, L.n_split, L.tps, s);
        else
            r = a.out_dt == CSA2_F32 ? simt_chunk<__nv_bfloat16, float>(ctx, a, c, qh, dh, pds, dqh, L.n_split, L.tps, s)
                                     : simt_chunk<__nv_bfloat16, __nv_bfloat16>(ctx, a, c, qh, dh, pds, dqh, L.n_split, L.tps, s);
        if (r != CSA2_OK) return r;
        if (rows > 0 && (a.dkv || a.dswa)) {
            RowSumArgs ra;
            ra.part = c.part;
            ra.passes = L.n_pass;
            ra.loc = loc;
            ra.tot = tot;
            ra.blk = blk;
            ra.rows = rows;
            ra.n_kv = n_kv;
            ra.kv = a.kv;
            ra.swa = a.swa;
            ra.kv_dt = a.kv_dt;
            ra.swa_dt = a.swa_dt;
            ra.rinv = rinv;
            ra.flags = a.flags;
            ra.acc = nb_max < n_bq ? reinterpret_cast<float*>(base + L.acc) : nullptr;
            ra.first = bq0 == 0;
            ra.last = bq0 + c.nb == n_bq;
            ra.dkv = a.dkv;
            ra.dswa = a.dswa;
            if (z.tc)
                bwd_rowsum_kernel<__nv_bfloat16><<<(unsigned)rows, 128, 0, s>>>(ra);
            else
                bwd_rowsum_kernel<float><<<(unsigned)rows, 128, 0, s>>>(ra);
        }
        if (csa2_launch_status() != CSA2_OK) return CSA2_ERR_CUDA;
    }
    if (a.dsink) {
        const int64_t n = sink_stretches(n_bq), per = (n_bq + n - 1) / n;
        float* part = n > 1 ? reinterpret_cast<float*>(base + L.sink) : a.dsink;
        bwd_sink_kernel<<<dim3((unsigned)((a.H + 31) / 32), (unsigned)n), 256, 0, s>>>(a.sink, a.lse, D, n_bq, a.H, per, part);
        if (n > 1) bwd_sink_sum_kernel<<<1, 128, 0, s>>>(part, (int)n, a.H, a.dsink);
    }
    return csa2_launch_status();
}

csa2_status bwd_impl(csa2_ctx* ctx, const BwdCall& a, int c, void* ws, size_t ws_bytes, void* stream) {
    if (!ctx || a.B < 0 || a.Q < 0 || a.N < 0 || a.k < 0 || a.window < 0 || a.window > 1024) return CSA2_ERR_INVALID_ARG;
    if (a.H < 1 || a.H > 128) return CSA2_ERR_INVALID_ARG;
    if (c != AG_C) return CSA2_ERR_UNSUPPORTED;
    if (a.flags & ~CSA2_ATTN_DEFAULT) return CSA2_ERR_INVALID_ARG;
    for (csa2_dtype d : {a.q_dt, a.kv_dt, a.swa_dt, a.out_dt})
        if (d != CSA2_F32 && d != CSA2_BF16) return CSA2_ERR_UNSUPPORTED;
    const int64_t n_bq = (int64_t)a.B * a.Q;
    if (n_bq > 65535) return CSA2_ERR_UNSUPPORTED;
    if (a.window > 0 && ((!a.swa && n_bq > 0) || a.swa_cap < a.window)) return CSA2_ERR_INVALID_ARG;
    if (a.swa_cap < 0) return CSA2_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)a.B * (a.N + a.swa_cap);
    if (rows > 0x7FFFFFFF) return CSA2_ERR_UNSUPPORTED;
    if (!aligned(a.q, 16) || !aligned(a.kv, 16) || !aligned(a.swa, 16) || !aligned(a.out, 16) || !aligned(a.dout, 16) ||
        !aligned(a.dq, 16) || !aligned(a.dkv, 16) || !aligned(a.dswa, 16) || !aligned(ws, 16) || !aligned(a.lse, 4) ||
        !aligned(a.dsink, 4) || !aligned(a.q_pos, 8))
        return CSA2_ERR_INVALID_ARG;
    if (n_bq > 0 && (!a.q || !a.q_pos || !a.out || !a.dout || !a.lse || !a.dq || !ws)) return CSA2_ERR_INVALID_ARG;
    if (n_bq > 0 && a.k > 0 && ((!a.idx && !a.nv) || !a.kv)) return CSA2_ERR_INVALID_ARG;
    DeviceGuard dev(ctx);
    if (!dev.ok) return CSA2_ERR_CUDA;
    cudaStream_t s = as_stream(stream);
    // rows that no call below visits have no gradient
    csa2_status r = CSA2_OK;
    if (a.k == 0 || n_bq == 0) r = zero_bytes(a.dkv, (size_t)a.B * a.N * AG_C * dt_bytes(a.kv_dt), s);
    if (r == CSA2_OK && (a.window == 0 || n_bq == 0))
        r = zero_bytes(a.dswa, (size_t)a.B * a.swa_cap * AG_C * dt_bytes(a.swa_dt), s);
    if (r == CSA2_OK && n_bq == 0) r = zero_bytes(a.dsink, (size_t)a.H * 4, s);
    if (r != CSA2_OK || n_bq == 0) return r;
    return bwd_run(ctx, a, ws, ws_bytes, s);
}

}  // namespace

void bwd_scan(uint32_t* blk, int64_t n, cudaStream_t s) { bwd_scan_kernel<<<1, 1024, 0, s>>>(blk, n); }

extern "C" size_t csa2_attn_bwd_workspace_bytes(csa2_ctx* ctx, csa2_dtype q_dt, csa2_dtype kv_dt, csa2_dtype swa_dt,
                                                csa2_dtype out_dt, int B, int Q, int H, int k, int window, int64_t N,
                                                int64_t swa_cap, unsigned flags) {
    if (!ctx || B <= 0 || Q <= 0 || H < 1 || H > 128 || k < 0 || window < 0 || N < 0 || swa_cap < 0) return 0;
    const int64_t rows = (k > 0 ? (int64_t)B * N : 0) + (window > 0 ? (int64_t)B * swa_cap : 0);
    const BwdSizes z = {(int64_t)B * Q, H, k + window, rows,
                        bwd_tc_applies(q_dt, kv_dt, k, swa_dt, window, out_dt, flags), ctx->num_sms};
    return bwd_layout(z, std::max<int64_t>(1, chunk_for(z, WS_TARGET - WS_SLACK))).total + WS_SLACK;
}

extern "C" csa2_status csa2_sparse_attn_bwd(csa2_ctx* ctx, const void* q, csa2_dtype q_dt, const void* kv,
                                            csa2_dtype kv_dt, int64_t N, const int32_t* idx, int k, const void* swa,
                                            csa2_dtype swa_dt, int64_t swa_cap, int64_t swa_pos0, int window,
                                            const int64_t* q_pos, const float* sink, const void* out, const void* dout,
                                            csa2_dtype out_dt, const float* lse, int B, int Q, int H, int c,
                                            float rope_base, unsigned flags, void* dq, void* dkv, void* dswa,
                                            float* dsink, void* ws, size_t ws_bytes, void* stream) {
    if (k > 2048) return CSA2_ERR_INVALID_ARG;
    const BwdCall a = {q, kv, swa, out, dout, q_dt, kv_dt, swa_dt, out_dt, N, swa_cap, swa_pos0, idx, nullptr, q_pos, k,
                       window, B, Q, H, sink, lse, rope_base, flags, dq, dkv, dswa, dsink};
    return bwd_impl(ctx, a, c, ws, ws_bytes, stream);
}

extern "C" csa2_status csa2_dense_attn_bwd(csa2_ctx* ctx, const void* q, csa2_dtype q_dt, const void* kv,
                                           csa2_dtype kv_dt, int64_t N, const int64_t* n_visible, int k_max,
                                           const void* swa, csa2_dtype swa_dt, int64_t swa_cap, int64_t swa_pos0,
                                           int window, const int64_t* q_pos, const float* sink, const void* out,
                                           const void* dout, csa2_dtype out_dt, const float* lse, int B, int Q, int H,
                                           int c, float rope_base, unsigned flags, void* dq, void* dkv, void* dswa,
                                           float* dsink, void* ws, size_t ws_bytes, void* stream) {
    if (k_max < 0 || k_max > (1 << 22)) return CSA2_ERR_INVALID_ARG;
    const BwdCall a = {q, kv, swa, out, dout, q_dt, kv_dt, swa_dt, out_dt, N, swa_cap, swa_pos0, nullptr, n_visible,
                       q_pos, k_max, window, B, Q, H, sink, lse, rope_base, flags, dq, dkv, dswa, dsink};
    return bwd_impl(ctx, a, c, ws, ws_bytes, stream);
}
