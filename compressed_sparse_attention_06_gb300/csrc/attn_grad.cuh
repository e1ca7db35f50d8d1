// What the operators behind the attention's forward pass share (its backward pass and
// the accumulated attention weight): the key slots of a query and their cache rows, the
// row loads, and the host side's device guard.
#pragma once

#include <cuda_runtime.h>

#include "attn_tc.cuh"
#include "csa2_internal.cuh"

constexpr int AG_C = 512;                // head dim
constexpr float AG_LOG2E = 1.4426950408889634f;

// RoPE angles in turns, as 64-bit fractions of a turn: position * fraction modulo 2^64 is the
// angle modulo a turn for any position, in integer arithmetic (64-bit floating point, which the
// exact product would take otherwise, is very slow on this part: a kernel that turned every
// entry's rows waited for it).  theta_j = base^(-2j/64); the fraction is exact to 2^-53 of it.
struct AgRope {
    uint64_t frac[32];
};
static inline AgRope make_ag_rope(float base) {
    AgRope r;
    for (int j = 0; j < 32; ++j) {
        const double turns = pow((double)base, -2.0 * (double)j / 64.0) / 6.283185307179586;
        r.frac[j] = (uint64_t)ldexp(turns - floor(turns), 64);       // (a base below 1 turns more than once)
    }
    return r;
}
__device__ __forceinline__ void ag_cos_sin(const AgRope& r, int64_t pos, int j, float& c, float& s) {
    const uint64_t turn = (uint64_t)pos * r.frac[j];
    sincospif((float)(uint32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);     // 2 turns / 2^32 = 2^-31
}

// The key slots of the queries: first the k cache slots (idx, or entries 0 .. nv-1 in
// the dense form), then `window` window slots.  Window slot w of a query at position t
// is position t - window + 1 + w; slots at negative positions are empty.
struct SlotArgs {
    const int32_t* idx;       // [B*Q, k], or NULL: dense form
    const int64_t* dense_nv;  // [B*Q], dense form
    const int64_t* q_pos;     // [B*Q]
    int64_t N, swa_cap, swa_pos0;
    int k, window, Q;
    int64_t n_kv;             // B * N: row ids below it are cache rows, then window rows
    unsigned int* st;
};

// Row id of key slot `slot` of query bq: b*N + entry, or n_kv + b*swa_cap + window slot;
// -1 for an empty slot.  An entry outside [0, N) is flagged (if `flag`) and empty.
__device__ __forceinline__ int64_t slot_row(const SlotArgs& a, int64_t bq, int slot, bool flag) {
    const int64_t b = bq / a.Q;
    if (slot < a.k) {
        int64_t id;
        if (a.dense_nv) {
            id = slot < a.dense_nv[bq] ? slot : -1;
        } else {
            id = a.idx[bq * a.k + slot];
        }
        if (id < 0) return -1;
        if (id >= a.N) {
            if (flag) csa2_flag(a.st, CSA2_DEVBIT_RANGE);
            return -1;
        }
        return b * a.N + id;
    }
    const int w = slot - a.k;
    if (w >= a.window) return -1;
    const int64_t p = a.q_pos[bq] - a.window + 1 + w;
    if (p < 0) return -1;
    int64_t s = (p - a.swa_pos0) % a.swa_cap;
    if (s < 0) s += a.swa_cap;
    return a.n_kv + b * a.swa_cap + s;
}

// 16 channels [16 lane, 16 lane + 16) of a stored row as f32 (exact for every format).
template <typename T>
__device__ __forceinline__ void ag_load16(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void ag_load16<float>(const float* p, float (&v)[16]) {
    const float4* q = reinterpret_cast<const float4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = q[i];
        v[4 * i] = u.x;
        v[4 * i + 1] = u.y;
        v[4 * i + 2] = u.z;
        v[4 * i + 3] = u.w;
    }
}
template <>
__device__ __forceinline__ void ag_load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 u = q[i];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}

// The lanes' sums of v[0 .. 7]: lane l gets that of v[l & 7].
__device__ __forceinline__ float ag_sums_of_8(float (&v)[8], int lane) {
#pragma unroll
    for (int n = 4, d = 16; n >= 1; n >>= 1, d >>= 1) {
        const bool top = lane & d;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float send = top ? v[k] : v[k + n], keep = top ? v[k + n] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
    }
    float s = v[0];                                          // of v[lane >> 2], over four lanes still
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    return __shfl_sync(0xffffffffu, s, (lane & 7) << 2);
}

// The same of a row of dtype dt (F32, BF16 or FP4) at row index `row` of `base`.
__device__ __forceinline__ void ag_load_row16(const void* base, int dt, int64_t row, int lane, float (&v)[16]) {
    if (dt == CSA2_F32) {
        ag_load16<float>(reinterpret_cast<const float*>(base) + row * AG_C + 16 * lane, v);
    } else if (dt == CSA2_BF16) {
        ag_load16<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(base) + row * AG_C + 16 * lane, v);
    } else {
        const uint8_t* r = reinterpret_cast<const uint8_t*>(base) + row * fp4_row_bytes(AG_C);
        const uint2 codes = *reinterpret_cast<const uint2*>(r + 8 * lane);
        const float s = e4m3_to_f32(r[AG_C / 2 + lane]);
        float lo[8], hi[8];
        e2m1x8_to_f32(codes.x, lo);
        e2m1x8_to_f32(codes.y, hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = lo[j] * s;
            v[8 + j] = hi[j] * s;
        }
    }
}

__device__ __forceinline__ float ag_sumsq16(const float (&v)[16]) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
    return ss;
}

__device__ __forceinline__ float ag_rms_factor(float sumsq) { return 1.0f / sqrtf(sumsq / (float)AG_C + 1e-6f); }

// RoPE by sign * angle on a lane's 16 channels [16 lane, +16): lanes 28..31 hold the
// rotated channels 448..511, pairs (2j, 2j+1); cs / sn: cos / sin of the 32 angles.
__device__ __forceinline__ void ag_rope16(float (&v)[16], int lane, const float* cs, const float* sn, float sign) {
    if (lane < 28) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = 8 * (lane - 28) + i;
        const float c = cs[j], s = sign * sn[j], x0 = v[2 * i], x1 = v[2 * i + 1];
        v[2 * i] = x0 * c - x1 * s;
        v[2 * i + 1] = x1 * c + x0 * s;
    }
}

template <typename T>
__device__ __forceinline__ void ag_store16(T* p, const float (&v)[16]);
template <>
__device__ __forceinline__ void ag_store16<float>(float* p, const float (&v)[16]) {
    float4* q = reinterpret_cast<float4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ uint32_t ag_pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ void ag_store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[16]) {
    uint4* q = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        q[i] = make_uint4(ag_pack_bf16x2(v[8 * i], v[8 * i + 1]), ag_pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                          ag_pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), ag_pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}

// Makes the context's device current for the length of a call (the launches and the
// function attributes then belong to the device that owns the stream and the tensors).
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(const csa2_ctx* ctx) {
        int cur = -1;
        if (cudaGetDevice(&cur) != cudaSuccess) {
            ok = false;
        } else if (cur != ctx->device) {
            ok = cudaSetDevice(ctx->device) == cudaSuccess;
            prev = cur;
        }
    }
    ~DeviceGuard() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

// ---- host side of the backward pass shared by its two paths ------------------------

constexpr int BWD_SCAN_ROWS = 256;       // rows per block of the scatter plan's scan

// One chunk of queries of the backward pass, as both paths take it.
struct BwdChunk {
    SlotArgs slots;           // pointers at the whole call's queries
    const void* q;            // [n_bq, H, 512] in q_dt
    csa2_dtype q_dt;
    const void* kv;
    csa2_dtype kv_dt;
    const void* swa;
    csa2_dtype swa_dt;
    const float* lse;         // [n_bq, H]
    const float* D;           // [n_bq, H]  dout . out
    const float* rinv;        // [rows] RMS factor of every row (1 without CSA2_KVNORM)
    int64_t bq0;              // the chunk's first query
    int nb;                   // its queries
    int H, n_slots;
    unsigned flags;
    AgRope rope;
    // the chunk's scatter plan: the contribution of (query bq, slot s) to its row goes to
    // place blk[row / BWD_SCAN_ROWS] + base[group][row] + rank[bq - bq0][s] of `part`
    const int32_t* rank;      // [nb, n_slots], -1 = empty slot
    const uint32_t* base;     // [groups, rows]
    const uint32_t* blk;
    int64_t rows;
    int group_q;              // queries per group
    void* part;
    void* dq;                 // [n_bq, H, 512] in q_dt
};
