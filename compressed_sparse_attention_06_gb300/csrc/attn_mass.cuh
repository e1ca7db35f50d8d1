// Accumulated attention weight: what its two paths share.
#pragma once

#include "attn_grad.cuh"

struct MassArgs {
    SlotArgs slots;
    const void* q;
    int q_dt;
    const void* kv;
    int kv_dt;
    const float *qh, *lse;    // qh: CUDA-core path only
    int H;
    unsigned flags;
    AgRope rope;
    int64_t n_bq;
    float *weights, *acc;     // either may be NULL
    unsigned long long* fix;  // addends of acc meet here in units of 2^-39, or NULL: straight to acc
    const float* rinv;        // RMS factors of the bf16 rows, made once per call, or NULL: taken from the rows
    float* passes;            // [n_bq, k] weights summed over head passes (H > 64) if weights is NULL
};

constexpr float MASS_FIX_ONE = 549755813888.0f;     // 2^39
constexpr float MASS_FIX_MAX = 256.0f;

// One addend of an entry.  A weight that no softmax gives (an lse that is not the
// forward's, NaN) is added as it is, so that acc shows it.
__device__ __forceinline__ void add_mass(float* acc, unsigned long long* fix, int64_t at, float w) {
    if (fix && w >= 0.0f && w <= MASS_FIX_MAX) {
        if (w > 0.0f) atomicAdd(fix + at, (unsigned long long)__float2ull_rn(w * MASS_FIX_ONE));
    } else {
        atomicAdd(acc + at, w);
    }
}

// Tensor-core path (attn_mass_tc.cu): bf16 or FP4 rows.
csa2_status mass_tc_run(csa2_ctx* ctx, const MassArgs& a, cudaStream_t s);
