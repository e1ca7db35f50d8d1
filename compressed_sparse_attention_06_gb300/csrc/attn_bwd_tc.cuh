// Tensor-core path of the attention's backward pass (attn_bwd_tc.cu), called per chunk of
// queries by attn_bwd.cu, which owns validation, the scatter plan and the row sums.
#pragma once

#include "attn_grad.cuh"

struct BwdTcArgs {
    BwdChunk c;               // part: bf16 [places, n_pass, 512]
    const uint8_t* img;       // [n_pass, nb] stacked images of the chunk's queries
    float* dqh;               // [n_pass * nb + ctas - 1, 64, 512] dq^ of every item
    int n_pass;               // 64-head passes
    uint32_t ctas, waves;     // waves of whole queries
    // the queries' slots, padded to whole tiles (filled in by bwd_tc_chunk)
    int n_pad;
    const int32_t* code;      // [nb, n_pad]
    const int32_t* place;     // [nb, n_pad]
    const float* fac;         // [nb, n_pad]
    const int32_t* n_of;      // [nb]
    const uint32_t* tile0;    // [nb + 1] 128-slot tiles of the queries before
    long long budget;
    int stall;                // test hook: no image is copied
};

// Whether the path takes these types and flags.
bool bwd_tc_applies(csa2_dtype q_dt, csa2_dtype kv_dt, int k, csa2_dtype swa_dt, int window, csa2_dtype out_dt,
                    unsigned flags);
// Bytes of dq^ for `queries` (times head passes) of n_slots slots each.
size_t bwd_tc_dq_bytes(int num_sms, int64_t queries, int n_slots);
size_t bwd_tc_image_bytes();
size_t bwd_tc_slots_bytes(int64_t nb, int n_slots);
// Exclusive scan of blk[0 .. n) in place (attn_bwd.cu).
void bwd_scan(uint32_t* blk, int64_t n, cudaStream_t s);
// Images, D, products and dq of a chunk (c.rank .. c.part filled in by the caller).
csa2_status bwd_tc_chunk(csa2_ctx* ctx, BwdTcArgs& a, const void* dout, const void* out, float* D, uint8_t* img,
                         void* slots, cudaStream_t s);
