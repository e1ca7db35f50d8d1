// Tensor-core (tcgen05) path of csa2_tree_attn: bf16 query, window and drafts, bf16 or FP4 rows,
// both RMSNorms.
#pragma once

#include "tree.cuh"

bool tree_tc_applies(csa2_dtype q_dt, csa2_dtype kv_dt, csa2_dtype swa_dt, unsigned flags);
size_t tree_tc_ws_bytes(const csa2_ctx* ctx, int B, int T, int H, int k, int window, bool dense);
csa2_status tree_tc_run(csa2_ctx* ctx, const TreeCall& c, void* ws, cudaStream_t s);
