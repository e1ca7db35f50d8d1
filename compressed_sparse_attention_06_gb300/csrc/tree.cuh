// Attention for trees of drafted tokens: what its CUDA-core and tensor-core paths share.
#pragma once

#include "attn_grad.cuh"
#include "attn_tc.cuh"

// Where the rows of a node's slots lie.
struct TreeRows {
    const int32_t* table;         // [B, max_pages], or NULL: kv is [B, N, row]
    int64_t N;                    // entries of a sequence, or of the whole pool
    int max_pages, page;
    const int32_t* idx;           // [B*T, k], or NULL: entries 0 .. n_visible[bt]-1
    const int64_t* n_visible;
    int k;
    int64_t swa_cap, swa_pos0;
    int window;
    const int64_t* pos;
    const int16_t* path;
    const int64_t* ctx_len;
    int T;
};

struct TreeCall {
    TreeRows r;
    const void* q;
    csa2_dtype q_dt;
    const void* kv;
    csa2_dtype kv_dt;
    const void* swa;
    const void* draft;
    csa2_dtype swa_dt;
    const float* sink;
    int B, H;
    AgRope rope;
    unsigned flags;
    void* out;
    csa2_dtype out_dt;
    float* lse;
};

// A node's slots: its cache entries, then the positions of its window, oldest first.
struct TreeNode {
    int64_t bt, b, t, len;        // t = -1: unused, no slots
    int kq, nw;
};

__device__ __forceinline__ TreeNode tree_node(const TreeRows& r, int64_t bt) {
    TreeNode n;
    n.bt = bt;
    n.b = bt / r.T;
    n.t = r.pos[bt];
    n.len = r.ctx_len[n.b];
    n.nw = (int)max((int64_t)0, min((int64_t)r.window, n.t + 1));
    n.kq = 0;                     // (k == 0: neither idx nor n_visible need be given)
    if (n.t >= 0 && r.k > 0) n.kq = r.idx ? r.k : (int)max((int64_t)0, min((int64_t)r.k, r.n_visible[bt]));
    return n;
}

enum { TREE_NONE = 0, TREE_CACHE = 1, TREE_RING = 2, TREE_DRAFT = 3 };

// Row of cache entry e of sequence b, or -1 (flagged if `flag`).
__device__ __forceinline__ int64_t tree_entry_row(const TreeRows& r, int64_t b, int32_t e, unsigned* st, bool flag) {
    if (e < 0) return -1;
    if (!r.table) {
        if (e < r.N) return b * r.N + e;
    } else {
        const int p = e / r.page;
        if (p < r.max_pages) {
            const int64_t row = (int64_t)r.table[b * r.max_pages + p] * r.page + (e - p * r.page);
            if (row >= 0 && row < r.N) return row;
        }
    }
    if (flag) csa2_flag(st, CSA2_DEVBIT_RANGE);
    return -1;
}

// Row of window position p of a node: the ring's below the committed length, else the draft row
// of the path's node there.
__device__ __forceinline__ int64_t tree_window_row(const TreeRows& r, const TreeNode& n, int64_t p, int& kind,
                                                   unsigned* st, bool flag) {
    if (p < n.len) {
        kind = TREE_RING;
        return n.b * r.swa_cap + ((p - r.swa_pos0) % r.swa_cap + r.swa_cap) % r.swa_cap;
    }
    const int64_t d = p - n.len;
    const int j = d < r.T ? r.path[n.bt * r.T + d] : -1;
    if (j >= 0 && j < r.T) {
        kind = TREE_DRAFT;
        return n.b * r.T + j;
    }
    if (flag) csa2_flag(st, CSA2_DEVBIT_RANGE);      // a path that does not belong to the positions
    kind = TREE_NONE;
    return -1;
}

// Slot `slot` of a node: its kind and row.
__device__ __forceinline__ int64_t tree_slot(const TreeRows& r, const TreeNode& n, int slot, int& kind, unsigned* st,
                                             bool flag) {
    kind = TREE_NONE;
    if (slot >= n.kq + n.nw) return -1;
    if (slot < n.kq) {
        const int64_t row = tree_entry_row(r, n.b, r.idx ? r.idx[n.bt * r.k + slot] : slot, st, flag);
        if (row >= 0) kind = TREE_CACHE;
        return row;
    }
    return tree_window_row(r, n, n.t - n.nw + 1 + (slot - n.kq), kind, st, flag);
}
