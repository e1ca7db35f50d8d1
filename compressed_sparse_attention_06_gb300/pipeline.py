"""Per-layer steps of the CSA2 hot path, strung from the C-ABI entry points.

Every arithmetic step runs in libcsa2.so; this module only allocates outputs
(torch device memory) and orders the calls on the current stream.

Layer modes (CSA2 page, «三种模式：谁算、谁复用»):
  Full    -- own indexer over all visible entries (+ block pool in the decoder),
  Reindex -- own indexer over the pooled candidates only,
  Reuse   -- upstream indices, attention only.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, Optional

import torch

from . import csa2 as C

TOPK = 512
POOL_BLOCK = 8
POOL_KEEP = 2048


def visible_entries(q_pos: torch.Tensor, m: int) -> torch.Tensor:
    """Entries visible to each query: entry j needs t >= m(j+1), so floor(t/m)
    (DSA-to-CSA/HCA page, «因果边界与短滑窗»); computed by csa2_visible_entries."""
    return C.csa2_visible_entries(q_pos, m)


@dataclass
class DecodeBuffers:
    """Preallocated outputs of a Full-mode decode step (reused across steps)."""
    scores: torch.Tensor         # the full scan's scores (the top-k reads its best blocks' entries)
    block_max: torch.Tensor
    block_hist: torch.Tensor     # the scan's summary of the block maxima, for the pool
    pool: torch.Tensor
    top_blocks: torch.Tensor     # the best top_n blocks: the top-k entries lie in them
    cand_scores: torch.Tensor
    idx: torch.Tensor
    out: torch.Tensor
    attn_ws: torch.Tensor
    pool_ws: torch.Tensor
    topk_ws: torch.Tensor
    qI_mx: torch.Tensor          # the indexer query packed to MXFP4 (FP4 QK path)


def top_blocks_for(k: int) -> int:
    """Blocks the top-k selection rescores: the k best blocks hold the top-k entries
    (every block ranked above a block b holds its maximum, which ranks above every
    entry of b), rounded up to a whole candidate tile of 32 blocks."""
    return (k + 31) // 32 * 32


def alloc_decode(B: int, Q: int, N: int, H: int, c: int, device, out_dtype=torch.bfloat16,
                 k: int = TOPK, block: int = POOL_BLOCK, n_keep: int = POOL_KEEP,
                 window: int = 128, h_idx: int = 64) -> DecodeBuffers:
    nb = (N + block - 1) // block
    n_top = top_blocks_for(k)
    return DecodeBuffers(
        scores=C.alloc((B, Q, N), dtype=torch.float32, device=device),
        block_max=C.alloc((B, Q, nb), dtype=torch.float32, device=device),
        block_hist=C.alloc((B, Q, C.BLOCK_HIST_BINS), dtype=torch.int32, device=device),
        pool=C.alloc((B, Q, n_keep), dtype=torch.int32, device=device),
        top_blocks=C.alloc((B, Q, n_top), dtype=torch.int32, device=device),
        cand_scores=C.alloc((B, Q, n_top * block), dtype=torch.float32, device=device),
        idx=C.alloc((B, Q, k), dtype=torch.int32, device=device),
        out=C.alloc((B, Q, H, c), dtype=out_dtype, device=device),
        attn_ws=C.alloc(max(16, C.csa2_sparse_attn_workspace_bytes(B, Q, H, k, window,
                                                                       torch.device(device).index, N=N,
                                                                       swa_cap=window)),
                            dtype=torch.uint8, device=device),
        pool_ws=C._ws(C.csa2_block_pool_workspace_bytes(B * Q, nb, n_keep, torch.device(device).index), device),
        topk_ws=C._ws(C.csa2_topk_workspace_bytes(B * Q, n_top * block, k, torch.device(device).index), device),
        qI_mx=C.alloc((B, Q, h_idx, C.mxfp4_row_bytes(128)), dtype=torch.uint8, device=device),
    )


def full_decode_step(qI, w, kI, q, kv, swa, q_pos, n_visible, sink, buf: DecodeBuffers, *,
                     window: int = 128, swa_pos0: int = 0, k: int = TOPK, block: int = POOL_BLOCK,
                     n_keep: int = POOL_KEEP, flags: int = C.ATTN_DEFAULT,
                     side_stream: Optional[torch.cuda.Stream] = None):
    """Full layer with the hierarchical pool (CSA2 page, «解码器里的分层索引»):
    scan all visible entries (scores, block maxima and their histogram), pick the
    pool (for the Reindex layers that follow) and the layer's own top-k in one call
    (the top-k of all entries lies inside the k best blocks, which lie inside the
    pool), and attend over the selected entries plus the window.  Shapes that call
    does not take run the pool, the best blocks' rescoring and the top-k one by one.

    With an MXFP4 indexer cache the QK product runs in FP4 (DSA-to-CSA/HCA page,
    «Lightning Indexer：公式 (13)–(17)»): a bf16/f32 qI is first packed to MXFP4 by
    the same rule as the keys (into buf.qI_mx); an already packed uint8 qI is used
    as given.

    side_stream: the attention's query half (csa2_attn_prepare) runs there, beside
    the selection, after the scan (which fills the GPU by itself)."""
    fused = pool_topk_applies(k, block, n_keep, buf.block_max.shape[-1])
    if mxq_applies(qI, kI, block):
        # the FP4 QK path with the query packed inside the scan (packed bytes kept in buf)
        C.csa2_index_score_mxq(qI, w, kI, n_visible, block=block, scores=buf.scores if fused else None,
                               want_scores=fused, want_block_max=True, block_max=buf.block_max,
                               block_hist=buf.block_hist, q_mx_out=buf.qI_mx)
        qI = buf.qI_mx
    else:
        qI = mxfp4_query(qI, kI, buf.qI_mx)
        C.csa2_index_score(qI, w, kI, n_visible, block=block, scores=buf.scores if fused else None,
                           want_scores=fused, want_block_max=True, block_max=buf.block_max,
                           block_hist=buf.block_hist)
    B, Q, H = q.shape[:3]
    prepared = side_stream is not None and H <= 64
    if prepared:
        side_stream.wait_stream(torch.cuda.current_stream(q.device))
        with torch.cuda.stream(side_stream):
            C.csa2_attn_prepare(q, q_pos, buf.attn_ws, k, window=window, N=kv.shape[1], swa_cap=swa.shape[1],
                                flags=flags)
    if fused:
        C.csa2_pool_topk(buf.block_max, buf.block_hist, buf.scores, n_visible, k, block=block, n_keep=n_keep,
                         out=buf.pool, out_idx=buf.idx)
    else:
        C.csa2_block_pool(buf.block_max, n_visible, block=block, n_keep=n_keep, out=buf.pool, ws=buf.pool_ws,
                          block_hist=buf.block_hist, n_top=buf.top_blocks.shape[-1], out_top=buf.top_blocks)
        C.csa2_index_score(qI, w, kI, n_visible, pool=buf.top_blocks, block=block, scores=buf.cand_scores)
        C.csa2_topk(buf.cand_scores, n_visible, k, pool=buf.top_blocks, block=block, out_idx=buf.idx,
                    ws=buf.topk_ws)
    if prepared:
        torch.cuda.current_stream(q.device).wait_stream(side_stream)
    C.csa2_sparse_attn(q, kv, buf.idx, swa, q_pos, sink, window=window, swa_pos0=swa_pos0,
                       flags=flags | (C.ATTN_PREPARED if prepared else 0), out=buf.out, ws=buf.attn_ws)
    return buf


def pool_topk_applies(k: int, block: int, n_keep: int, n_blocks: int) -> bool:
    """The shapes csa2_pool_topk takes (its header states them)."""
    chunk = -(-(-(-n_blocks // 16)) // 1024) * 1024
    return 1 <= k <= n_keep - 1 and k * block <= 8192 and block <= 16 and chunk <= 16384


def mxq_applies(qI, kI, block: int) -> bool:
    """Shapes csa2_index_score_mxq takes: a bf16 query of 64 heads x 128 over MXFP4 keys,
    blocks of 8, a cache length that is a multiple of 8."""
    return (qI.dtype == torch.bfloat16 and kI.dtype == torch.uint8 and tuple(qI.shape[2:]) == (64, 128)
            and block == 8 and kI.shape[1] % 8 == 0)


def mxfp4_query(qI, kI, out=None):
    """The indexer query as the scan takes it: packed to MXFP4 when the keys are
    MXFP4 (uint8 rows) and the query is not packed yet; unchanged otherwise."""
    if kI.dtype != torch.uint8 or qI.dtype == torch.uint8:
        return qI
    return C.csa2_fp4_pack(qI, C.MXFP4_E8M0x32, out=out)


def reindex_step(qI, w, kI, pool, n_visible, cand_scores=None, idx=None, k: int = TOPK, block: int = POOL_BLOCK):
    """Reindex layer: own indexer query over the pooled candidates, then top-k
    (FP4 QK product over an MXFP4 cache, as in full_decode_step)."""
    qI = mxfp4_query(qI, kI)
    sc, _ = C.csa2_index_score(qI, w, kI, n_visible, pool=pool, block=block, scores=cand_scores)
    ids, _ = C.csa2_topk(sc, n_visible, k, pool=pool, block=block, out_idx=idx)
    return ids


def reuse_attention(q, kv, idx, swa, q_pos, sink, out=None, window: int = 128, swa_pos0: int = 0,
                    flags: int = C.ATTN_DEFAULT):
    """Reuse layer (and the attention of Full/Reindex layers): upstream indices, own
    query and own window."""
    o, _ = C.csa2_sparse_attn(q, kv, idx, swa, q_pos, sink, window=window, swa_pos0=swa_pos0, flags=flags,
                              out=out)
    return o


def full_topk_step(qI, w, kI, n_visible, k: int = TOPK, scores=None, idx=None):
    """Full layer without a pool (encoder / prefill): full scores, then top-k
    (FP4 QK product over an MXFP4 cache, as in full_decode_step)."""
    qI = mxfp4_query(qI, kI)
    sc, _ = C.csa2_index_score(qI, w, kI, n_visible, scores=scores)
    ids, _ = C.csa2_topk(sc, n_visible, k, out_idx=idx)
    return sc, ids


@dataclass
class PrefillBuffers:
    scores: torch.Tensor
    idx: torch.Tensor
    out: torch.Tensor
    n_visible: torch.Tensor
    attn_ws: torch.Tensor
    topk_ws: torch.Tensor


def alloc_prefill(Q: int, N: int, H: int, c: int, device, q_pos: torch.Tensor, m: int,
                  out_dtype=torch.bfloat16, k: int = TOPK, window: int = 128, swa_cap: int = 0) -> PrefillBuffers:
    """swa_cap: rows of the window buffer the attention will read (sizes the workspace
    for the per-call table of row RMS factors)."""
    return PrefillBuffers(
        scores=C.alloc((1, Q, N), dtype=torch.float32, device=device),
        idx=C.alloc((1, Q, k), dtype=torch.int32, device=device),
        out=C.alloc((1, Q, H, c), dtype=out_dtype, device=device),
        n_visible=visible_entries(q_pos, m),
        attn_ws=C.alloc(max(16, C.csa2_sparse_attn_workspace_bytes(1, Q, H, k, window,
                                                                       torch.device(device).index, N=N,
                                                                       swa_cap=swa_cap)),
                            dtype=torch.uint8, device=device),
        topk_ws=C._ws(C.csa2_topk_workspace_bytes(Q, N, k, torch.device(device).index), device),
    )


def prefill_chunk_step(Ca, Cb, Za, Zb, Ba, Bb, prev_Cb, prev_Zb, kv_cache, n_ctx_entries: int, pos0: torch.Tensor,
                       m: int, qI, w, kI, q, swa, swa_pos0: int, q_pos, sink, buf: PrefillBuffers, *,
                       k: int = TOPK, window: int = 128, write_flags: int = C.W_NORM | C.W_ROPE):
    """Encoder prefill chunk (Full layer): the overlapped compressor turns the chunk's
    tokens into new cache entries (carrying the previous block's state), then every
    query of the chunk scores all entries it can see, takes its top-k and attends
    over them plus its window."""
    C.csa2_compress(Ca, Za, m, cb=Cb, zb=Zb, ba=Ba, bb=Bb, prev_cb=prev_Cb, prev_zb=prev_Zb, pos0=pos0,
                    flags=write_flags, out=kv_cache[0, n_ctx_entries:], out_seq_stride=0)
    qI = mxfp4_query(qI, kI)
    C.csa2_index_score(qI, w, kI, buf.n_visible, scores=buf.scores)
    C.csa2_topk(buf.scores, buf.n_visible, k, out_idx=buf.idx, ws=buf.topk_ws)
    C.csa2_sparse_attn(q, kv_cache, buf.idx, swa, q_pos, sink, window=window, swa_pos0=swa_pos0, out=buf.out,
                       ws=buf.attn_ws)
    return buf


def layer_backward(q, kv, idx, swa, q_pos, sink, out, lse, dout, ca, za, m: int, *, cb=None, zb=None, ba=None, bb=None,
                   prev_cb=None, prev_zb=None, pos0=0, window: int = 128, swa_pos0: int = 0,
                   flags: int = C.ATTN_DEFAULT, write_flags: int = C.W_NORM | C.W_ROPE):
    """Backward pass of a layer whose whole cache kv [B, N, c] csa2_compress made in one call
    (N = n_tokens / m entries a sequence): the attention's gradients, then the compressor's
    from the rows' gradient.  Returns ((dq, dkv, dswa, dsink), CompressGrads)."""
    att = C.csa2_sparse_attn_bwd(q, kv, idx, swa, q_pos, sink, out, lse, dout, window=window, swa_pos0=swa_pos0,
                                 flags=flags)
    dkv = att[1] if ca.dim() == 3 else att[1][0]
    com = C.csa2_compress_bwd(ca, za, m, dkv, cb=cb, zb=zb, ba=ba, bb=bb, prev_cb=prev_cb, prev_zb=prev_zb, pos0=pos0,
                              flags=write_flags)
    return att, com


@dataclass
class CutCaches:
    """What an eviction leaves: the kept entries' old ids, and every cache cut to them."""
    idx: torch.Tensor            # [B, keep] int32 ascending, -1 padded
    n_entries: torch.Tensor      # [B] int64: entries each sequence kept
    acc: torch.Tensor            # [B, keep] f32: their accumulated weights
    caches: Dict[str, torch.Tensor]


def evict_caches(acc, n_entries, caches: Dict[str, torch.Tensor], keep: int, recent: int = 0) -> CutCaches:
    """Cut every sequence to `keep` entries: its newest `recent` and the others of the largest
    accumulated attention weight (csa2_attn_mass).  caches: any [B, N, ..] tensors whose row j
    belongs to entry j (main KV, indexer keys); new ones are returned, with acc cut alike.
    Rows behind a shorter sequence's entries are zero in them.  (To leave room behind the kept entries,
    or to cut into buffers at hand, pad csa2_evict_select's ids with -1 and call csa2_cache_gather.)
    A sequence's next entry goes to row n_entries[b]: it comes from csa2_compress over its finished
    block, as csa2_compress_step writes entry i to row i."""
    idx = C.csa2_evict_select(acc, n_entries, keep, recent=recent)
    B = acc.shape[0]

    def cut(t):
        return C.csa2_cache_gather(t, idx, out=C.alloc((B, keep, *t.shape[2:]), dtype=t.dtype, device=t.device).zero_())

    return CutCaches(idx, n_entries.clamp(min=0, max=min(keep, acc.shape[1])), cut(acc), {name: cut(t) for name, t in caches.items()})


@dataclass
class PagedCache:
    """Caches of B sequences in pages that sequences may share (csa2_pages_*): every pool
    [n_pages, page, ..] holds one kind of rows (main KV, indexer keys, of any layers) of entry e of
    sequence b on page table[b, e // page]; refs counts the places that hold a page.  pages_append, pages_cut
    and pages_compact change the tensors in place, so that a captured step goes on where the last one ended."""
    pools: Dict[str, torch.Tensor]
    refs: torch.Tensor           # [n_pages] int32
    table: torch.Tensor          # [B, max_pages] int32, -1: none
    n_entries: torch.Tensor      # [B] int64

    @property
    def page(self) -> int:
        return next(iter(self.pools.values())).shape[1]


def alloc_pages(B: int, n_pages: int, page: int, max_pages: int, rows: Dict[str, tuple], device) -> PagedCache:
    """An empty paged cache; rows: name -> (shape of a row, dtype), e.g. {"kv": ((288,), torch.uint8)}."""
    return PagedCache({k: C.alloc((n_pages, page, *shape), dtype=dt, device=device) for k, (shape, dt) in rows.items()},
                      torch.zeros(n_pages, dtype=torch.int32, device=device),
                      torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
                      torch.zeros(B, dtype=torch.int64, device=device))


def pages_append(cache: PagedCache, rows: Dict[str, torch.Tensor], count: torch.Tensor) -> torch.Tensor:
    """Append rows[name][b, :count[b]] to every sequence in every pool (count [B] int64; rows of every pool,
    [B, n, ..] with one n, and no more than those), copying the beginning of a page that another sequence
    shares first.  Returns how many entries each sequence got: fewer than count where there were no more
    rows, or the pool or the table's row had no room."""
    given = {name: tuple(rows[name].shape[:2]) if name in rows else None for name in cache.pools}
    if len(set(given.values())) != 1 or None in given.values():
        raise ValueError(f"pages_append takes as many rows for every pool, not {given}")
    count = count.clamp(max=next(iter(given.values()))[1])
    granted, copies = C.csa2_pages_reserve(cache.refs, cache.table, cache.n_entries, count, cache.page)
    for name, pool in cache.pools.items():
        C.csa2_page_copy(pool, copies)
        C.csa2_page_write(pool, cache.table, rows[name], cache.n_entries, granted)
    cache.n_entries.add_(granted)
    return granted


def pages_fork(cache: PagedCache, parent: torch.Tensor) -> PagedCache:
    """Continuations of sequences parent [B_out] int32 (negative: an empty one; one that is no sequence is
    flagged and empty): they share their origins' pages until one of them appends.  The pools and refs are
    the same tensors; the origins stay."""
    table, B = C.csa2_pages_fork(cache.refs, cache.table, parent), cache.n_entries.numel()
    if B == 0:
        n = torch.zeros(parent.shape, dtype=torch.int64, device=parent.device)
    else:
        n = cache.n_entries[parent.clamp(min=0, max=B - 1).long()].masked_fill((parent < 0) | (parent >= B), 0)
    return PagedCache(cache.pools, cache.refs, table, n)


def pages_cut(cache: PagedCache, keep: Optional[torch.Tensor] = None) -> None:
    """Cut every sequence to its first keep[b] entries (None: to nothing; negative or more than it has:
    as it is) and give back the pages behind them."""
    C.csa2_pages_free(cache.refs, cache.table, cache.page, keep)
    if keep is None:
        cache.n_entries.zero_()
    else:
        cache.n_entries.copy_(torch.where(keep < 0, cache.n_entries, torch.minimum(keep, cache.n_entries)))


def pages_compact(cache: PagedCache, *others: PagedCache) -> torch.Tensor:
    """Move the pages in use to the front of every pool.  others: all the other caches over the same pools
    (what pages_fork made of this one, or this one was made of); with one left out that holds pages nothing
    moves, and csa2_ctx_check raises.  Returns the number of pages in use, [1] int64."""
    caches = (cache, *others)
    if any(c.refs is not cache.refs and c.refs.data_ptr() != cache.refs.data_ptr() for c in others):
        raise ValueError("pages_compact takes caches over the same pools")
    if not others:
        moves, n_used = C.csa2_pages_compact(cache.refs, cache.table)
    else:
        tables = torch.cat([c.table.flatten() for c in caches])
        moves, n_used = C.csa2_pages_compact(cache.refs, tables.unsqueeze(0))
        for c, t in zip(caches, tables.split([c.table.numel() for c in caches])):
            c.table.copy_(t.view_as(c.table))
    for pool in cache.pools.values():
        C.csa2_page_copy(pool, moves)
    return n_used


@dataclass
class DraftPlan:
    """A step's drafted trees, planned once for all layers: positions and paths of their nodes."""
    ctx_len: torch.Tensor        # [B] int64 committed tokens
    pos: torch.Tensor            # [B, T] int64, -1: unused node
    path: torch.Tensor           # [B, T, T] int16


def plan_draft(parent: torch.Tensor, ctx_len: torch.Tensor) -> DraftPlan:
    """parent [B, T] int32: the node that a drafted token follows (-1: the committed context,
    less: an unused node)."""
    return DraftPlan(ctx_len, *C.csa2_tree_plan(parent, ctx_len))


def draft_attention(q, cache: PagedCache, plan: DraftPlan, swa, draft, sink=None, idx=None, n_visible=None,
                    k_max: int = 0, kv: str = "kv", window: int = 128, swa_pos0: int = 0, flags: int = C.ATTN_DEFAULT,
                    out=None, ws=None):
    """A layer's attention for every drafted token over the pages of pool `kv`: its selected entries
    idx [B, T, k] (Full, Reindex and Reuse layers; the indexer itself does not read pages, so keys kept in
    them are read out by csa2_page_read first), or all visible ones (n_visible [B, T] <= k_max,
    the heavily compressed cache), its window of committed rows (the ring swa) and its own path's
    draft rows.  idx and n_visible name entries of the cache, so they stop at cache.n_entries: what a node past
    the end of a block of m drafted tokens would see of that block (visible_entries counts it) is not an entry
    before those tokens are accepted and their entry is appended."""
    o, _ = C.csa2_tree_attn(q, cache.pools[kv], plan.pos, plan.path, plan.ctx_len, swa, draft, idx=idx,
                            n_visible=n_visible, k_max=k_max, table=cache.table, sink=sink, window=window,
                            swa_pos0=swa_pos0, flags=flags, out=out, ws=ws)
    return o


def accept_draft(plan: DraftPlan, leaf: torch.Tensor, layers, swa_pos0: int = 0) -> torch.Tensor:
    """After verification: the accepted path's rows (up to node leaf[b] [B] int32, negative: none) enter
    the window ring of every layer, layers = [(draft, swa), ..] (none where no layer has a ring).  Returns the
    sequences' new lengths."""
    new_len = C.alloc(tuple(plan.ctx_len.shape), dtype=torch.int64, device=plan.ctx_len.device)
    for draft, swa in list(layers) or [(None, None)]:
        C.csa2_tree_commit(draft, plan.pos, plan.path, plan.ctx_len, leaf, swa, swa_pos0=swa_pos0, new_len=new_len)
    return new_len
