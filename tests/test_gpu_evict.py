"""Accumulated attention weight and eviction against the f64 oracle, and the decode that goes on
over the cut cache.

Tolerance of the weights: p = exp(z - lse) in fp32 with |z| <= 23: z to 23 * 2^-22 (sums of 512
products, its rounding and exp's), so p to 6e-6; the lse given is the same number on both sides.
The tensor-core path keeps q^ as two bf16 numbers (2^-17 of it left out, z to 23 * 2^-17 / sqrt(3)
at the very worst, about 1e-5 of a typical z of one).  5e-5 (|o| + rms) covers both."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_06_gb300 import csa2 as C
from compressed_sparse_attention_06_gb300 import pipeline as P
from compressed_sparse_attention_06_gb300 import workloads as W
from oracle import csa2_oracle as O
from oracle import csa2_oracle_grad as G
from tests.helpers import assert_close, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 5e-5


def _cache(seed, B, N, kind):
    x = W.normal_tensor((B, N, 512), seed, 2, torch.float32, DEV) * 1.3
    if kind == "fp4":
        kv = C.csa2_fp4_pack(x)
        return kv, O.nvfp4_unpack(to_np(kv).reshape(-1, 288)).reshape(B, N, 512)
    kv = x.to(torch.bfloat16) if kind == "bf16" else x
    return kv, to_np(kv)


def _idx(seed, B, Q, N, k, pad=0):
    idx = torch.full((B, Q, k), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(Q):
            n = k - (pad if (b + i) % 2 else 0)
            idx[b, i, :n] = W.distinct_sample(N, n, seed + b, i).to(torch.int32)
    return idx.to(DEV)


@pytest.mark.parametrize("kind,q_dtype", [("bf16", torch.bfloat16), ("fp4", torch.bfloat16), ("f32", torch.float32),
                                          ("fp4", torch.float32)])
@pytest.mark.parametrize("B,Q,H,N,k,pad", [(2, 1, 64, 900, 512, 100), (1, 1, 1, 1, 1, 0), (2, 7, 40, 300, 65, 64),
                                           (1, 3, 128, 400, 200, 1), (1, 170, 64, 100, 33, 5)])
def test_mass(kind, q_dtype, B, Q, H, N, k, pad):
    kv, kv_np = _cache(31, B, N, kind)
    q = W.normal_tensor((B, Q, H, 512), 31, 1, q_dtype, DEV)
    idx = _idx(31, B, Q, N, k, pad)
    if k > 4:
        idx[0, 0, 1] = idx[0, 0, 0]                        # the same entry twice
    q_pos = torch.arange(B * Q, device=DEV).view(B, Q) * 11
    _, lse = C.csa2_sparse_attn(q, kv, idx, None, q_pos, None, window=0, want_lse=True)
    acc0 = torch.rand(B, N, generator=torch.Generator(DEV).manual_seed(5), device=DEV)
    acc = acc0.clone()
    w, same = C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, acc=acc, want_weights=True)
    C.csa2_ctx_check()
    assert same is acc
    again = acc0.clone()
    C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, acc=again)
    assert torch.equal(acc, again)                         # the same bits every time
    only, none = C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, want_weights=True)
    assert none is None and torch.equal(only, w)
    for b in range(B):
        ow, om = G.attn_mass(to_np(q[b]), kv_np[b], to_np(idx[b]), to_np(q_pos[b]), to_np(lse[b]))
        assert_close(to_np(w[b]), ow, TOL, "weights")
        assert_close(to_np(acc[b]), to_np(acc0[b]) + om, TOL, "acc")
    assert not w[idx < 0].any()
    free = torch.ones(B, N, dtype=torch.bool, device=DEV)
    free.scatter_(1, idx.clamp(min=0).flatten(1).long(), False)
    assert torch.equal(acc[free], acc0[free])


@pytest.mark.parametrize("kind,Q,flags", [("bf16", 330, 7), ("fp4", 330, 7), ("bf16", 3, 0), ("fp4", 3, 0), ("f32", 3, 0),
                                          ("bf16", 200, 4), ("fp4", 200, 2), ("f32", 200, 1)])
def test_mass_flags_and_many_tiles_of_a_cta(kind, Q, flags):
    """Several queries of several tiles for each CTA, so every ring and image turns over.  q enters
    as two bf16 numbers, 2^-18 of each value away at most: of a logit with normalised rows that is
    an RSS of 2^-18 x 1.3, a weight's relative error below 2e-5 at five deviations."""
    H, N, k = 16, 600, 290
    kv, kv_np = _cache(41, 1, N, kind)
    q = W.normal_tensor((1, Q, H, 512), 41, 1, torch.float32 if kind == "f32" else torch.bfloat16, DEV)
    idx = _idx(41, 1, Q, N, k, 130)
    q_pos = torch.arange(Q, device=DEV).view(1, Q) * 13
    _, lse = C.csa2_sparse_attn(q, kv, idx, None, q_pos, None, window=0, want_lse=True, flags=flags)
    w, _ = C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, want_weights=True, flags=flags)
    C.csa2_ctx_check()
    ow, _ = G.attn_mass(to_np(q[0]), kv_np[0], to_np(idx[0]), to_np(q_pos[0]), to_np(lse[0]), flags=flags)
    assert_close(to_np(w[0]), ow, TOL, "weights")
    assert not w[idx < 0].any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_mass_dense(kind):
    B, Q, H, N = 2, 5, 24, 140
    kv, kv_np = _cache(32, B, N, kind)
    q = W.normal_tensor((B, Q, H, 512), 32, 1, torch.float32 if kind == "f32" else torch.bfloat16, DEV)
    nv = torch.tensor([[0, 1, 64, 139, 140], [128, 65, 7, 140, 2]], dtype=torch.int64, device=DEV)
    q_pos = nv * 128 + 5
    _, lse = C.csa2_dense_attn(q, kv, nv, N, None, q_pos, None, window=0, want_lse=True)
    acc = torch.zeros(B, N, device=DEV)
    w, _ = C.csa2_attn_mass(q, kv, q_pos, lse, n_visible=nv, k_max=N, acc=acc, want_weights=True)
    C.csa2_ctx_check()
    for b in range(B):
        sel = np.where(np.arange(N) < to_np(nv[b])[:, None], np.arange(N), -1)
        ow, om = G.attn_mass(to_np(q[b]), kv_np[b], sel, to_np(q_pos[b]), to_np(lse[b]))
        assert_close(to_np(w[b]), ow, TOL, "weights")
        assert_close(to_np(acc[b]), om, TOL, "acc")


@pytest.mark.parametrize("Q", [1, 2])
def test_mass_shows_a_query_of_nan_and_skips_an_empty_one(Q):
    """A NaN query makes its entries' sums NaN (and no others); an lse of -inf counts nothing."""
    kv, _ = _cache(33, 1, 20, "bf16")
    q = W.normal_tensor((1, Q, 64, 512), 33, 1, torch.bfloat16, DEV)
    q[0, 0] = float("nan")
    idx = torch.full((1, Q, 4), -1, dtype=torch.int32, device=DEV)
    idx[0, 0] = torch.tensor([3, 5, 7, -1])
    if Q > 1:
        idx[0, 1] = torch.tensor([8, 9, 10, 11])
    lse = torch.zeros(1, Q, 64, device=DEV)
    acc = torch.ones(1, 20, device=DEV)
    C.csa2_attn_mass(q, kv, torch.zeros(1, Q, dtype=torch.int64, device=DEV), lse, idx=idx, acc=acc)
    assert torch.isnan(acc[0]).nonzero().flatten().tolist() == [3, 5, 7]
    acc = torch.ones(1, 20, device=DEV)
    q[0, 0] = 1.0
    w, _ = C.csa2_attn_mass(q, kv, torch.zeros(1, Q, dtype=torch.int64, device=DEV), torch.full_like(lse, -float("inf")),
                            idx=idx, acc=acc, want_weights=True)
    C.csa2_ctx_check()
    assert not w.any() and bool((acc == 1).all())


@pytest.mark.parametrize("kv_dt", [C.F32, C.BF16, C.FP4_E4M3x16])
@pytest.mark.parametrize("Q", [1, 3])
def test_mass_of_a_cache_without_entries(kv_dt, Q):
    """N = 0 through the C entry (the cache has an address, but no entry yet): weights of 0, an index
    is flagged, and the call succeeds."""
    q = W.normal_tensor((1, Q, 64, 512), 46, 1, torch.bfloat16, DEV)
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    idx = torch.full((1, Q, 4), -1, dtype=torch.int32, device=DEV)
    pos, lse = torch.zeros(1, Q, dtype=torch.int64, device=DEV), torch.zeros(1, Q, 64, device=DEV)
    weights = torch.full((1, Q, 4), float("nan"), device=DEV)
    a = [t.data_ptr() for t in (q, buf, idx, pos, lse, weights)]
    assert C._lib().csa2_attn_mass_workspace_bytes(C.ctx(0), kv_dt, 1, Q, 64, 4, 0, 1) <= 1 << 19

    def call():
        return C._lib().csa2_attn_mass(C.ctx(0), a[0], C.BF16, a[1], kv_dt, 0, a[2], None, 4, a[3], a[4], 1, Q, 64, 512,
                                       10000.0, 7, a[5], a[1], a[1] + (1 << 19), 1 << 19, None)

    torch.cuda.synchronize()
    assert call() == C.OK
    C.csa2_ctx_check()
    assert not weights.any() and not buf[:1 << 19].any()
    idx[0, 0, 1] = 0
    torch.cuda.synchronize()
    assert call() == C.OK
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE


def test_mass_flags_an_out_of_range_index():
    kv, _ = _cache(34, 1, 20, "bf16")
    q = W.normal_tensor((1, 1, 64, 512), 34, 1, torch.bfloat16, DEV)
    acc = torch.zeros(1, 20, device=DEV)
    idx = torch.tensor([[[1, 20, -5]]], dtype=torch.int32, device=DEV)
    w, _ = C.csa2_attn_mass(q, kv, torch.zeros(1, 1, dtype=torch.int64, device=DEV), torch.zeros(1, 1, 64, device=DEV),
                            idx=idx, acc=acc, want_weights=True)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE
    assert w[0, 0, 0] > 0 and not w[0, 0, 1:].any() and acc.count_nonzero() == 1


@pytest.mark.parametrize("B,ld,keep,recent", [
    (1, 1, 1, 0), (3, 7, 3, 1), (2, 1000, 400, 400), (2, 1000, 999, 0), (4, 9001, 4001, 128), (2, 20000, 1, 0),
    (1, 70001, 35000, 1000), (3, 65536, 65535, 7), (3, 65537, 60000, 0), (2, 300001, 299999, 131072), (3, 200000, 17, 16), (2, 8192, 9000, 100), (70, 300, 100, 10)])
def test_select(B, ld, keep, recent):
    """Ties (a coarse grid of weights), rows of any length from 0 to ld, signed zeros, infinities."""
    g = torch.Generator(DEV).manual_seed(ld)
    acc = torch.randint(-3, 60, (B, ld), generator=g, device=DEV).float() / 7.0
    acc[:, ::5] = torch.rand(acc[:, ::5].shape, generator=g, device=DEV) ** 8
    acc[:, 3::11] = -0.0
    acc[:, 4::13] = 0.0
    if ld > 100:
        acc[0, 50], acc[0, 60], acc[-1, 70] = float("inf"), -float("inf"), float("nan")
    n = torch.randint(0, ld + 1, (B,), generator=g, device=DEV)
    n[0] = ld
    if B > 2:
        n[1] = 0
        n[2] = min(keep, ld)
    idx = C.csa2_evict_select(acc, n, keep, recent=recent)
    C.csa2_ctx_check()
    a = acc.cpu().numpy()
    for b in range(B):
        assert np.array_equal(idx[b].cpu().numpy(), G.evict_keep(a[b], int(n[b]), keep, recent)), f"row {b}"


@pytest.mark.parametrize("ld", [30000, 130000])
def test_select_all_equal_and_length_above_ld(ld):
    acc = torch.full((2, ld), 0.25, device=DEV)
    idx = C.csa2_evict_select(acc, torch.tensor([ld, ld + 1], device=DEV), 12345, recent=45)
    want = torch.cat([torch.arange(12300), torch.arange(ld - 45, ld)]).to(torch.int32)
    assert torch.equal(idx[0].cpu(), want) and torch.equal(idx[1].cpu(), want)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE


@pytest.mark.parametrize("shape,dtype", [((288,), torch.uint8), ((68,), torch.uint8), ((512,), torch.bfloat16),
                                         ((), torch.float32), ((512,), torch.float32), ((4,), torch.uint8)])
def test_gather(shape, dtype):
    B, N, keep = 3, 501, 233
    g = torch.Generator(DEV).manual_seed(9)
    n = B * N * (int(np.prod(shape)) if shape else 1) * torch.empty((), dtype=dtype).element_size()
    src = torch.randint(0, 255, (n,), generator=g, device=DEV, dtype=torch.uint8).view(dtype).view(B, N, *shape)
    idx = torch.stack([W.distinct_sample(N, keep, 9, b, DEV) for b in range(B)]).to(torch.int32)
    idx[1, 200:] = -1
    out = torch.zeros((B, keep, *shape), dtype=dtype, device=DEV)
    C.csa2_cache_gather(src, idx, out=out)
    C.csa2_ctx_check()
    want = torch.zeros_like(out)
    for b in range(B):
        at = idx[b] >= 0
        want[b, at] = src[b, idx[b, at].long()]
    assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))       # the -1 rows are as they were
    idx[2, 0] = N
    C.csa2_cache_gather(src, idx, out=out)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE
    inside = src.view(-1)[:out[:, :2].numel()].view(B, 2, *shape)            # rows moved within one buffer
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_cache_gather(src, torch.zeros((B, 2), dtype=torch.int32, device=DEV), out=inside)
    assert e.value.status == C.ERR_INVALID_ARG


@pytest.mark.parametrize("shape,dtype", [((512,), torch.bfloat16), ((), torch.float32)])
@pytest.mark.parametrize("bad", [-2, -7, -2 ** 31, 50, 2 ** 31 - 1])
def test_gather_flags_every_id_outside_the_cache(shape, dtype, bad):
    """-1 alone leaves a row without a word; any other id outside [0, N) leaves it and is flagged."""
    src = W.normal_tensor((2, 50, *shape), 44, 1, dtype, DEV)
    idx = torch.tensor([[3, bad, -1], [-1, 49, 0]], dtype=torch.int32, device=DEV)
    out = torch.full((2, 3, *shape), 7.0, dtype=dtype, device=DEV)
    C.csa2_cache_gather(src, idx, out=out)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE
    for b, i, row in ((0, 0, 3), (1, 1, 49), (1, 2, 0)):
        assert torch.equal(out[b, i], src[b, row])
    for b, i in ((0, 1), (0, 2), (1, 0)):
        assert bool((out[b, i] == 7.0).all())
    idx[0, 1] = -1
    C.csa2_cache_gather(src, idx, out=out)
    C.csa2_ctx_check()


@pytest.mark.parametrize("N,keep", [(10, 20), (10, 10), (10, 6)])
def test_cut_caches_count_the_entries_they_hold(N, keep):
    """A length above the cache's is taken as the cache's (and flagged), one below 0 as 0: the count that
    goes on with the cut cache is the number of its ids, so nothing behind them becomes visible."""
    acc = torch.rand(4, N, generator=torch.Generator(DEV).manual_seed(3), device=DEV)
    kv = W.normal_tensor((4, N, 512), 45, 1, torch.bfloat16, DEV)
    n = torch.tensor([N + 5, N, 3, -2], dtype=torch.int64, device=DEV)
    cut = P.evict_caches(acc, n, {"kv": kv}, keep, recent=2)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE
    assert torch.equal(cut.n_entries, (cut.idx >= 0).sum(1))
    assert cut.n_entries.tolist() == [min(N, keep), min(N, keep), 3, 0]


@pytest.mark.parametrize("B", [0, 3])
def test_an_empty_cache_is_cut_to_nothing(B):
    """No entry (or no sequence) yet: no id, no count, rows of 0."""
    kv = torch.empty((B, 0, 512), dtype=torch.bfloat16, device=DEV)
    cut = P.evict_caches(torch.empty((B, 0), device=DEV), torch.zeros(B, dtype=torch.int64, device=DEV), {"kv": kv}, 5, recent=1)
    C.csa2_ctx_check()
    assert bool((cut.idx == -1).all()) and cut.idx.shape == (B, 5) and not cut.n_entries.any()
    assert cut.caches["kv"].shape == (B, 5, 512) and not cut.caches["kv"].any() and not cut.acc.any()


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_decode_goes_on_over_the_cut_cache(kind):
    """Decode steps account their weights, the cache is cut, and attention over the kept entries of a
    query's selection is what it was over the full cache."""
    B, N, H, keep = 2, 3000, 64, 1200
    kv, kv_np = _cache(35, B, N, kind)
    ki = C.csa2_fp4_pack(W.normal_tensor((B, N, 128), 35, 6, torch.float32, DEV), C.MXFP4_E8M0x32)
    swa = W.normal_tensor((B, 128, 512), 35, 3, torch.bfloat16, DEV)
    sink = W.normal_tensor((H,), 35, 4, torch.float32, DEV)
    acc = torch.zeros(B, N, device=DEV)
    total = [np.zeros(N) for _ in range(B)]
    for step in range(3):
        q = W.normal_tensor((B, 1, H, 512), 36, step, torch.bfloat16, DEV)
        idx = _idx(40 + step, B, 1, N, 512)
        q_pos = torch.full((B, 1), N + step, dtype=torch.int64, device=DEV)
        _, lse = C.csa2_sparse_attn(q, kv, idx, swa, q_pos, sink, want_lse=True)
        C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, acc=acc)
        for b in range(B):
            total[b] += G.attn_mass(to_np(q[b]), kv_np[b], to_np(idx[b]), to_np(q_pos[b]), to_np(lse[b]))[1]
    for b in range(B):
        assert_close(to_np(acc[b]), total[b], TOL, "acc")
    n = torch.tensor([N, N - 100], dtype=torch.int64, device=DEV)
    cut = P.evict_caches(acc, n, {"kv": kv, "ki": ki}, keep, recent=64)
    C.csa2_ctx_check()
    assert cut.n_entries.tolist() == [keep, keep]
    a = acc.cpu().numpy()
    for b in range(B):
        ids = G.evict_keep(a[b], int(n[b]), keep, 64)
        assert np.array_equal(to_np(cut.idx[b]), ids)
        assert torch.equal(cut.caches["kv"][b], kv[b, torch.tensor(ids).long()])
        assert torch.equal(cut.caches["ki"][b], ki[b, torch.tensor(ids).long()])
        assert torch.equal(cut.acc[b], acc[b, torch.tensor(ids).long()])
    # a selection over the cut cache, and the same entries in the full one
    new = _idx(50, B, 1, keep, 512)
    old = torch.gather(cut.idx, 1, new[:, 0].long())[:, None].contiguous()
    q = W.normal_tensor((B, 1, H, 512), 37, 0, torch.bfloat16, DEV)
    q_pos = torch.full((B, 1), N + 9, dtype=torch.int64, device=DEV)
    o1, _ = C.csa2_sparse_attn(q, cut.caches["kv"], new, swa, q_pos, sink)
    o2, _ = C.csa2_sparse_attn(q, kv, old, swa, q_pos, sink)
    assert torch.equal(o1, o2)


def test_mass_captured():
    kv, _ = _cache(38, 1, 400, "fp4")
    q = W.normal_tensor((1, 3, 64, 512), 38, 1, torch.bfloat16, DEV)
    idx = _idx(38, 1, 3, 400, 100)
    q_pos = torch.tensor([[5, 6, 7]], dtype=torch.int64, device=DEV)
    _, lse = C.csa2_sparse_attn(q, kv, idx, None, q_pos, None, window=0, want_lse=True)
    ws = torch.empty(C._lib().csa2_attn_mass_workspace_bytes(C.ctx(0), C.FP4_E4M3x16, 1, 3, 64, 100, 400, 1), dtype=torch.uint8, device=DEV)
    acc, ref = torch.zeros(1, 400, device=DEV), torch.zeros(1, 400, device=DEV)
    graph = torch.cuda.CUDAGraph()
    check, C._check = C._check, lambda fn, st: None if st == C.OK else (_ for _ in ()).throw(C.Csa2Error(fn, st))
    try:
        with torch.cuda.graph(graph):
            C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, acc=acc, ws=ws)
    finally:
        C._check = check
    for _ in range(3):
        graph.replay()
        C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, acc=ref)
    torch.cuda.synchronize()
    assert torch.equal(acc, ref)


def test_mass_expired_wait_is_reported_and_the_context_stays_usable():
    kv, _ = _cache(39, 1, 300, "bf16")
    q = W.normal_tensor((1, 1, 64, 512), 39, 1, torch.bfloat16, DEV)
    idx = _idx(39, 1, 1, 300, 200)
    q_pos = torch.zeros(1, 1, dtype=torch.int64, device=DEV)
    _, lse = C.csa2_sparse_attn(q, kv, idx, None, q_pos, None, window=0, want_lse=True)
    ref, _ = C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, want_weights=True)
    C.csa2_ctx_check()
    C.csa2_ctx_test_stall_next(2_000_000)
    C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, want_weights=True)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_TIMEOUT
    w, _ = C.csa2_attn_mass(q, kv, q_pos, lse, idx=idx, want_weights=True)
    C.csa2_ctx_check()
    assert torch.equal(w, ref)


@pytest.mark.parametrize("H", [24, 100])
def test_mass_dense_fp4(H):
    """The dense form over FP4 rows, one head pass and two, and a query of one entry and of none."""
    B, Q, N = 2, 4, 300
    kv, kv_np = _cache(47, B, N, "fp4")
    q = W.normal_tensor((B, Q, H, 512), 47, 1, torch.bfloat16, DEV)
    nv = torch.tensor([[0, 1, 129, 300], [256, 128, 7, 299]], dtype=torch.int64, device=DEV)
    q_pos = nv * 128 + 5
    _, lse = C.csa2_dense_attn(q, kv, nv, N, None, q_pos, None, window=0, want_lse=True)
    acc = torch.zeros(B, N, device=DEV)
    w, _ = C.csa2_attn_mass(q, kv, q_pos, lse, n_visible=nv, k_max=N, acc=acc, want_weights=True)
    C.csa2_ctx_check()
    for b in range(B):
        sel = np.where(np.arange(N) < to_np(nv[b])[:, None], np.arange(N), -1)
        ow, om = G.attn_mass(to_np(q[b]), kv_np[b], sel, to_np(q_pos[b]), to_np(lse[b]))
        assert_close(to_np(w[b]), ow, TOL, "weights")
        assert_close(to_np(acc[b]), om, TOL, "acc")


def _captured(call):
    """A graph of one call, captured on a stream of its own; the guard checks, which wait, are left out."""
    graph = torch.cuda.CUDAGraph()
    check, C._check = C._check, lambda fn, st: None if st == C.OK else (_ for _ in ()).throw(C.Csa2Error(fn, st))
    try:
        with torch.cuda.graph(graph):
            call()
    finally:
        C._check = check
    return graph


@pytest.mark.parametrize("ld,keep", [(9001, 4001), (130000, 70000)])
def test_select_and_gather_captured(ld, keep):
    """Two graphs of a selection with its gather, replayed in turn after the weights changed in place;
    each has buffers of its own."""
    sides = []
    for i in range(2):
        s = dict(acc=torch.rand((2, ld), generator=torch.Generator(DEV).manual_seed(i), device=DEV),
                 n=torch.tensor([ld, ld // 2], dtype=torch.int64, device=DEV),
                 kv=W.normal_tensor((2, ld, 16), 48, i, torch.float32, DEV),
                 idx=torch.empty((2, keep), dtype=torch.int32, device=DEV), out=torch.zeros((2, keep, 16), device=DEV),
                 ws=torch.empty(max(16, C._lib().csa2_evict_select_workspace_bytes(2, ld)), dtype=torch.uint8, device=DEV))

        def call(s=s):
            C.csa2_evict_select(s["acc"], s["n"], keep, recent=100, out=s["idx"], ws=s["ws"])
            C.csa2_cache_gather(s["kv"], s["idx"], out=s["out"])

        call()
        C.csa2_ctx_check()
        s["graph"] = _captured(call)
        sides.append(s)
    for turn in range(3):
        for s in sides:
            s["acc"].mul_(-1.5).add_(0.25)
            s["out"].zero_()
            s["graph"].replay()
    torch.cuda.synchronize()
    C.csa2_ctx_check()
    for s in sides:
        a = s["acc"].cpu().numpy()
        for b in range(2):
            ids = G.evict_keep(a[b], int(s["n"][b]), keep, 100)
            assert np.array_equal(to_np(s["idx"][b]), ids)
            have = ids >= 0
            assert torch.equal(s["out"][b][torch.tensor(have)], s["kv"][b, torch.tensor(ids[have]).long()])
            assert not s["out"][b][torch.tensor(~have)].any()


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
def test_an_entry_is_appended_to_a_cut_cache(fmt):
    """After a cut the next entry comes from csa2_compress over its finished block and goes behind the
    entries that its sequence kept: the same row as csa2_compress_step writes to the uncut cache, and
    attention over it and kept entries is what it was over the uncut one."""
    B, N, H, m, keep, cap = 2, 200, 64, 4, 60, 72
    n = (N + 1) * m                                          # tokens: N entries, and the block of one more
    ca, za, cb, zb = (W.normal_tensor((B, n, 512), 49, i, torch.bfloat16, DEV) for i in range(4))
    ba, bb = (W.normal_tensor((m, 512), 49, i, torch.float32, DEV) for i in (4, 5))
    kw = dict(ba=ba, bb=bb, flags=C.W_NORM | C.W_ROPE, out_fmt=fmt)
    row = (288,) if fmt == "fp4" else (512,)
    full = torch.zeros((B, N + 1, *row), dtype=torch.uint8 if fmt == "fp4" else torch.bfloat16, device=DEV)
    first = [t[:, :N * m].contiguous() for t in (ca, za, cb, zb)]
    full[:, :N] = C.csa2_compress(first[0], first[1], m, cb=first[2], zb=first[3], **kw)
    state = C.csa2_compress_state(B, 512, m, torch.bfloat16, DEV, overlap=True)
    C.csa2_compress_state_seed(first[0], first[1], m, state, cb=first[2], zb=first[3])
    # the cut: `keep` entries of the first sequence, the 40 that the second one has
    have = torch.tensor([N, 40], dtype=torch.int64, device=DEV)
    acc = torch.rand((B, N), generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    idx = torch.full((B, cap), -1, dtype=torch.int32, device=DEV)
    idx[:, :keep] = C.csa2_evict_select(acc, have, keep, recent=8)
    cache = torch.zeros((B, cap, *row), dtype=full.dtype, device=DEV)
    C.csa2_cache_gather(full[:, :N].contiguous(), idx, out=cache)
    count = have.clamp(max=keep)
    # the next block: token by token into the uncut cache, at once for the cut one
    for p in range(N * m, n):
        C.csa2_compress_step(ca[:, p].contiguous(), za[:, p].contiguous(), m,
                             torch.full((B,), p, dtype=torch.int64, device=DEV), state, cb=cb[:, p].contiguous(),
                             zb=zb[:, p].contiguous(), out=full, out_seq_stride=N + 1, **kw)
    last = [t[:, N * m:].contiguous() for t in (ca, za, cb, zb)]
    new = C.csa2_compress(last[0], last[1], m, cb=last[2], zb=last[3], prev_cb=cb[:, (N - 1) * m:N * m].contiguous(),
                          prev_zb=zb[:, (N - 1) * m:N * m].contiguous(), pos0=torch.full((B,), N * m, device=DEV), **kw)
    cache[torch.arange(B, device=DEV), count] = new[:, 0]
    C.csa2_ctx_check()
    assert torch.equal(new[:, 0], full[:, N])
    # a selection of the new entry and some kept ones, and the same entries of the uncut cache
    cut_sel = torch.stack([torch.cat([c.view(1), torch.arange(0, 40, 3, device=DEV)]) for c in count])[:, None].int().contiguous()
    ids = torch.cat([idx, torch.zeros_like(idx[:, :1])], 1)
    ids[torch.arange(B, device=DEV), count] = N
    old_sel = torch.gather(ids, 1, cut_sel[:, 0].long())[:, None].contiguous()
    q = W.normal_tensor((B, 1, H, 512), 49, 9, torch.bfloat16, DEV)
    q_pos = torch.full((B, 1), n, dtype=torch.int64, device=DEV)
    o1, _ = C.csa2_sparse_attn(q, cache, cut_sel, None, q_pos, None, window=0)
    o2, _ = C.csa2_sparse_attn(q, full, old_sel, None, q_pos, None, window=0)
    C.csa2_ctx_check()
    assert torch.equal(o1, o2)
