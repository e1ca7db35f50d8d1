"""Backward pass of the attention against the f64 gradient oracle: both dtypes' paths, sparse
and dense form, odd sizes, head counts, queries without keys, repeated indices, chunked
workspaces, flags, and the same bits from every run.

Tolerances, as |g - o| <= tol (|o| + rms(o)):
  * fp32 path (fp32 inputs): products and sums of at most 2,048 terms in fp32; the sums' rounding
    is about sqrt(2048) 2^-24 = 3e-6 of the terms' rms, a logit of size up to 23 moves by
    23 * 2^-22, so p by 6e-6; 1e-4 as for the forward pass.
  * the same path with bf16 inputs and outputs: one rounding of the result more, at most 2^-8 of
    |o| (8 significant bits).
  * tensor-core path: a gradient is a sum of terms dS k^, or dS q^ and p do'.  In each term p r (or
    dS r) and the other factor are rounded to bf16, q^'s rounding moves the logit by as much as
    one more rounding, and the terms' sum over a query's heads is rounded too: four independent
    relative errors of at most 2^-8 each, 2^-8 * 0.42 = 1.65e-3 rms over a uniform mantissa, so
    3.3e-3 of the root sum of squares T of the element's terms; the largest of 1e6 elements is
    6.5 times that, 2.2e-2 T (a single term: at most 4 * 2^-8 = 1.6e-2 T).  do' is rounded in its
    64 rotated channels only, which moves dP = do'.k^ by 1.65e-3 of the root sum of squares of
    those 64 products; p / sqrt(c) times that enters T beside dS, because it does not shrink
    where dP comes close to D (a peaked softmax).  The result's own rounding adds 2^-8 |o|.  T also holds what the
    norms' projections make of the same errors, which is all there is where a channel of the
    only key is near 0."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_06_gb300 import csa2 as C
from compressed_sparse_attention_06_gb300 import workloads as W
from oracle import csa2_oracle as O
from oracle import csa2_oracle_grad as G
from tests.helpers import assert_close, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32_TOL, BF16_TOL, TC_TOL = 1e-4, 1e-4 + 2.0 ** -8, "terms"


def _case(seed, B, Q, H, N, k, window, cap, pos, dtype, n_pad=0, sink=True, dense=False, flags=C.ATTN_DEFAULT, scale=1.0):
    s = dict(window=window, flags=flags, k=k)
    s["q"] = W.normal_tensor((B, Q, H, 512), seed, 1, dtype, DEV, std=scale)
    s["kv"] = W.normal_tensor((B, N, 512), seed, 2, dtype, DEV, std=1.3 * scale)
    s["swa"] = W.normal_tensor((B, max(cap, 1), 512), seed, 3, dtype, DEV, std=scale)
    s["q_pos"] = torch.tensor(pos, dtype=torch.int64, device=DEV).reshape(B, Q)
    s["sink"] = W.normal_tensor((H,), seed, 4, torch.float32, DEV) if sink else None
    s["dout"] = W.normal_tensor((B, Q, H, 512), seed, 5, dtype, DEV)
    if dense:
        s["nv"] = torch.tensor([[(37 * (b + 3 * i)) % (k + 1) for i in range(Q)] for b in range(B)], dtype=torch.int64,
                               device=DEV)
    else:
        idx = torch.full((B, Q, k), -1, dtype=torch.int32)
        for b in range(B):
            for i in range(Q):
                n = max(0, k - (n_pad if (b + i) % 2 else 0))
                if n:
                    idx[b, i, :n] = W.distinct_sample(N, n, seed + 7 + b, i).to(torch.int32)
        s["idx"] = idx.to(DEV)
    return s


def _forward(s):
    """out and lse in the case's dtype from the library's own forward pass."""
    kw = dict(window=s["window"], flags=s["flags"], want_lse=True)
    if "nv" in s:
        o, l = C.csa2_dense_attn(s["q"], s["kv"], s["nv"], s["k"], s["swa"], s["q_pos"], s["sink"], **kw)
    else:
        o, l = C.csa2_sparse_attn(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], **kw)
    s["out"], s["lse"] = o, l
    return s


def _backward(s, **kw):
    kw = dict(window=s["window"], flags=s["flags"], **kw)
    if "nv" in s:
        return C.csa2_dense_attn_bwd(s["q"], s["kv"], s["nv"], s["k"], s["swa"], s["q_pos"], s["sink"], s["out"], s["lse"],
                                     s["dout"], **kw)
    return C.csa2_sparse_attn_bwd(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], s["out"], s["lse"],
                                  s["dout"], **kw)


def _oracle(s):
    B, Q = s["q"].shape[:2]
    parts = []
    for b in range(B):
        sel = [np.arange(int(s["nv"][b, i])) for i in range(Q)] if "nv" in s else to_np(s["idx"][b])
        parts.append(G.attn_bwd(to_np(s["q"][b]), to_np(s["kv"][b]), sel, to_np(s["swa"][b]), 0, to_np(s["q_pos"][b]),
                                None if s["sink"] is None else to_np(s["sink"]), s["window"], to_np(s["out"][b]),
                                to_np(s["lse"][b]), to_np(s["dout"][b]), s["flags"]))
    want = [np.stack([p[0][i] for p in parts]) for i in range(3)] + [sum(p[0][3] for p in parts)]
    return want, [np.stack([p[1][i] for p in parts]) for i in range(3)]


def _check(s, got, tol):
    want, terms = _oracle(s)
    assert_close(to_np(got[3]), want[3], 1e-4, "dsink")
    for name, g, o, t in zip(("dq", "dkv", "dswa"), got, want, terms):
        g = to_np(g.float())
        if tol != TC_TOL:
            assert_close(g, o, tol, name)
            continue
        err, bound = np.abs(g - o), 2.2e-2 * t + 2.0 ** -8 * np.abs(o) + 1e-30
        assert bool(np.isfinite(g).all()), name
        worst = float((err / bound).max())
        at = np.unravel_index(int((err / bound).argmax()), err.shape)
        assert worst <= 1.0, f"{name}{at}: {worst:.2f} times the bound, {g[at]:.6g} for {o[at]:.6g} (T {t[at]:.3g})"


@pytest.mark.parametrize("B,Q,H,N,k,window,cap,pos,n_pad", [
    (1, 1, 1, 1, 1, 1, 1, [[0]], 0),                                   # one of everything
    (1, 4, 16, 300, 65, 33, 40, [[299, 5, 0, 600]], 3),                # ragged chunks, partial windows
    (2, 2, 9, 50, 31, 0, 0, [[4, 9], [1, 2]], 30),                     # no window
    (2, 3, 24, 40, 0, 17, 64, [[3, 90, 16], [0, 1, 63]], 0),           # window only
])
def test_fp32_path(B, Q, H, N, k, window, cap, pos, n_pad):
    s = _forward(_case(11, B, Q, H, N, k, window, cap, pos, torch.float32, n_pad))
    got = _backward(s)
    C.csa2_ctx_check()
    _check(s, got, F32_TOL)


@pytest.mark.parametrize("flags", [0, C.QNORM, C.KVNORM, C.ROPE, C.QNORM | C.KVNORM])
@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, BF16_TOL)], ids=["f32", "bf16"])
def test_flags(flags, dtype, tol):
    """Without both norms bf16 inputs run the fp32 path too (both norms alone: the tensor cores).
    Small values keep unnormalised logits of order one."""
    s = _forward(_case(12, 1, 3, 10, 60, 20, 9, 12, [[70, 3, 11]], dtype, 4, flags=flags, scale=0.25))
    _check(s, _backward(s), TC_TOL if dtype == torch.bfloat16 and flags == C.QNORM | C.KVNORM else tol)


@pytest.mark.parametrize("B,Q,H,N,k,window,cap,pos,n_pad", [
    (1, 1, 64, 700, 512, 128, 128, [[699]], 0),                        # one query
    (1, 3, 64, 300, 100, 128, 128, [[5, 127, 900]], 41),               # partial windows, ragged tile
    (2, 5, 40, 997, 301, 100, 140, [[9, 4000, 301, 99, 77], [0, 50, 3, 1000, 2]], 57),
    (1, 2, 1, 20, 1, 0, 0, [[3, 4]], 0),                               # one head, one key
    (1, 2, 100, 600, 300, 64, 64, [[70, 500]], 10),                    # two head passes, the second partial
    (1, 2, 128, 1500, 1024, 128, 128, [[1499, 20]], 0),
    (2, 3, 64, 50, 0, 128, 256, [[3, 200, 127], [0, 1, 5000]], 0),     # window only
])
def test_tensor_core_path(B, Q, H, N, k, window, cap, pos, n_pad):
    s = _forward(_case(13, B, Q, H, N, k, window, cap, pos, torch.bfloat16, n_pad))
    got = _backward(s)
    C.csa2_ctx_check()
    _check(s, got, TC_TOL)


def test_many_queries_share_rows():
    """More queries than SMs over few entries: long lists per row."""
    Q = 330
    s = _forward(_case(14, 1, Q, 64, 90, 40, 16, 64, [[20 + i for i in range(Q)]], torch.bfloat16, 7))
    got = _backward(s)
    C.csa2_ctx_check()
    _check(s, got, TC_TOL)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, TC_TOL)])
def test_dense(dtype, tol):
    s = _forward(_case(15, 2, 4, 20, 150, 150, 20, 30, [[5, 40, 0, 300], [7, 8, 9, 100]], dtype, dense=True))
    got = _backward(s)
    C.csa2_ctx_check()
    _check(s, got, tol)


@pytest.mark.parametrize("Q,H,k,window", [(200, 70, 300, 0), (153, 16, 200, 100), (40, 128, 700, 3)])
def test_whole_waves_and_a_shared_rest(Q, H, k, window):
    """More (head pass, query) pairs than CTAs, so some are dealt out whole and the tiles of the rest
    are shared, or fewer, so all are; queries of 0 to 6 tiles, some of none."""
    pos = [[(11 * i) % 400 - 5 for i in range(Q)]]
    s = _forward(_case(23, 1, Q, H, k, k, window, max(window, 1), pos, torch.bfloat16, dense=True))
    assert bool((s["nv"] == 0).any())
    got = _backward(s)
    C.csa2_ctx_check()
    _check(s, got, TC_TOL)
    for a, b in zip(got, _backward(s)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, TC_TOL)])
@pytest.mark.parametrize("sink", [True, False])
def test_queries_without_keys_and_repeated_indices(dtype, tol, sink):
    """Query 1 attends to nothing (no index, a negative position): its gradient is 0 even where its
    values are NaN; query 2 has the same index five times over."""
    s = _case(16, 1, 4, 64, 80, 12, 10, 16, [[30, -1, 31, 2]], dtype, 0, sink=sink)
    s["idx"][0, 1] = -1
    s["idx"][0, 2, :5] = 33
    _forward(s)
    clean = _backward(s)
    _check(s, clean, tol)
    assert not clean[0][0, 1].any()
    if not sink:
        assert torch.isinf(s["lse"][0, 1]).all()
        s["q"][0, 1] = float("nan")
        s["dout"][0, 1] = float("nan")
        again = _backward(s)
        C.csa2_ctx_check()
        for a, b in zip(again, clean):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_behind_empty_slots_are_not_read(dtype):
    """NaN and infinity in rows that no slot points to stay out of every gradient."""
    s = _forward(_case(17, 1, 3, 64, 100, 20, 8, 64, [[12, 20, 30]], dtype, 5))
    clean = _backward(s)
    used = set(s["idx"].flatten().tolist())
    free = [i for i in range(100) if i not in used]
    s["kv"][0, free] = float("nan")
    s["swa"][0, 40:] = float("inf")
    got = _backward(s)
    C.csa2_ctx_check()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])
    keep = sorted(used - {-1})
    assert torch.equal(got[1][0, keep], clean[1][0, keep])
    assert torch.equal(got[2][0, :31], clean[2][0, :31])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("chunk", [23, 8, 1])
def test_rows_that_no_query_attends_to_have_no_gradient(dtype, chunk):
    """Their gradient is 0 in one chunk and in several, where they hold NaN and infinity too."""
    Q = 23
    s = _forward(_case(25, 1, Q, 24, 300, 6, 5, 64, [[i for i in range(Q)]], dtype, 2))
    used = sorted(set(s["idx"].flatten().tolist()) - {-1})
    free = [i for i in range(300) if i not in set(used)]
    s["kv"][0, free[::2]] = float("nan")
    s["kv"][0, free[1::2]] = float("inf")
    s["swa"][0, Q:] = float("nan")
    dt = {torch.float32: C.F32, torch.bfloat16: C.BF16}[dtype]

    def size(q):
        return C._lib().csa2_attn_bwd_workspace_bytes(C.ctx(0), dt, dt, dt, dt, 1, q, 24, 6, 5, 300, 64, 7)

    # (in chunks of fewer queries the rows' sums are carried in 745 KB more)
    ws = torch.empty(size(chunk) + (4 * 512 * 364 + (1 << 16) if chunk < Q else 0), dtype=torch.uint8, device=DEV)
    got = _backward(s, ws=ws)
    C.csa2_ctx_check()
    assert not got[1][0, free].any() and not got[2][0, Q:].any()
    assert all(bool(torch.isfinite(x.float()).all()) for x in got)
    assert bool(got[1][0, used].float().abs().sum(-1).gt(0).all())


@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, TC_TOL)])
def test_chunked_workspace_and_same_bits(dtype, tol):
    """A workspace for a few queries at a time gives the gradients too (rows' sums carried in
    fp32); two calls give the same bits; one too small for a query is refused."""
    s = _forward(_case(18, 2, 23, 33, 70, 30, 12, 40, [[i * 3 for i in range(23)], [i + 9 for i in range(23)]], dtype, 3))
    one = _backward(s)
    two = _backward(s)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    dt = {torch.float32: C.F32, torch.bfloat16: C.BF16}[dtype]
    full = C._lib().csa2_attn_bwd_workspace_bytes(C.ctx(0), dt, dt, dt, dt, 2, 23, 33, 30, 12, 70, 40, 7)
    for part in (2, 5):
        ws = torch.empty(full // part, dtype=torch.uint8, device=DEV)
        got = _backward(s, ws=ws)
        C.csa2_ctx_check()
        _check(s, got, tol)
    with pytest.raises(C.Csa2Error) as e:
        _backward(s, ws=torch.empty(4096, dtype=torch.uint8, device=DEV))
    assert e.value.status == C.ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, TC_TOL)])
@pytest.mark.parametrize("part", [2, 6])
def test_chunked_dense_with_two_head_passes(dtype, tol, part):
    """Chunks of the dense form, more than 64 heads, a last chunk smaller than the others, and two calls
    at once on two streams with a workspace each: the same bits as one after the other."""
    s = _forward(_case(31, 1, 29, 100, 150, 150, 12, 40, [[i * 9 for i in range(29)]], dtype, dense=True))
    dt = {torch.float32: C.F32, torch.bfloat16: C.BF16}[dtype]
    size = C._lib().csa2_attn_bwd_workspace_bytes(C.ctx(0), dt, dt, dt, dt, 1, 29, 100, 150, 12, 150, 40, 7) // part
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    got = _backward(s, ws=ws[0])
    C.csa2_ctx_check()
    _check(s, got, tol)
    check, C._check = C._check, lambda fn, st: None if st == C.OK else (_ for _ in ()).throw(C.Csa2Error(fn, st))
    both, streams = [], [torch.cuda.Stream() for _ in ws]
    try:
        for w, stream in zip(ws, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                both.append(_backward(s, ws=w))
    finally:
        C._check = check
    torch.cuda.synchronize()
    C.csa2_ctx_check()
    for one in both:
        for a, b in zip(one, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_workspace_at_any_16_bytes(dtype):
    """A workspace of the size asked for, 16 bytes and more behind a 256-byte boundary: the same bits,
    and nothing around it is written; one 16-byte step smaller still runs (in chunks)."""
    s = _forward(_case(24, 1, 9, 64, 200, 90, 20, 32, [[40 + i for i in range(9)]], dtype, 8))
    ref = _backward(s)
    dt = {torch.float32: C.F32, torch.bfloat16: C.BF16}[dtype]
    need = C._lib().csa2_attn_bwd_workspace_bytes(C.ctx(0), dt, dt, dt, dt, 1, 9, 64, 90, 20, 200, 32, 7)
    raw = torch.full((need + 1024,), 0xA5, dtype=torch.uint8, device=DEV)
    assert raw.data_ptr() % 256 == 0
    for off in (0, 16, 48, 128, 240):
        raw.fill_(0xA5)
        for a, b in zip(_backward(s, ws=raw[off:off + need]), ref):
            assert torch.equal(a, b)
        C.csa2_ctx_check()
        assert bool((raw[:off] == 0xA5).all()) and bool((raw[off + need:] == 0xA5).all()), off
    raw.fill_(0xA5)
    first = _backward(s, ws=raw[16:need])                    # (the same chunks wherever it begins)
    C.csa2_ctx_check()
    assert bool((raw[:16] == 0xA5).all()) and bool((raw[need:] == 0xA5).all())
    for a, b in zip(_backward(s, ws=raw[256:240 + need]), first):
        assert torch.equal(a, b)
    with pytest.raises(C.Csa2Error) as e:
        _backward(s, ws=raw[8:8 + need])
    assert e.value.status == C.ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_out_of_range_index_is_flagged(dtype):
    s = _forward(_case(19, 1, 2, 64, 50, 6, 4, 8, [[9, 10]], dtype))
    clean_idx = s["idx"].clone()
    clean_idx[0, 0, 5] = -1
    s["idx"][0, 0, 5] = 50
    got = _backward(s)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE
    s["idx"] = clean_idx
    for a, b in zip(got, _backward(s)):
        assert torch.equal(a, b)
    C.csa2_ctx_check()


def test_unwanted_gradients_and_no_queries():
    s = _forward(_case(20, 1, 2, 8, 30, 5, 4, 8, [[9, 10]], torch.bfloat16))
    full = _backward(s)
    dq, dkv, dswa, dsink = _backward(s, want_dkv=False, want_dswa=False, want_dsink=False)
    assert dkv is None and dswa is None and dsink is None and torch.equal(dq, full[0])
    for n in ("q", "out", "dout", "lse", "q_pos", "idx"):
        s[n] = s[n][:, :0].contiguous()
    dq, dkv, dswa, dsink = _backward(s)
    C.csa2_ctx_check()
    assert dq.numel() == 0 and not dkv.any() and not dswa.any() and not dsink.any()


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("window", [0, 4])
def test_no_sequences(dense, window):
    """B = 0: the sink's gradient, which has no batch axis, is 0 (the buffer held NaN)."""
    s = _case(26, 1, 2, 8, 30, 5, window, 8, [[9, 10]], torch.bfloat16, dense=dense)
    for n in ("q", "kv", "swa", "q_pos", "dout", "nv" if dense else "idx"):
        s[n] = s[n][:0].contiguous()
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((0, 2, 8), device=DEV)
    dsink = torch.full((8,), float("nan"), device=DEV)
    got = _backward(s, dsink=dsink)
    C.csa2_ctx_check()
    assert [x.numel() for x in got[:3]] == [0, 0, 0] and got[3] is dsink and not dsink.any()


@pytest.mark.parametrize("dt,dtype", [(C.F32, torch.float32), (C.BF16, torch.bfloat16)])
@pytest.mark.parametrize("dense", [False, True])
def test_cache_without_entries(dt, dtype, dense):
    """N = 0 and no window through the C entry (the cache has an address, but no entry yet): gradients
    of 0 beside the sink's, and an index into the cache is flagged, as in the forward pass."""
    Q, H, k = 3, 8, 5
    q, dout = (W.normal_tensor((1, Q, H, 512), 27, i, dtype, DEV) for i in (1, 2))
    out, sink = torch.zeros_like(q), W.normal_tensor((H,), 27, 3, torch.float32, DEV)
    lse = sink.expand(1, Q, H).contiguous()
    pos = torch.zeros(1, Q, dtype=torch.int64, device=DEV)
    sel = torch.zeros(1, Q, dtype=torch.int64, device=DEV) if dense else torch.full((1, Q, k), -1, dtype=torch.int32, device=DEV)
    kv = torch.zeros(512, device=DEV)
    dq, dsink = torch.full_like(q, float("nan")), torch.full((H,), float("nan"), device=DEV)
    ws = torch.empty(C._lib().csa2_attn_bwd_workspace_bytes(C.ctx(0), dt, dt, dt, dt, 1, Q, H, k, 0, 0, 0, 7),
                     dtype=torch.uint8, device=DEV)
    p = [t.data_ptr() for t in (q, kv, sel, pos, sink, out, dout, lse, dq, dsink, ws)]

    def call():
        torch.cuda.synchronize()
        fn = C._lib().csa2_dense_attn_bwd if dense else C._lib().csa2_sparse_attn_bwd
        return fn(C.ctx(0), p[0], dt, p[1], dt, 0, p[2], k, None, dt, 0, 0, 0, p[3], p[4], p[5], p[6], dt, p[7], 1, Q, H, 512,
                  10000.0, 7, p[8], None, None, p[9], p[10], ws.numel(), None)

    assert call() == C.OK
    C.csa2_ctx_check()
    assert not dq.any() and not dsink.any()
    sel.view(-1)[1] = 1
    assert call() == C.OK
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_DEVICE
    assert not dq.any()


@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, TC_TOL)])
@pytest.mark.parametrize("base", [0.05, 1.0, 500000.0])
def test_any_rope_base(dtype, tol, base, monkeypatch):
    """The same angles as the forward pass for any base; one below 1 turns some pairs more than once a
    position.  The weights go by the same angles.  (The call takes the base as a 32-bit number.)"""
    s = _case(28, 1, 3, 20, 90, 40, 9, 12, [[70, 3, 11]], dtype, 4)
    kw = dict(window=9, rope_base=base)
    s["out"], s["lse"] = C.csa2_sparse_attn(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], want_lse=True, **kw)
    got = C.csa2_sparse_attn_bwd(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], s["out"], s["lse"], s["dout"], **kw)
    w, _ = C.csa2_attn_mass(s["q"], s["kv"], s["q_pos"], s["lse"], idx=s["idx"], want_weights=True, rope_base=base)
    C.csa2_ctx_check()
    base, oracle = float(np.float32(base)), G.attn_bwd
    monkeypatch.setattr(G, "attn_bwd", lambda *a: oracle(*a, base=base))
    _check(s, got, tol)
    ow, _ = G.attn_mass(to_np(s["q"][0]), to_np(s["kv"][0]), to_np(s["idx"][0]), to_np(s["q_pos"][0]), to_np(s["lse"][0]), base=base)
    assert_close(to_np(w[0]), ow, 5e-5, "weights")


@pytest.mark.parametrize("dtype,tol", [(torch.float32, F32_TOL), (torch.bfloat16, TC_TOL)])
def test_window_ring_that_begins_elsewhere(dtype, tol, monkeypatch):
    """swa_pos0 other than 0, positions before it among the window's."""
    s = _case(29, 2, 3, 20, 60, 12, 20, 32, [[70, 9, 25], [40, 44, 3]], dtype, 4)
    kw = dict(window=20, swa_pos0=21)
    s["out"], s["lse"] = C.csa2_sparse_attn(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], want_lse=True, **kw)
    got = C.csa2_sparse_attn_bwd(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], s["out"], s["lse"], s["dout"], **kw)
    C.csa2_ctx_check()
    oracle = G.attn_bwd
    monkeypatch.setattr(G, "attn_bwd", lambda q, kv, sel, swa, pos0, *a: oracle(q, kv, sel, swa, 21, *a))
    _check(s, got, tol)


F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("q_dt,kv_dt,swa_dt,out_dt", [(H, F, H, H), (H, H, F, H), (H, H, H, F), (F, H, H, H), (F, H, F, H),
                                                      (H, F, F, F), (F, F, H, F), (F, F, F, H)])
def test_mixed_types(q_dt, kv_dt, swa_dt, out_dt):
    """Any mixture runs in fp32 on the CUDA cores; each gradient has its tensor's type, and one rounding
    of it more where that is bf16."""
    s = _case(30, 1, 3, 20, 90, 40, 9, 12, [[70, 3, 11]], F, 4)
    s.update(q=s["q"].to(q_dt), kv=s["kv"].to(kv_dt), swa=s["swa"].to(swa_dt), dout=s["dout"].to(out_dt))
    s["out"], s["lse"] = C.csa2_sparse_attn(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], window=9, want_lse=True,
                                            out=torch.empty(s["q"].shape, dtype=out_dt, device=DEV))
    got = _backward(s)
    C.csa2_ctx_check()
    assert [g.dtype for g in got] == [q_dt, kv_dt, swa_dt, F]
    _check(s, got, BF16_TOL)


def test_captured_and_on_another_stream():
    """A captured call, replayed after its inputs changed in place, equals an eager call."""
    s = _forward(_case(21, 1, 5, 64, 200, 90, 20, 32, [[40, 41, 42, 43, 44]], torch.bfloat16, 8))
    ref = _backward(s)
    ws = torch.empty(C._lib().csa2_attn_bwd_workspace_bytes(C.ctx(0), 1, 1, 1, 1, 1, 5, 64, 90, 20, 200, 32, 7),
                     dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(x) for x in ref]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    kw = dict(dq=outs[0], dkv=outs[1], dswa=outs[2], dsink=outs[3], ws=ws)
    check, C._check = C._check, lambda fn, st: None if st == C.OK else (_ for _ in ()).throw(C.Csa2Error(fn, st))
    try:
        with torch.cuda.graph(graph, stream=stream):
            _backward(s, **kw)
    finally:
        C._check = check
    s["dout"].mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, _backward(s)):
        assert torch.equal(a, b)
    C.csa2_ctx_check()


def test_expired_wait_is_reported_and_the_context_stays_usable():
    """The image producer issues nothing: every role's bounded wait expires, the call reports a
    timeout, and the next call is right."""
    s = _forward(_case(22, 1, 2, 64, 200, 90, 20, 32, [[40, 41]], torch.bfloat16))
    ref = _backward(s)
    C.csa2_ctx_check()
    C.csa2_ctx_test_stall_next(2_000_000)
    _backward(s)
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_TIMEOUT
    for a, b in zip(ref, _backward(s)):
        assert torch.equal(a, b)
    C.csa2_ctx_check()
