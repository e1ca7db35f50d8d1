"""Backward pass of the compressor against the f64 gradient oracle, and the whole chain compressor
-> attention -> attention's backward -> compressor's backward against central differences.

Tolerances (|g - o| <= tol (|o| + rms)): fp32 sums of at most 256 rows and 1,024 channels and one
exp a row: 256 * 2^-24 = 1.5e-5 at the worst of linear growth; 5e-5.  A bf16 gradient row is
rounded once more: bf16 keeps 8 significant bits, so a value in [1, 2) lies at most 2^-8 from
the nearest one, 2^-8 of |o|."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,n,c,m,overlap,prev,bias,flags", [
    (1, 1, 512, 1, False, False, False, 3),
    (2, 12, 512, 2, False, False, True, 3),
    (1, 8, 512, 4, True, False, True, 3),
    (2, 20, 512, 4, True, True, True, 1),
    (1, 9, 128, 3, True, True, False, 2),
    (1, 15, 1024, 5, True, True, True, 3),          # ten rows: read again
    (2, 384, 512, 128, False, False, True, 3),      # the heavily compressed form
    (1, 4, 512, 4, True, True, True, 0),            # one entry
    (3, 4000, 128, 2, False, False, True, 3),       # more entries than CTAs
])
def test_compress_bwd(dtype, B, n, c, m, overlap, prev, bias, flags):
    def t(i, *shape, dt=dtype):
        return W.normal_tensor(shape, 61, i, dt, DEV)

    ca, za = t(1, B, n, c), t(2, B, n, c)
    cb, zb = (t(3, B, n, c), t(4, B, n, c)) if overlap else (None, None)
    pc, pz = (t(5, B, m, c), t(6, B, m, c)) if prev else (None, None)
    ba = t(7, m, c, dt=torch.float32) if bias else None
    bb = t(8, m, c, dt=torch.float32) if bias and overlap else None
    dout = t(9, B, n // m, c)
    pos0 = torch.tensor([40 + 1000003 * b for b in range(B)], dtype=torch.int64, device=DEV)
    g = C.csa2_compress_bwd(ca, za, m, dout, cb=cb, zb=zb, ba=ba, bb=bb, prev_cb=pc, prev_zb=pz, pos0=pos0, flags=flags)
    C.csa2_ctx_check()
    again = C.csa2_compress_bwd(ca, za, m, dout, cb=cb, zb=zb, ba=ba, bb=bb, prev_cb=pc, prev_zb=pz, pos0=pos0,
                                flags=flags)
    tol = TOL + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    sums = {"Ba": 0.0, "Bb": 0.0}
    for b in range(B):
        opt = dict(Ba=None if ba is None else to_np(ba), Bb=None if bb is None else to_np(bb))
        if overlap:
            opt.update(Cb=to_np(cb[b]), Zb=to_np(zb[b]))
        if prev:
            opt.update(prev_Cb=to_np(pc[b]), prev_Zb=to_np(pz[b]))
        w = G.compress_bwd(to_np(ca[b]), to_np(za[b]), m, to_np(dout[b]), flags=flags, pos0=int(pos0[b]), **opt)
        for name, got in (("Ca", g.dca), ("Za", g.dza), ("Cb", g.dcb), ("Zb", g.dzb), ("prev_Cb", g.dprev_cb),
                          ("prev_Zb", g.dprev_zb)):
            if got is not None:
                assert_close(to_np(got[b].float()), w[name], tol, f"{name} of stream {b}")
        sums = {k: v + w[k] for k, v in sums.items()}
    if bias:
        assert_close(to_np(g.dba), sums["Ba"], TOL, "Ba")
        if overlap:
            assert_close(to_np(g.dbb), sums["Bb"], TOL, "Bb")
    for x, y in zip(g, again):
        assert (x is None) == (y is None) and (x is None or torch.equal(x, y))


@pytest.mark.parametrize("c,m,overlap,entries", [
    (128, 5, False, 1217), (128, 5, True, 1300), (128, 12, False, 2500), (256, 6, False, 1500), (256, 7, True, 1217),
    (384, 7, False, 1700), (128, 12, True, 1217), (512, 5, False, 1300)])
def test_other_windows_with_more_entries_than_ctas(c, m, overlap, entries, _guarded_buffers):
    """Windows that are not compiled for their size, narrow rows, biases, and more entries than 1,216
    CTAs: every CTA's slab lies inside the workspace (guard bytes around it), and every gradient and
    bias sum is the oracle's.  A bias sum adds a run's terms, then at most 2,500 / 32 = 79 slabs, then
    32 sums: about 115 additions one behind the other of partial sums of at most 4 rms of the
    result, each off by 2^-24 of it, so sqrt(115) * 4 * 2^-24 = 2.6e-6 rms beside the terms' own
    errors (independent, so they add up as the terms do); TOL holds for both."""
    def t(i, *shape, dt=torch.float32):
        return W.normal_tensor(shape, 64, i, dt, DEV)

    n = entries * m
    ca, za, dout = t(1, n, c), t(2, n, c), t(3, entries, c)
    cb, zb = (t(4, n, c), t(5, n, c)) if overlap else (None, None)
    ba, bb = t(6, m, c), t(7, m, c) if overlap else None
    g = C.csa2_compress_bwd(ca, za, m, dout, cb=cb, zb=zb, ba=ba, bb=bb, flags=C.W_NORM | C.W_ROPE)
    C.csa2_ctx_check()
    assert _guarded_buffers.checked > 0
    opt = dict(Ba=to_np(ba))
    if overlap:
        opt.update(Cb=to_np(cb), Zb=to_np(zb), Bb=to_np(bb))
    w = G.compress_bwd(to_np(ca), to_np(za), m, to_np(dout), flags=C.W_NORM | C.W_ROPE, **opt)
    for name, got in (("Ca", g.dca), ("Za", g.dza), ("Cb", g.dcb), ("Zb", g.dzb)):
        if got is not None:
            assert_close(to_np(got), w[name], TOL, name)
    for name, got in (("Ba", g.dba), ("Bb", g.dbb)):
        if got is not None:
            assert_close(to_np(got), w[name], TOL, name)


def test_unbatched_and_empty():
    ca, za = (W.normal_tensor((8, 512), 62, i, torch.float32, DEV) for i in (1, 2))
    dout = W.normal_tensor((4, 512), 62, 3, torch.float32, DEV)
    one = C.csa2_compress_bwd(ca, za, 2, dout)
    bat = C.csa2_compress_bwd(ca[None].contiguous(), za[None].contiguous(), 2, dout[None].contiguous())
    assert torch.equal(one.dca, bat.dca[0]) and torch.equal(one.dza, bat.dza[0]) and one.dba is None
    ba = torch.zeros(2, 512, device=DEV)
    g = C.csa2_compress_bwd(ca[:0], za[:0], 2, dout[:0], ba=ba)
    C.csa2_ctx_check()
    assert g.dca.numel() == 0 and not g.dba.any()


def test_layer_backward_matches_differences():
    """The training step of a layer -- compress the tokens into entries, attend over a selection of
    them and the window -- differentiated by the library in fp32, against central differences of
    the f64 oracle along random directions of each input.  The library's gradient is off by
    fp32 rounding, about 1e-5 of its norm; the differences (step 1e-4 along unit directions) by
    the cube term, about 1e-8: 1e-3 of the gradient's norm is allowed."""
    m, n, H, Q, window = 4, 64, 8, 3, 6
    N = n // m

    def t(i, *shape):
        return W.normal_tensor(shape, 63, i, torch.float32, DEV)

    x = dict(Ca=t(1, n, 512), Za=t(2, n, 512), Cb=t(3, n, 512), Zb=t(4, n, 512), Ba=t(5, m, 512), Bb=t(6, m, 512),
             q=t(7, 1, Q, H, 512), swa=t(8, 1, 16, 512), sink=t(9, H))
    pos = torch.tensor([[63, 50, 30]], dtype=torch.int64, device=DEV)
    idx = torch.tensor([[[0, 3, 7, 15, 9], [2, 5, 11, -1, -1], [0, 1, 2, 3, 6]]], dtype=torch.int32, device=DEV)
    dout = t(10, 1, Q, H, 512)
    kv = C.csa2_compress(x["Ca"], x["Za"], m, cb=x["Cb"], zb=x["Zb"], ba=x["Ba"], bb=x["Bb"], flags=C.W_NORM | C.W_ROPE)
    out, lse = C.csa2_sparse_attn(x["q"], kv[None].contiguous(), idx, x["swa"], pos, x["sink"], window=window, want_lse=True)
    att, com = P.layer_backward(x["q"], kv[None].contiguous(), idx, x["swa"], pos, x["sink"], out, lse, dout, x["Ca"],
                                x["Za"], m, cb=x["Cb"], zb=x["Zb"], ba=x["Ba"], bb=x["Bb"], window=window,
                                write_flags=C.W_NORM | C.W_ROPE)
    C.csa2_ctx_check()
    got = dict(Ca=com.dca, Za=com.dza, Cb=com.dcb, Zb=com.dzb, Ba=com.dba, Bb=com.dbb, q=att[0], swa=att[2], sink=att[3])
    f = {k: to_np(v) for k, v in x.items()}

    def loss(v):
        e = O.compress_write(O.compress(v["Ca"], v["Za"], m, v["Ba"], v["Cb"], v["Zb"], v["Bb"]), O.NORM_W | O.ROPE_W, m)
        o = [O.sparse_attn(v["q"][0, i], e, to_np(idx[0, i]), v["swa"][0], 0, int(pos[0, i]), v["sink"], window)[0]
             for i in range(Q)]
        return float((np.array(o) * to_np(dout[0])).sum())

    rng = np.random.default_rng(4)
    for k in f:
        grad = to_np(got[k])
        for _ in range(2):
            d = rng.standard_normal(f[k].shape)
            d /= np.linalg.norm(d)
            h = 1e-4
            want = (loss({**f, k: f[k] + h * d}) - loss({**f, k: f[k] - h * d})) / (2 * h)
            assert abs(float((grad * d).sum()) - want) <= 1e-3 * np.linalg.norm(grad) + 1e-6, k


@pytest.mark.parametrize("m", [2, 5])
@pytest.mark.parametrize("base", [0.05, 1.0, 500000.0])
def test_any_rope_base(m, base):
    """(The call takes the base as a 32-bit number: so does the oracle.)"""
    ca, za = (W.normal_tensor((4 * m, 512), 66, i, torch.float32, DEV) for i in (1, 2))
    dout = W.normal_tensor((4, 512), 66, 3, torch.float32, DEV)
    g = C.csa2_compress_bwd(ca, za, m, dout, pos0=1000, rope_base=base, flags=C.W_NORM | C.W_ROPE)
    C.csa2_ctx_check()
    w = G.compress_bwd(to_np(ca), to_np(za), m, to_np(dout), flags=C.W_NORM | C.W_ROPE, pos0=1000,
                       base=float(np.float32(base)))
    assert_close(to_np(g.dca), w["Ca"], TOL, "Ca")
    assert_close(to_np(g.dza), w["Za"], TOL, "Za")


@pytest.mark.parametrize("m", [2, 5])
def test_compress_bwd_captured_and_on_another_stream(m):
    """A graph of the call, replayed after its inputs changed in place, and a call on a side stream give
    an eager call's bits; compiled and general window."""
    n, c = 40 * m, 256
    ca, za, dout = (W.normal_tensor((n if i < 3 else 40, c), 65, i, torch.bfloat16, DEV) for i in (1, 2, 3))
    ba = W.normal_tensor((m, c), 65, 4, torch.float32, DEV)
    ws = torch.empty(C._lib().csa2_compress_bwd_workspace_bytes(1, n, c, m, 0), dtype=torch.uint8, device=DEV)

    def call():
        return C.csa2_compress_bwd(ca, za, m, dout, ba=ba, flags=C.W_NORM | C.W_ROPE, ws=ws)

    graph = torch.cuda.CUDAGraph()
    check, C._check = C._check, lambda fn, st: None if st == C.OK else (_ for _ in ()).throw(C.Csa2Error(fn, st))
    try:
        with torch.cuda.graph(graph):
            held = call()
    finally:
        C._check = check
    dout.mul_(-3.0)
    za.add_(1.0 / 3.0)
    ba.neg_()
    graph.replay()
    torch.cuda.synchronize()
    eager = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        aside = call()
    torch.cuda.synchronize()
    C.csa2_ctx_check()
    for a, b, d in zip(held, eager, aside):
        assert (a is None and b is None and d is None) or (torch.equal(a, b) and torch.equal(b, d))
