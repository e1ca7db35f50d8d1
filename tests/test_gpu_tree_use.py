"""Drafted trees as a server runs them: more groups than the GPU takes at once, captured graphs, several
streams, rows that hold no numbers, and a kernel whose rows never come.  Tolerances as in
tests/test_gpu_tree.py."""
import contextlib

import pytest
import torch

from compressed_sparse_attention_06_gb300 import csa2 as C
from compressed_sparse_attention_06_gb300 import workloads as W
from tests.test_gpu_tree import BF, DEV, F32, Case

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def _unguarded():
    """Calls without the guards' look at the buffers after each, which waits for the GPU."""
    check, C._check = C._check, lambda fn, st: None if st == C.OK else pytest.fail(fn)
    try:
        yield
    finally:
        C._check = check


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("B,T,H,N,k,pad,dense", [
    (1, 80, 64, 2000, 1500, 1400, False),      # a round of whole groups and four that are dealt out, some of them short
    (1, 155, 20, 3000, 2040, 2039, False),     # two rounds and three
    (7, 88, 16, 1400, 0, 0, True),             # the nodes of a group see different entries
    (3, 5, 128, 5000, 0, 0, True),             # no whole round, a node a group
    (1, 1, 3, 9000, 2048, 0, False),           # one group over all of the GPU
])
def test_groups_in_rounds_and_shares(kind, B, T, H, N, k, pad, dense):
    c = Case(91, B, T, H, N, k, kind, page=64, pad=pad, dense=dense, unused=T // 9)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(out, lse, **BF)
    again, la = c.run(out_dtype=torch.float32)
    assert torch.equal(out, again) and torch.equal(lse, la)
    half, _ = c.run()
    assert torch.equal(half, out.to(torch.bfloat16))


@pytest.mark.parametrize("kind,dt", [("f32", torch.float32), ("bf16", torch.bfloat16), ("fp4", torch.bfloat16)])
@pytest.mark.parametrize("window", [0, 12])
def test_no_entries_and_repeated_entries(kind, dt, window):
    c = Case(92, 2, 5, 24, 40, 0, kind, dt=dt, window=window)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    tol = F32 if dt == torch.float32 else BF
    c.check(out, lse, **tol)
    if window == 0:
        assert not out.any() and torch.equal(lse, c.sink.expand_as(lse))
    c = Case(92, 2, 5, 24, 40, 30, kind, dt=dt, window=window)
    c.kw["idx"][:, :, 10:20] = c.kw["idx"][:, :, :1]                   # an entry counts as often as it is named
    c.sel[:, :, 10:20] = c.sel[:, :, :1]
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(out, lse, **tol)


@pytest.mark.parametrize("kind,dt", [("f32", torch.float32), ("bf16", torch.bfloat16)])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_without_numbers_reach_only_who_attends(kind, dt, dense, bad):
    """A draft, a ring row and an entry with a NaN or an infinity: the nodes that attend to it get NaN, the
    others the same bits as before, those of the same group too."""
    B, T, H, N, k, win = 2, 8, 16, 200, 0 if dense else 60, 10
    c = Case(93, B, T, H, N, k, kind, dt=dt, window=win, dense=dense, lens=[50, 4])
    c.parent = torch.tensor([[-1, 0, 1, 0, 3, 4, 5, 3]] * B, dtype=torch.int32, device=DEV)     # 0-1-2, 0-3-4-5-6, 3-7
    out, lse = c.run()
    C.csa2_ctx_check()

    def check(hit):
        o, l = c.run()
        C.csa2_ctx_check()
        hit = torch.tensor(hit, device=DEV).expand(B, T)
        assert bool(torch.isnan(o[hit].float()).all()) and bool(torch.isnan(l[hit]).all())
        assert torch.equal(o[~hit], out[~hit]) and torch.equal(l[~hit], lse[~hit])

    keep = c.draft.clone()
    c.draft[:, 4, 77] = bad
    check([[i in (4, 5, 6) for i in range(T)]])
    c.draft = keep
    keep = c.swa.clone()
    # the ring's row of position len - win + 2 (sequence 0): the nodes of depth 0 and 1 see it
    c.swa[0, (50 - win + 2 - c.kw["swa_pos0"]) % c.swa.shape[1], 500] = bad
    check([[i in (0, 1, 3) for i in range(T)], [False] * T])
    c.swa = keep
    if dense:
        c.kv[1, N - 1, 3] = bad
        hit = [[False] * T, [len(c.sel[1][i]) == N for i in range(T)]]
    else:
        c.kv[1, int(c.sel[1][5][7]), 3] = bad
        hit = [[False] * T, [bool((c.sel[1][i] == c.sel[1][5][7]).any()) for i in range(T)]]
    check(hit)


@pytest.mark.parametrize("flags", [0, 1, 2, 4, 5, 7])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e30])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_without_numbers_whatever_the_norms(flags, bad, dt):
    """The same with and without the norms: an infinity's logits may be minus infinity, and a large value's
    square no number in fp32.  A query's head without numbers is alone in it."""
    B, T, H, N, win = 1, 6, 16, 50, 4
    c = Case(96, B, T, H, N, 30, "f32" if dt == torch.float32 else "bf16", dt=dt, window=win, lens=[20])
    c.parent = torch.tensor([[-1, 0, 0, 2, 3, -2]], dtype=torch.int32, device=DEV)               # 0-1, 0-2-3-4
    out, lse = c.run(flags=flags, out_dtype=torch.float32)
    C.csa2_ctx_check()

    def check(hit):
        o, l = c.run(flags=flags, out_dtype=torch.float32)
        C.csa2_ctx_check()
        assert bool(torch.isnan(o[0, hit]).all()) and bool(torch.isnan(l[0, hit]).all())
        rest = [i for i in range(T) if i not in hit]
        assert torch.equal(o[0, rest], out[0, rest]) and torch.equal(l[0, rest], lse[0, rest])

    def with_(name, at):
        keep = getattr(c, name).clone()
        getattr(c, name)[at] = bad
        return keep

    finite = abs(bad) < 1e38
    if not finite or flags & C.KVNORM:
        for name, at, hit in (("draft", (0, 2, 77), [2, 3, 4]), ("swa", (0, (19 - c.kw["swa_pos0"]) % c.swa.shape[1], 5), [0, 1, 2, 3]),
                              ("kv", (0, int(c.sel[0][1][3]), 500), [i for i in range(5) if (c.sel[0][i] == c.sel[0][1][3]).any()])):
            keep = with_(name, at)
            check(hit)
            setattr(c, name, keep)
    if not finite or flags & C.QNORM:
        keep = with_("q", (0, 3, 7, 100))
        o, l = c.run(flags=flags, out_dtype=torch.float32)
        C.csa2_ctx_check()
        hit = torch.zeros(1, T, H, dtype=torch.bool, device=DEV)
        hit[0, 3, 7] = True
        assert bool(torch.isnan(o[hit]).all()) and bool(torch.isnan(l[hit]).all())
        assert torch.equal(o[~hit], out[~hit]) and torch.equal(l[~hit], lse[~hit])
        c.q = keep


@pytest.mark.parametrize("kind,dt", [("f32", torch.float32), ("bf16", torch.bfloat16)])
@pytest.mark.parametrize("k", [1, 100])
def test_nothing_but_rows_without_numbers(kind, dt, k):
    c = Case(95, 1, 2, 8, 128, k, kind, dt=dt, window=0)
    c.kv[:] = float("nan")
    for sink in (None, c.sink):
        out, lse = c.run(sink=sink)
        C.csa2_ctx_check()
        assert bool(torch.isnan(out.float()).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("kind,dense", [("bf16", True), ("fp4", False)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_outputs_off_a_sector(kind, dense, dt):
    """An output that starts 16 bytes behind a multiple of 32 gets the same values."""
    c = Case(98, 2, 11, 24, 700, 0 if dense else 300, kind, page=16, dense=dense)
    want, _ = c.run(out_dtype=dt)
    n, off = want.numel(), 16 // want.element_size()
    buf = torch.full((n + 4 * off,), 7.0, dtype=dt, device=DEV)
    out = buf[off:off + n].view(want.shape)
    assert out.data_ptr() % 32 == 16
    c.run(out=out)
    C.csa2_ctx_check()
    assert torch.equal(out, want) and bool((buf[:off] == 7).all()) and bool((buf[off + n:] == 7).all())


@pytest.mark.parametrize("kind,T,k,dense", [("bf16", 1, 2048, False), ("fp4", 3, 1500, False), ("bf16", 19, 1400, True)])
@pytest.mark.parametrize("off", [16, 32, 48, 240])
def test_workspace_off_a_sector(kind, T, k, dense, off):
    """Groups that are dealt out leave partial outputs in the workspace, which may begin at any multiple of
    16 bytes: the same bits from each, and nothing written beside it."""
    c = Case(97, 1, T, 24, 3000 if not dense else k, 0 if dense else k, kind, page=16, dense=dense)
    need = C.load().csa2_tree_attn_workspace_bytes(C.ctx(c.q.device.index), C.BF16, C.FP4_E4M3x16 if kind == "fp4" else C.BF16,
                                                   C.BF16, 1, T, 24, k, c.kw["window"], int(dense), C.ATTN_DEFAULT)
    buf = torch.full((need + 512,), 7, dtype=torch.uint8, device=DEV)
    assert buf.data_ptr() % 256 == 0
    want, lw = c.run(ws=buf[:need])
    out, lse = c.run(ws=buf.fill_(7)[off:off + need])
    C.csa2_ctx_check()
    assert torch.equal(out, want) and torch.equal(lse, lw)
    assert bool((buf[:off] == 7).all()) and bool((buf[off + need:] == 7).all())


def test_captured_and_replayed():
    """Two graphs captured over one workspace, replayed in turn with other inputs, lengths and trees."""
    cases = [Case(94 + i, 2, 9, 32, 700, 300, "bf16", page=64, lens=[10, 999]) for i in range(4)]
    a, b = cases[0], Case(99, 3, 80, 8, 900, 0, "fp4", page=16, dense=True)

    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)

    def bind(c):
        B, T = c.parent.shape
        pos, path = torch.empty(B, T, dtype=torch.int64, device=DEV), torch.empty(B, T, T, dtype=torch.int16, device=DEV)
        out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], dtype=torch.float32, device=DEV)

        def call():
            C.csa2_tree_plan(c.parent, c.len, pos=pos, path=path)
            C.csa2_tree_attn(c.q, c.kv, pos, path, c.len, c.swa, c.draft, **c.kw, sink=c.sink, out=out, lse=lse, ws=ws)
        return call, out, lse

    graphs = []
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in (a, b):
        call, out, lse = bind(c)
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with _unguarded(), torch.cuda.graph(g, stream=s):
            call()
        graphs.append((g, out, lse))
    for c in cases:
        swa_pos0 = c.kw["swa_pos0"]
        for x in ("q", "kv", "swa", "draft", "sink", "len", "parent"):
            getattr(a, x).copy_(getattr(c, x))
        a.kw["table"].copy_(c.kw["table"])
        a.kw["idx"].copy_(c.kw["idx"])
        c.kw["swa_pos0"] = a.kw["swa_pos0"]                            # (an argument: it stays as captured)
        want = c.run()
        c.kw["swa_pos0"] = swa_pos0
        want_b = b.run()
        for g, _, _ in graphs:
            g.replay()
        C.csa2_ctx_check()
        for (_, out, lse), (o, l) in zip(graphs, (want, want_b)):
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_streams_at_once():
    cases = [Case(101 + i, 2, 20, 64, 3000, 1000, kind, page=64) for i, kind in enumerate(("bf16", "fp4", "bf16"))]
    want = [c.run() for c in cases]
    C.csa2_ctx_check()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    with _unguarded():
        for _ in range(4):
            for c, s in zip(cases, streams):
                with torch.cuda.stream(s):
                    got.append(c.run())
        torch.cuda.synchronize()
    C.csa2_ctx_check()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(l, want[i % 3][1])


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_rows_written_just_before(kind):
    """Cache rows written and copied, a path committed and the attention queued behind one another without a
    wait, with other rows every time: each call reads what the ones before it wrote."""
    B, T, N, page = 3, 6, 256, 16
    c = Case(121, B, T, 32, N, 100, kind, page=page, lens=[300, 9, 4000], window=40, spare=T)
    pos, path = C.csa2_tree_plan(c.parent, c.len)
    n_pages = B * N // page
    table = torch.arange(n_pages, dtype=torch.int32, device=DEV).view(B, -1)
    first, count = torch.zeros(B, dtype=torch.int64, device=DEV), torch.full((B,), N, device=DEV)
    leaf = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    leaf[0] = 0
    half = torch.arange(n_pages, dtype=torch.int32, device=DEV).view(-1, 2)          # every even page over the next one
    steps = []
    for i in range(6):
        x = W.normal_tensor((B, N, 512), 130 + i, 1, torch.float32, DEV) * (1.0 + i)
        steps.append((C.csa2_fp4_pack(x) if kind == "fp4" else x.to(torch.bfloat16),
                      W.normal_tensor((B, T, 512), 140 + i, 1, torch.bfloat16, DEV) * (6.0 - i)))
    pool = torch.zeros(n_pages, page, steps[0][0].shape[-1], dtype=steps[0][0].dtype, device=DEV)
    swa, length = c.swa.clone(), torch.zeros_like(c.len)
    kw = dict(idx=c.kw["idx"], window=40, swa_pos0=c.kw["swa_pos0"], table=table, sink=c.sink, want_lse=True)

    def step(rows, draft, wait):
        C.csa2_page_write(pool, table, rows, first, count)
        wait()
        C.csa2_page_copy(pool, half)
        wait()
        a = C.csa2_tree_attn(c.q, pool, pos, path, c.len, swa, draft, **kw)
        wait()
        C.csa2_tree_commit(draft, pos, path, c.len, leaf, swa, swa_pos0=kw["swa_pos0"], new_len=length)
        wait()
        after = C.csa2_tree_plan(c.parent, length)
        wait()
        b = C.csa2_tree_attn(c.q, pool, *after, length, swa, draft, **kw)
        wait()
        return *a, *b

    want = [step(r, d, torch.cuda.synchronize) for r, d in steps]
    swa.copy_(c.swa)
    pool.zero_()
    torch.cuda.synchronize()
    with _unguarded():
        got = [step(r, d, lambda: None) for r, d in steps]
    torch.cuda.synchronize()
    C.csa2_ctx_check()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind,dense", [("bf16", False), ("bf16", True), ("fp4", False)])
def test_queries_that_never_come_time_out(kind, dense):
    c = Case(111, 2, 12, 32, 900, 0 if dense else 500, kind, page=64, dense=dense)
    want, lw = c.run()
    C.csa2_ctx_check()
    C.csa2_ctx_test_stall_next(1 << 27)
    c.run()
    with pytest.raises(C.Csa2Error) as e:
        C.csa2_ctx_check()
    assert e.value.status == C.ERR_TIMEOUT
    out, lse = c.run()
    C.csa2_ctx_check()
    assert torch.equal(out, want) and torch.equal(lse, lw)
