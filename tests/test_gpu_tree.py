"""Drafted trees against the f64 oracle: plans, commits and the attention of every node.

Tolerances.  The fp32 path sums 512 products of |z| <= 23 and exponentials in fp32: 23 * 2^-22 for a
logit, so 1e-4 (|o| + rms), lse 1e-5, as the framework's other fp32 attention.  The tensor-core path
rounds q^ to bf16 (relative 2^-8 / sqrt(3) rms a term, so 2^-8 / sqrt(3) of a logit of unit terms) and
p to bf16 (the same of each addend); the addends' errors add up as root sums of squares, below
3.2e-3 of the rms of the node's o (q^ counted whole, though only its rotated dims are rounded), 1.6e-2 at five deviations, and half a bf16 step (2^-8) of the
output: 2e-2 (|o| + rms), lse 2e-3.  The rms is each node's own: o is a mean of as many rows as the
node attends to, so a node with few rows has larger o, and errors, than one with many."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_06_gb300 import csa2 as C
from compressed_sparse_attention_06_gb300 import pipeline as P
from compressed_sparse_attention_06_gb300 import workloads as W
from oracle import csa2_oracle as O
from oracle import csa2_oracle_draft as D
from tests.helpers import assert_close, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _tree(seed, B, T, unused=0):
    rng = np.random.default_rng(seed)
    par = np.array([[-1 if i == 0 or rng.random() < 0.15 else rng.integers(max(0, i - 6), i) for i in range(T)] for _ in range(B)])
    if unused:
        par[0, -unused:] = -2
    return torch.tensor(par, dtype=torch.int32, device=DEV)


def _rows(seed, shape, kind):
    """Cache rows of a kind and their values."""
    x = W.normal_tensor((*shape, 512), seed, 2, torch.float32, DEV) * 1.3
    if kind == "fp4":
        kv = C.csa2_fp4_pack(x)
        return kv, O.nvfp4_unpack(to_np(kv).reshape(-1, 288)).reshape(*shape, 512)
    kv = x.to(torch.bfloat16) if kind == "bf16" else x
    return kv, to_np(kv)


class Case:
    """Inputs of a call, and its entries as the oracle takes them (per sequence [N, 512])."""

    def __init__(self, seed, B, T, H, N, k, kind, dt=torch.bfloat16, window=128, page=0, dense=False, unused=0, lens=None, pad=0,
                 spare=0):
        rng = np.random.default_rng(seed)
        self.parent = _tree(seed, B, T, unused)
        lens = rng.integers(0, 5000, B) if lens is None else lens
        self.len = torch.tensor(lens, dtype=torch.int64, device=DEV)
        self.kw = dict(window=window, swa_pos0=int(rng.integers(0, 300)))
        self.q = W.normal_tensor((B, T, H, 512), seed, 1, dt, DEV)
        self.swa = W.normal_tensor((B, max(1, window + spare), 512), seed, 3, dt, DEV)
        self.draft = W.normal_tensor((B, T, 512), seed, 4, dt, DEV)
        self.sink = W.normal_tensor((H,), seed, 5, torch.float32, DEV)
        if page:
            mp = (N + page - 1) // page
            n_pages = B * mp + 3
            perm = rng.permutation(n_pages)
            table = perm[:B * mp].reshape(B, mp)
            table[:, :mp // 2] = table[0, :mp // 2]                    # a shared beginning
            self.table = torch.tensor(table, dtype=torch.int32, device=DEV)
            self.kv, v = _rows(seed, (n_pages, page), kind)
            self.entries = [v[table[b]].reshape(mp * page, 512)[:N] for b in range(B)]
        else:
            self.table = None
            self.kv, v = _rows(seed, (B, N), kind)
            self.entries = list(v)
        self.kw["table"] = self.table
        if dense:
            nv = rng.integers(0, N + 1, (B, T))
            nv[0, 0] = N
            self.sel = [[np.arange(n) for n in row] for row in nv]
            self.kw.update(n_visible=torch.tensor(nv, dtype=torch.int64, device=DEV), k_max=N)
        else:
            idx = np.full((B, T, k), -1)
            for b in range(B):
                for i in range(T):
                    n = min(N, k - (pad if (b + i) % 2 else 0))
                    idx[b, i, :n] = rng.permutation(N)[:n]
            self.sel = idx
            self.kw["idx"] = torch.tensor(idx, dtype=torch.int32, device=DEV) if k else None

    def run(self, **kw):
        pos, path = C.csa2_tree_plan(self.parent, self.len)
        return C.csa2_tree_attn(self.q, self.kv, pos, path, self.len, self.swa, self.draft,
                                **{**self.kw, "sink": self.sink, "want_lse": True, **kw})

    def check(self, out, lse, tol, ltol, sink=True, flags=7, base=10000.0):
        for b in range(self.q.shape[0]):
            o, l = D.tree_attn(to_np(self.q[b]), self.entries[b], self.sel[b], to_np(self.swa[b]), self.kw["swa_pos0"],
                               to_np(self.draft[b]), to_np(self.parent[b]), int(self.len[b]), to_np(self.sink) if sink else None,
                               self.kw["window"], flags=flags, base=base)
            for i in range(o.shape[0]):
                assert_close(to_np(out[b, i]), o[i], tol, f"out of node {i} of sequence {b}")
            if lse is not None:
                assert_close(to_np(lse[b]), l, ltol, f"lse of sequence {b}")


F32 = dict(tol=1e-4, ltol=1e-5)
BF = dict(tol=2e-2, ltol=2e-3)


@pytest.mark.parametrize("B,T", [(1, 1), (3, 2), (2, 33), (5, 64), (2, 256)])
def test_plan(B, T):
    par = _tree(T, B, T, unused=T // 8)
    if T == 256:
        par[1] = torch.arange(T) - 1                                   # one chain as deep as it gets
    lens = torch.arange(B, device=DEV) * 1000003
    pos, path = C.csa2_tree_plan(par, lens)
    C.csa2_ctx_check()
    for b in range(B):
        p, a = D.tree_plan(to_np(par[b]), int(lens[b]))
        assert np.array_equal(to_np(pos[b]), p) and np.array_equal(path[b].cpu().numpy(), a)


def test_plan_flags_what_is_no_tree():
    par = torch.tensor([[-1, 1, 0, 5], [-1, 0, 1, 2], [-1, -5, 1, 0]], dtype=torch.int32, device=DEV)
    pos, path = C.csa2_tree_plan(par, torch.tensor([7, -1, 0], device=DEV))
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert pos.tolist() == [[7, -1, 8, -1], [-1] * 4, [0, -1, -1, 1]]
    assert path[0, 2].tolist() == [0, 2, -1, -1] and (path[1] == -1).all()


@pytest.mark.parametrize("kind,dt", [("f32", torch.float32), ("bf16", torch.float32), ("fp4", torch.float32), ("f32", torch.bfloat16)])
@pytest.mark.parametrize("B,T,H,N,k,window,page,pad", [
    (1, 1, 1, 1, 1, 1, 0, 0), (2, 5, 16, 300, 65, 128, 16, 64), (1, 13, 17, 97, 33, 100, 7, 5), (2, 3, 128, 80, 64, 0, 0, 1),
    (1, 1, 64, 900, 512, 128, 64, 100), (3, 40, 8, 50, 0, 9, 0, 0),
])
def test_fp32_path(kind, dt, B, T, H, N, k, window, page, pad):
    c = Case(51, B, T, H, N, k, kind, dt=dt, window=window, page=page, pad=pad, unused=T // 5)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(out, lse, **F32)


@pytest.mark.parametrize("flags", [0, 1, 2, 4, 5])
@pytest.mark.parametrize("sink", [True, False])
def test_fp32_path_flags(flags, sink):
    c = Case(52, 2, 4, 20, 60, 30, "f32", dt=torch.float32, window=40, page=4)
    c.q *= 0.2
    out, lse = c.run(flags=flags, sink=c.sink if sink else None, rope_base=500.0)
    C.csa2_ctx_check()
    c.check(out, lse, **F32, sink=sink, flags=flags, base=500.0)


def test_fp32_dense():
    c = Case(53, 2, 6, 16, 333, 0, "f32", dt=torch.float32, page=16, dense=True)
    out, lse = c.run()
    C.csa2_ctx_check()
    c.check(out, lse, **F32)


BF_CASES = [
    (1, 1, 64, 900, 512, 128, 64, 100), (1, 1, 1, 1, 1, 1, 0, 0), (2, 7, 40, 300, 65, 128, 16, 64), (1, 13, 64, 97, 33, 100, 7, 5),
    (2, 3, 128, 400, 200, 128, 0, 1), (1, 9, 100, 300, 130, 37, 32, 0), (2, 40, 16, 500, 256, 128, 64, 100), (3, 20, 8, 50, 0, 9, 0, 0),
    (1, 70, 64, 200, 128, 1, 1, 0), (2, 4, 64, 60, 50, 0, 5, 3), (1, 200, 64, 700, 290, 128, 64, 130),
]


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("B,T,H,N,k,window,page,pad", BF_CASES)
def test_bf16_path(kind, B, T, H, N, k, window, page, pad):
    c = Case(61, B, T, H, N, k, kind, window=window, page=page, pad=pad, unused=T // 5)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(out, lse, **BF)
    half, _ = c.run(want_lse=False)
    assert half.dtype == torch.bfloat16
    assert torch.equal(half, out.to(torch.bfloat16))                   # and the same bits every time


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("B,T,H,N,window,page", [(1, 1, 64, 1000, 128, 64), (2, 5, 64, 333, 128, 16), (1, 33, 64, 700, 100, 64),
                                                 (2, 17, 16, 129, 128, 0), (1, 6, 128, 400, 128, 32), (2, 9, 40, 5, 20, 3),
                                                 (1, 64, 8, 300, 1, 64), (1, 3, 100, 260, 0, 7), (3, 40, 64, 600, 128, 64)])
def test_bf16_dense(kind, B, T, H, N, window, page):
    c = Case(62, B, T, H, N, 0, kind, window=window, page=page, dense=True, unused=T // 6)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(out, lse, **BF)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("flags,base", [(3, 10000.0), (7, 500.0), (7, 1e7)])
@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("B,T,H,N,k,dense", [(2, 5, 40, 300, 100, False), (1, 2, 64, 3000, 1500, False), (2, 9, 24, 150, 0, True),
                                             (1, 3, 16, 2500, 0, True)])
def test_bf16_path_flags(kind, flags, base, sink, B, T, H, N, k, dense):
    """Without rotations, with other angles, with and without a sink, whole groups and ones that are dealt out."""
    c = Case(55, B, T, H, N, k, kind, window=40, page=16, dense=dense, unused=T // 4)
    out, lse = c.run(flags=flags, sink=c.sink if sink else None, rope_base=base, out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(out, lse, **BF, sink=sink, flags=flags, base=base)


@pytest.mark.parametrize("window,T", [(1, 6), (4, 12), (128, 12), (128, 200)])
@pytest.mark.parametrize("dt,kind", [(torch.float32, "f32"), (torch.bfloat16, "bf16")])
def test_chain_equals_the_sparse_attention_over_a_ring(window, T, dt, kind):
    """A draft that is one chain, longer than the window too; sequences shorter than it."""
    B, H, N, k = 3, 24, 300, 40
    c = Case(63, B, T, H, N, k, kind, dt=dt, window=window, lens=[0, 2, 777], spare=T)
    c.parent = (torch.arange(T, device=DEV, dtype=torch.int32) - 1).expand(B, T).contiguous()
    out, lse = c.run(out_dtype=torch.float32)
    ring, pos0 = c.swa.clone(), c.kw["swa_pos0"]
    pos = c.len.unsqueeze(-1) + torch.arange(T, device=DEV)
    ring[torch.arange(B, device=DEV).unsqueeze(-1), (pos - pos0) % ring.shape[1]] = c.draft
    ref, rl = C.csa2_sparse_attn(c.q, c.kv, c.kw["idx"], ring, pos, c.sink, window=window, swa_pos0=pos0, want_lse=True,
                                 out_dtype=torch.float32)
    C.csa2_ctx_check()
    if dt == torch.float32:
        assert_close(to_np(out), to_np(ref), 1e-4, "out")
        assert_close(to_np(lse), to_np(rl), 1e-5, "lse")
    else:
        assert_close(to_np(out), to_np(ref), 2 * BF["tol"], "out")     # both have the path's error
        assert_close(to_np(lse), to_np(rl), 2 * BF["ltol"], "lse")


@pytest.mark.parametrize("kind,dt", [("f32", torch.float32), ("bf16", torch.bfloat16)])
def test_nodes_with_nothing_and_bad_entries(kind, dt):
    """Unused nodes give 0 and the sink; entries outside the cache or on no page are skipped and flagged;
    a NaN in rows that nobody attends to stays there."""
    c = Case(64, 2, 6, 16, 64, 20, kind, dt=dt, window=8, page=16, unused=2)
    c.kw["idx"][0, 4:] = 63                                            # (the selection of unused nodes is not read)
    good, lg = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(good, lg, **(F32 if kind == "f32" else BF))
    assert not good[0, 4:].any() and torch.equal(lg[0, 4:], c.sink.expand(2, -1))
    none, ln = c.run(out_dtype=torch.float32, sink=None)
    assert not none[0, 4:].any() and (ln[0, 4:] == -float("inf")).all()
    spare = torch.ones(c.kv.shape[0], dtype=torch.bool, device=DEV)
    spare[c.table.flatten().long()] = False
    c.kv[spare] = float("nan")
    c.kw["idx"][1, 2, 3:] = -1
    c.sel[1][2, 3:] = -1
    want, lw = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    c.check(want, lw, **(F32 if kind == "f32" else BF))
    c.kw["idx"][1, 2, 3:] = torch.tensor([64, 2 ** 31 - 1, 64 * 16] * 5 + [999, 64], dtype=torch.int32, device=DEV)
    bad, lb = c.run(out_dtype=torch.float32)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert torch.equal(bad, want) and torch.equal(lb, lw)
    c.kw["idx"][1, 2, 3:] = -1
    c.kw["idx"][1, 2, 4] = 50                                          # on a page that is none
    for page in (-1, c.kv.shape[0]):
        t = c.table.clone()
        t[1, 3] = page
        o2, _ = c.run(out_dtype=torch.float32, table=t, idx=torch.where(c.kw["idx"] >= 48, 50, c.kw["idx"]))
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        assert torch.isfinite(o2).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_far_positions_and_large_pools(dt):
    """Positions past 32 bits; pages whose rows lie past 2^31 bytes of the pool.  A RoPE frequency is a
    64-bit float, and so is its product with the position: at 2^40 the angle is off by at most
    2^40 * 2^-52 = 2^-12 rad, once in q^ (a logit's rotated part, below one for unit terms) and once in
    the output, so 2 * 2^-12 more is allowed than elsewhere."""
    n_pages, page = 40000, 64
    kv = torch.zeros(n_pages, page, 512, dtype=torch.bfloat16, device=DEV)
    c = Case(65, 2, 3, 8, 128, 50, "bf16", dt=dt, window=16, page=page, lens=[2 ** 33 + 5, 2 ** 40])
    far = torch.tensor([n_pages - 1, 33000, 32768, 39000, 1, 2, 3], device=DEV)
    kv[far] = c.kv
    c.kv, c.kw["table"] = kv, far[c.table.long()].to(torch.int32)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    tol = F32 if dt == torch.float32 else BF
    c.check(out, lse, tol["tol"] + 2 * 2.0 ** -12, tol["ltol"] + 2.0 ** -12)


@pytest.mark.parametrize("kind,dt", [("bf16", torch.bfloat16), ("fp4", torch.bfloat16), ("f32", torch.float32), ("fp4", torch.float32)])
@pytest.mark.parametrize("dense", [False, True])
def test_operands_that_are_not_given(kind, dt, dense):
    """No window without a ring, no entries without a cache: the same path, and bits, as with one that is not used."""
    c = Case(67, 2, 5, 24, 150, 0 if dense else 70, kind, dt=dt, window=0, page=16, dense=dense)
    pos, path = C.csa2_tree_plan(c.parent, c.len)
    ws = [int(C.load().csa2_tree_attn_workspace_bytes(C.ctx(0), C._dt(c.q), {"f32": C.F32, "bf16": C.BF16, "fp4": C.FP4_E4M3x16}[kind],
                                                      C._dt(c.q), 2, 5, 24, 150 if dense else 70, 0, int(dense), 7))]
    buf = torch.empty(max(16, ws[0]), dtype=torch.uint8, device=DEV)   # (no more than the path takes)
    kw = {**c.kw, "sink": c.sink, "want_lse": True, "ws": buf}
    want = C.csa2_tree_attn(c.q, c.kv, pos, path, c.len, c.swa, c.draft, **kw)
    got = C.csa2_tree_attn(c.q, c.kv, pos, path, c.len, None, None, **kw)
    C.csa2_ctx_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c = Case(68, 2, 5, 24, 150, 0, "bf16" if dt == torch.bfloat16 else "f32", dt=dt, window=30)
    pos, path = C.csa2_tree_plan(c.parent, c.len)                      # (of this case's lengths)
    kw = dict(window=30, swa_pos0=c.kw["swa_pos0"], sink=c.sink, want_lse=True)
    want = C.csa2_tree_attn(c.q, c.kv, pos, path, c.len, c.swa, c.draft, **kw)
    got = C.csa2_tree_attn(c.q, None, pos, path, c.len, c.swa, c.draft, **kw)
    none = C.csa2_tree_attn(c.q, None, pos, path, c.len, None, None, **{**kw, "window": 0})
    C.csa2_ctx_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not none[0].any() and torch.equal(none[1], c.sink.expand_as(none[1]))


@pytest.mark.parametrize("kind,dt", [("f32", torch.float32), ("bf16", torch.bfloat16), ("fp4", torch.bfloat16)])
@pytest.mark.parametrize("dense", [False, True])
def test_table_without_columns(kind, dt, dense):
    """Every entry lies behind such a table: skipped and flagged, whatever the pool holds."""
    c = Case(69, 3, 4, 16, 64, 0 if dense else 20, kind, dt=dt, window=9, page=16, dense=dense)
    none = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    out, lse = c.run(table=none)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    gone = dict(n_visible=torch.zeros_like(c.kw["n_visible"])) if dense else dict(idx=torch.full_like(c.kw["idx"], -1))
    want, lw = c.run(**gone)
    C.csa2_ctx_check()
    # (the dense form has no slots for entries it does not see, so its window's add up in another order)
    tol = F32 if dt == torch.float32 else BF
    assert_close(to_np(out), to_np(want), 2 * tol["tol"], "out")
    assert_close(to_np(lse), to_np(lw), 2 * tol["ltol"], "lse")
    out, lse = c.run(table=none, **gone)                               # nothing asked for is no error
    C.csa2_ctx_check()
    assert torch.equal(out, want) and torch.equal(lse, lw)


def test_path_that_does_not_belong_is_flagged():
    c = Case(66, 1, 4, 8, 30, 5, "bf16", window=16)
    pos, path = C.csa2_tree_plan(c.parent, c.len)
    for p in (pos + 2, pos):
        bad = path.clone()
        if p is pos:
            bad[0, 3] = 9
        out, _ = C.csa2_tree_attn(c.q, c.kv, p, bad, c.len, c.swa, c.draft, idx=c.kw["idx"], window=16)
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cap,T", [(128, 7), (5, 40), (1, 3)])
def test_commit(dt, cap, T):
    B = 4
    par = _tree(70 + T, B, T)
    par[1] = torch.arange(T) - 1
    lens = torch.tensor([0, 3, 2 ** 34, 100], device=DEV)
    pos, path = C.csa2_tree_plan(par, lens)
    draft, swa = W.normal_tensor((B, T, 512), 71, 1, dt, DEV), W.normal_tensor((B, cap, 512), 71, 2, dt, DEV)
    leaf = torch.tensor([T - 1, T - 1, -1, 0], dtype=torch.int32, device=DEV)
    want, new = swa.clone(), lens.clone()
    for b in range(B):
        if leaf[b] >= 0:
            p, a = D.tree_plan(to_np(par[b]), int(lens[b]))
            for j in a[leaf[b]][a[leaf[b]] >= 0]:
                want[b, (int(p[j]) - 9) % cap] = draft[b, int(j)]
            new[b] = int(p[leaf[b]]) + 1
    C.csa2_tree_commit(draft, pos, path, lens, leaf, swa, swa_pos0=9, new_len=lens)
    C.csa2_ctx_check()
    assert torch.equal(swa, want) and torch.equal(lens, new)
    C.csa2_tree_commit(draft, pos, path, lens, torch.full_like(leaf, T), swa, swa_pos0=9, new_len=lens)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert torch.equal(swa, want) and torch.equal(lens, new)


def test_selection_from_keys_in_pages():
    """A Full layer over pages: its keys are read out, scored and selected from, and the selection's rows read
    through the table; the same as over blocks of their own."""
    B, T, H, n, N, k = 2, 5, 16, 200, 208, 40
    rows = {"kv": ((512,), torch.bfloat16), "ki": ((128,), torch.bfloat16)}
    x = {name: W.normal_tensor((B, n, *shape), 85, i, dt, DEV) for i, (name, (shape, dt)) in enumerate(rows.items())}
    cache = P.alloc_pages(B, 40, 16, 13, rows, DEV)
    P.pages_append(cache, x, torch.tensor([n, 150], device=DEV))
    plan = P.plan_draft(_tree(86, B, T), cache.n_entries * 4)
    seen = torch.minimum(P.visible_entries(plan.pos.clamp(min=0), 4), cache.n_entries.unsqueeze(-1))
    qI, w = W.normal_tensor((B, T, 64, 128), 87, 1, torch.bfloat16, DEV), W.normal_tensor((B, T, 64), 87, 2, torch.float32, DEV)
    ids = torch.arange(N, dtype=torch.int32, device=DEV).expand(B, N)
    ids = torch.where(ids < cache.n_entries.unsqueeze(-1), ids, -1).int().contiguous()
    keys = C.csa2_page_read(cache.pools["ki"], cache.table, ids, out=torch.zeros(B, N, 128, dtype=torch.bfloat16, device=DEV))
    _, idx = P.full_topk_step(qI, w, keys, seen, k=k)
    q, draft = W.normal_tensor((B, T, H, 512), 88, 1, torch.bfloat16, DEV), W.normal_tensor((B, T, 512), 88, 2, torch.bfloat16, DEV)
    swa = W.normal_tensor((B, 20, 512), 88, 3, torch.bfloat16, DEV)
    out = P.draft_attention(q, cache, plan, swa, draft, idx=idx, window=12)
    C.csa2_ctx_check()
    _, want_idx = P.full_topk_step(qI, w, torch.nn.functional.pad(x["ki"], (0, 0, 0, N - n)), seen, k=k)
    assert torch.equal(idx, want_idx)
    want, _ = C.csa2_tree_attn(q, x["kv"], plan.pos, plan.path, plan.ctx_len, swa, draft, idx=idx, window=12)
    C.csa2_ctx_check()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 5, 256])
def test_accept_without_layers(T):
    """Where no layer has a window ring the lengths are those of a commit with one; bad leaves are flagged."""
    B = 4
    par = _tree(75, B, T, unused=1)
    par[1] = torch.arange(T) - 1
    plan = P.plan_draft(par, torch.tensor([12, 0, 2 ** 34, 7], device=DEV))
    swa, draft = W.normal_tensor((B, 9, 512), 76, 1, torch.bfloat16, DEV), W.normal_tensor((B, T, 512), 76, 2, torch.bfloat16, DEV)
    for leaf in ([T - 1, T - 1, -1, 0], [-7, 0, T // 2, T - 1]):
        leaf = torch.tensor(leaf, dtype=torch.int32, device=DEV)
        for none in ([], iter(())):
            assert torch.equal(P.accept_draft(plan, leaf, none), P.accept_draft(plan, leaf, [(draft, swa)] * 2))
        C.csa2_ctx_check()
        for b in range(B):
            end = int(plan.pos[b, leaf[b]]) if leaf[b] >= 0 else -1
            assert int(P.accept_draft(plan, leaf, [])[b]) == (end + 1 if end >= 0 else int(plan.ctx_len[b]))
    length = plan.ctx_len.clone()
    C.csa2_tree_commit(None, plan.pos, plan.path, length, leaf, None, new_len=length)      # in place
    assert torch.equal(length, P.accept_draft(plan, leaf, []))
    assert torch.equal(P.accept_draft(plan, torch.full_like(leaf, T), []), plan.ctx_len)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_draft_accept_draft(kind):
    """Two rounds of drafting over one paged cache: the second round's nodes see what the first committed,
    as single tokens queried over the ring do; a fork goes on with another branch."""
    B, H, m, win = 2, 16, 4, 12
    x = W.normal_tensor((B, 60, 512), 81, 2, torch.float32, DEV)
    rows = C.csa2_fp4_pack(x) if kind == "fp4" else x.to(torch.bfloat16)
    cache = P.alloc_pages(B, 40, 8, 12, {"kv": (tuple(rows.shape[2:]), rows.dtype)}, DEV)
    P.pages_append(cache, {"kv": rows}, torch.tensor([60, 41], device=DEV))
    ctx_len = torch.tensor([60 * m + 1, 41 * m], device=DEV)
    swa = W.normal_tensor((B, 20, 512), 81, 3, torch.bfloat16, DEV)
    sink = W.normal_tensor((H,), 81, 4, torch.float32, DEV)
    for step, leaf in enumerate(([5, 3], [2, -1])):
        T = 7
        plan = P.plan_draft(_tree(90 + step, B, T), ctx_len)
        q = W.normal_tensor((B, T, H, 512), 82 + step, 1, torch.bfloat16, DEV)
        draft = W.normal_tensor((B, T, 512), 82 + step, 2, torch.bfloat16, DEV)
        seen = torch.minimum(P.visible_entries(plan.pos, m), cache.n_entries.unsqueeze(-1))
        idx = torch.where(torch.arange(30, device=DEV) < seen.unsqueeze(-1), torch.arange(30, device=DEV), -1).to(torch.int32)
        out = P.draft_attention(q, cache, plan, swa, draft, sink, idx=idx, window=win)
        dense = P.draft_attention(q, cache, plan, swa, draft, sink, n_visible=seen.clamp(max=30), k_max=30, window=win)
        before = swa.clone()
        leaf = torch.tensor(leaf, dtype=torch.int32, device=DEV)
        ctx_len = P.accept_draft(plan, leaf, [(draft, swa)])
        C.csa2_ctx_check()
        dense_rows = C.csa2_page_read(cache.pools["kv"], cache.table, torch.arange(40, dtype=torch.int32, device=DEV).expand(B, 40)
                                      .contiguous())
        for b in range(B):
            if leaf[b] < 0:
                assert torch.equal(swa[b], before[b])
                continue
            # the accepted path again, token by token, over the ring it was committed to
            nodes = plan.path[b, leaf[b].item()].long()
            nodes = nodes[nodes >= 0]
            one = slice(b, b + 1)
            ref, _ = C.csa2_sparse_attn(q[one][:, nodes].contiguous(), dense_rows[one].contiguous(), idx[one][:, nodes].contiguous(),
                                        swa[one].contiguous(), plan.pos[one][:, nodes].contiguous(), sink, window=win)
            assert_close(to_np(out[b, nodes]), to_np(ref[0]), 2 * BF["tol"], "accepted path")
            assert_close(to_np(dense[b, nodes]), to_np(ref[0]), 2 * BF["tol"], "accepted path, dense")
    C.csa2_ctx_check()
