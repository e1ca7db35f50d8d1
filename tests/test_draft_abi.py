"""Refusals of the drafted trees' and the pages' entry points.  Host-only: a stand-in context and
addresses that are never read, since every call is rejected before anything is launched."""
import ctypes

import pytest
import torch

from compressed_sparse_attention_06_gb300 import build_lib
from compressed_sparse_attention_06_gb300 import csa2 as C

BAD, UNS = C.ERR_INVALID_ARG, C.ERR_UNSUPPORTED
P = 0x10000000                                     # an aligned address that no call reads


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return C.load()


@pytest.fixture(scope="module")
def ctx():
    buf = ctypes.create_string_buffer(256)         # a zeroed context: device 0, no status word
    yield ctypes.cast(buf, ctypes.c_void_p)


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(B=-1), BAD), (dict(T=0), BAD), (dict(T=257), BAD), (dict(B=65536), UNS),
    (dict(parent=None), BAD), (dict(len=None), BAD), (dict(pos=None), BAD), (dict(path=None), BAD), (dict(pos=P + 4), BAD),
    (dict(path=P + 1), BAD), (dict(B=0, pos=None), C.OK),
])
def test_plan_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, parent=P, len=P, B=2, T=4, pos=P, path=P, stream=None)
    a.update(kw)
    assert lib.csa2_tree_plan(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(B=-1), BAD), (dict(T=0), BAD), (dict(T=257), BAD), (dict(N=-1), BAD), (dict(k=-1), BAD),
    (dict(k=2049), BAD), (dict(window=-1), BAD), (dict(window=1025), BAD), (dict(window=129), BAD), (dict(H=0), BAD),
    (dict(H=129), BAD), (dict(c=256), UNS), (dict(flags=8), BAD), (dict(q_dt=2), UNS), (dict(kv_dt=3), UNS), (dict(out_dt=7), UNS),
    (dict(swa_dt=2), UNS), (dict(B=300, T=256), UNS), (dict(nv=P), BAD), (dict(idx=None), BAD), (dict(kv=None), BAD),
    (dict(swa=None), BAD), (dict(draft=None), BAD), (dict(pos=None), BAD), (dict(path=None), BAD), (dict(len=None), BAD),
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(q=P + 8), BAD), (dict(kv=P + 8), BAD), (dict(draft=P + 2), BAD),
    (dict(out=P + 4), BAD), (dict(ws=P + 8), BAD), (dict(lse=P + 2), BAD), (dict(table=P, page=0), BAD),
    (dict(table=P, page=65537), BAD), (dict(table=P, page=64, N=100), BAD), (dict(table=P, max_pages=-1), BAD),
    (dict(table=P + 2), BAD), (dict(idx=None, nv=P, k=(1 << 22) + 1), BAD), (dict(N=1 << 40), UNS),
    (dict(cap=100), BAD), (dict(B=0, q=None), C.OK),
])
def test_attention_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, q=P, q_dt=C.BF16, kv=P, kv_dt=C.BF16, N=128, table=None, max_pages=2, page=64, idx=P, nv=None, k=16, swa=P,
             swa_dt=C.BF16, cap=128, pos0=0, window=128, draft=P, pos=P, path=P, len=P, sink=None, B=1, T=4, H=64, c=512,
             base=10000.0, flags=7, out=P, out_dt=C.BF16, lse=None, ws=P, ws_bytes=0, stream=None)
    a.update(kw)
    assert lib.csa2_tree_attn(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(B=-1), BAD), (dict(T=300), BAD), (dict(cap=0), BAD), (dict(c=128), UNS), (dict(dt=2), UNS),
    (dict(B=65536), UNS), (dict(draft=None), BAD), (dict(leaf=None), BAD), (dict(swa=None), BAD), (dict(swa=P + 8), BAD),
    (dict(new_len=P + 4), BAD),
])
def test_commit_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, draft=P, dt=C.BF16, pos=P, path=P, len=P, leaf=P, B=2, T=4, c=512, swa=P, cap=128, pos0=0, new_len=None,
             stream=None)
    a.update(kw)
    assert lib.csa2_tree_commit(*a.values()) == want


STATE = [(dict(ctx=None), BAD), (dict(n=-1), BAD), (dict(n=1 << 31), UNS), (dict(B=-1), BAD), (dict(B=65536), UNS),
         (dict(mp=-1), BAD), (dict(refs=None), BAD), (dict(table=None), BAD), (dict(refs=P + 2), BAD), (dict(table=P + 1), BAD)]


@pytest.mark.parametrize("kw,want", STATE + [
    (dict(B_out=-1), BAD), (dict(B_out=65536), UNS), (dict(parent=None), BAD), (dict(out=None), BAD), (dict(out=P + 4 * 16 * 2 - 4), BAD),
    (dict(out=P), BAD), (dict(B_out=0, parent=None), C.OK),
])
def test_fork_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, refs=P, n=100, table=P, B=2, mp=16, parent=P, B_out=4, out=2 * P, stream=None)
    a.update(kw)
    assert lib.csa2_pages_fork(*a.values()) == want


@pytest.mark.parametrize("kw,want", STATE + [(dict(page=0), BAD), (dict(page=65537), BAD), (dict(keep=P + 4), BAD)])
def test_free_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, refs=P, n=100, table=P, B=2, mp=16, page=64, keep=None, stream=None)
    a.update(kw)
    assert lib.csa2_pages_free(*a.values()) == want


@pytest.mark.parametrize("kw,want", STATE + [
    (dict(page=0), BAD), (dict(first=None), BAD), (dict(count=None), BAD), (dict(granted=None), BAD), (dict(copies=None), BAD),
    (dict(ws=None), BAD), (dict(ws=P + 8), BAD), (dict(ws_bytes=(100 + 2 * 2 * 1) * 4 - 1), BAD), (dict(first=P + 4), BAD),
])
def test_reserve_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, refs=P, n=100, table=P, B=2, mp=16, page=64, first=P, count=P, granted=P, copies=P, ws=P, ws_bytes=1 << 20,
             stream=None)
    a.update(kw)
    assert lib.csa2_pages_reserve(*a.values()) == want
    assert lib.csa2_pages_reserve_workspace_bytes(100, 2, 16) == (100 + 4) * 4


@pytest.mark.parametrize("kw,want", STATE + [
    (dict(moves=None), BAD), (dict(ws=None), BAD), (dict(ws_bytes=415), BAD), (dict(n_used=P + 4), BAD), (dict(ws=P + 4), BAD),
])
def test_compact_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, refs=P, n=100, table=P, B=2, mp=16, moves=P, n_used=P, ws=P, ws_bytes=416, stream=None)
    a.update(kw)
    assert lib.csa2_pages_compact(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(n_pages=-1), BAD), (dict(n=-1), BAD), (dict(bytes=2), BAD), (dict(bytes=6), UNS),
    (dict(n_pages=1 << 31), UNS), (dict(pool=None), BAD), (dict(pairs=None), BAD), (dict(pool=P + 2), BAD), (dict(n=0, pool=None), C.OK),
])
def test_copy_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, pool=P, n_pages=10, bytes=1024, pairs=P, n=4, stream=None)
    a.update(kw)
    assert lib.csa2_page_copy(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(n_pages=-1), BAD), (dict(page=0), BAD), (dict(rb=2), BAD), (dict(rb=6), UNS),
    (dict(rb=(1 << 20) + 4), BAD), (dict(B=65536), UNS), (dict(n=-1), BAD), (dict(mp=-1), BAD), (dict(n_pages=1 << 30, page=65536), UNS),
    (dict(pool=None), BAD), (dict(table=None), BAD), (dict(dense=None), BAD), (dict(dense=P + 4096), BAD), (dict(dense=P - 1024), BAD),
    (dict(dense=P - 256 * 2 * 5 - 2), BAD),
])
def test_rows_refuse(lib, ctx, kw, want):
    a = dict(ctx=ctx, pool=P, n_pages=10, page=16, rb=256, table=P, B=2, mp=4, dense=2 * P, n=5, x=P, y=P, stream=None)
    a.update(kw)
    assert lib.csa2_page_write(*a.values()) == want
    del a["y"]
    a = dict(list(a.items())[:8] + [("idx", P), ("n", a["n"]), ("dense", a["dense"]), ("stream", None)])
    assert lib.csa2_page_read(*a.values()) == want


def test_binding_checks_shapes():
    """The binding hands sizes of its tensors to the library: tensors that do not fit are refused there."""
    refs, table = torch.zeros(8, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="first"):
        C.csa2_pages_reserve(refs, table, one[:1], one, 4)
    with pytest.raises(ValueError, match="table"):
        C.csa2_pages_fork(refs, table.long(), one.int())
    with pytest.raises(ValueError, match="rows"):
        C.csa2_page_write(torch.zeros(8, 4, 6), table, torch.zeros(2, 3, 5), one, one)
    with pytest.raises(ValueError, match="pairs"):
        C.csa2_page_copy(torch.zeros(8, 4, 6), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="ctx_len"):
        C.csa2_tree_plan(torch.zeros(2, 4, dtype=torch.int32), one[:1])
    q, pos, path = torch.zeros(2, 3, 4, 512), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3, 3, dtype=torch.int16)
    with pytest.raises(ValueError, match="rows of 512"):
        C.csa2_tree_attn(q, torch.zeros(2, 5, 288), pos, path, one, None, None, window=0)
    with pytest.raises(ValueError, match="draft"):
        C.csa2_tree_attn(q, None, pos, path, one, torch.zeros(2, 9, 512), torch.zeros(2, 2, 512), window=9)


def test_commit_of_lengths_alone(lib, ctx):
    """Without a ring there has to be something to write; half a ring is none."""
    a = dict(ctx=ctx, draft=None, dt=C.BF16, pos=P, path=P, len=P, leaf=P, B=2, T=4, c=512, swa=None, cap=0, pos0=0, new_len=None,
             stream=None)
    assert lib.csa2_tree_commit(*a.values()) == BAD
    assert lib.csa2_tree_commit(*{**a, "new_len": P + 4}.values()) == BAD
    assert lib.csa2_tree_commit(*{**a, "new_len": P, "leaf": None}.values()) == BAD
    assert lib.csa2_tree_commit(*{**a, "new_len": P, "B": 0}.values()) == C.OK
    x = torch.zeros(2, 4, 512)
    i = torch.zeros(2, 4, dtype=torch.int64)
    for draft, swa in ((x, None), (None, x)):
        with pytest.raises(ValueError, match="neither"):
            C.csa2_tree_commit(draft, i, torch.zeros(2, 4, 4, dtype=torch.int16), i[:, 0], i[:, 0].int(), swa)
