"""Refusals of the backward, weight and eviction entry points.  Host-only: a stand-in context
and addresses that are never read, since every call is rejected before anything is launched."""
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


def _bwd(lib, context, dense=False, **kw):
    a = dict(ctx=context, q=P, q_dt=C.BF16, kv=P, kv_dt=C.BF16, N=100, sel=P, k=16, swa=P, swa_dt=C.BF16, cap=128, pos0=0,
             window=128, q_pos=P, sink=None, out=P, dout=P, out_dt=C.BF16, lse=P, B=1, Q=4, H=64, c=512, base=10000.0,
             flags=7, dq=P, dkv=P, dswa=P, dsink=P, ws=P, ws_bytes=1, stream=None)
    a.update(kw)
    return (lib.csa2_dense_attn_bwd if dense else lib.csa2_sparse_attn_bwd)(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(B=-1), BAD), (dict(Q=-1), BAD), (dict(N=-1), BAD), (dict(k=-1), BAD), (dict(k=2049), BAD),
    (dict(window=1025), BAD), (dict(window=-1), BAD), (dict(H=0), BAD), (dict(H=129), BAD), (dict(c=256), UNS),
    (dict(flags=8), BAD), (dict(kv_dt=C.FP4_E4M3x16), UNS), (dict(q_dt=C.MXFP4_E8M0x32), UNS), (dict(out_dt=7), UNS),
    (dict(swa_dt=2), UNS), (dict(B=2, Q=40000), UNS), (dict(cap=127), BAD), (dict(swa=None), BAD), (dict(cap=-1), BAD),
    (dict(q=P + 8), BAD), (dict(kv=P + 2), BAD), (dict(dout=P + 4), BAD), (dict(dq=P + 8), BAD), (dict(dkv=P + 8), BAD),
    (dict(dswa=P + 8), BAD), (dict(lse=P + 2), BAD), (dict(q=None), BAD), (dict(q_pos=None), BAD), (dict(out=None), BAD),
    (dict(dout=None), BAD), (dict(lse=None), BAD), (dict(dq=None), BAD), (dict(ws=None), BAD), (dict(kv=None), BAD),
    (dict(sel=None), BAD), (dict(N=1 << 31), UNS),
])
def test_attention_backward_refuses(lib, ctx, kw, want):
    assert _bwd(lib, ctx, **kw) == want


def test_dense_backward_refuses(lib, ctx):
    assert _bwd(lib, ctx, dense=True, sel=None) == BAD
    assert _bwd(lib, ctx, dense=True, k=(1 << 22) + 1) == BAD
    assert _bwd(lib, ctx, dense=True, k=-1) == BAD


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(k=2049), BAD), (dict(H=129), BAD), (dict(c=128), UNS), (dict(flags=16), BAD),
    (dict(kv_dt=C.MXFP4_E8M0x32), UNS), (dict(q_dt=2), UNS), (dict(weights=None, acc=None), BAD), (dict(q=None), BAD),
    (dict(kv=None), BAD), (dict(lse=None), BAD), (dict(q_pos=None), BAD), (dict(nv=P), BAD), (dict(idx=None), BAD),
    (dict(B=65536), UNS), (dict(kv=P + 8), BAD), (dict(ws_bytes=799), BAD), (dict(ws=None, ws_bytes=800), BAD), (dict(N=-1), BAD),
    (dict(Q=1, kv_dt=C.F32, ws_bytes=64 * 2048 - 1), BAD), (dict(Q=1, H=100, ws_bytes=63), BAD),
])
def test_mass_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, q=P, q_dt=C.BF16, kv=P, kv_dt=C.BF16, N=100, idx=P, nv=None, k=16, q_pos=P, lse=P, B=1, Q=4, H=64,
             c=512, base=10000.0, flags=7, weights=P, acc=P, ws=P, ws_bytes=1, stream=None)
    a.update(kw)
    assert lib.csa2_attn_mass(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(B=-1), BAD), (dict(ld=-1), BAD), (dict(ld=1 << 31), BAD), (dict(keep=0), BAD),
    (dict(recent=-1), BAD), (dict(recent=9), BAD), (dict(n=None), BAD), (dict(out=None), BAD), (dict(acc=None), BAD),
    (dict(B=65536), UNS), (dict(n=P + 4), BAD), (dict(ld=65537), BAD), (dict(ld=65537, ws=P, ws_bytes=49152 + 79), BAD),
    (dict(ld=65537, ws=P + 8, ws_bytes=1 << 20), BAD),
])
def test_select_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, acc=P, B=2, ld=100, n=P, keep=8, recent=2, out=P, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    assert lib.csa2_evict_select(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(rb=0), BAD), (dict(rb=6), UNS), (dict(rb=(1 << 20) + 4), BAD), (dict(keep=-1), BAD),
    (dict(src=None), BAD), (dict(idx=None), BAD), (dict(dst=None), BAD), (dict(src=P + 2), BAD), (dict(dst=P), BAD),
    (dict(dst=P + 2 * 100 * 64 - 4), BAD), (dict(N=-1), BAD),
])
def test_gather_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, src=P, rb=64, B=2, N=100, idx=P, keep=8, dst=2 * P, stream=None)
    a.update(kw)
    assert lib.csa2_cache_gather(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ctx=None), BAD), (dict(n=33), BAD), (dict(m=0), BAD), (dict(c=96), BAD), (dict(c=1152), BAD), (dict(zb=P, cb=None), BAD),
    (dict(prev_cb=P), BAD), (dict(cb=None, zb=None, prev_cb=P, prev_zb=P), BAD), (dict(flags=4), BAD), (dict(in_dt=2), UNS),
    (dict(dout_dt=3), UNS), (dict(dprev_cb=P), BAD), (dict(ca=P + 8), BAD), (dict(dba=P + 4), BAD), (dict(pos0=P + 4), BAD),
    (dict(cb=None, zb=None, dbb=P), BAD),
])
def test_compressor_backward_refuses(lib, ctx, kw, want):
    a = dict(ctx=ctx, ca=P, za=P, cb=P, zb=P, in_dt=C.BF16, ba=None, bb=None, prev_cb=None, prev_zb=None, B=1, n=32, c=512,
             m=4, pos0=None, base=10000.0, flags=3, dout=P, dout_dt=C.BF16, stride=8, dca=P, dza=P, dcb=P, dzb=P,
             dprev_cb=None, dprev_zb=None, dba=P, dbb=None, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    assert lib.csa2_compress_bwd(*a.values()) == want


def test_workspace_sizes(lib, ctx):
    small = lib.csa2_attn_bwd_workspace_bytes(ctx, C.BF16, C.BF16, C.BF16, C.BF16, 1, 4, 64, 512, 128, 2048, 128, 7)
    assert small > 0
    # the largest calls stay near 16 GiB by running in chunks
    big = lib.csa2_attn_bwd_workspace_bytes(ctx, C.F32, C.F32, C.F32, C.F32, 1, 65535, 128, 2048, 1024, 34816, 70000, 7)
    assert big <= 16 << 30
    assert lib.csa2_attn_bwd_workspace_bytes(None, 1, 1, 1, 1, 1, 4, 64, 512, 128, 2048, 128, 7) == 0
    assert lib.csa2_attn_mass_workspace_bytes(ctx, C.BF16, 8, 1, 64, 512, 1 << 20, 1) == 0      # no per-entry table for Q = 1
    assert lib.csa2_evict_select_workspace_bytes(8, 65536) == 0
    assert lib.csa2_evict_select_workspace_bytes(2, 65537) == 2 * 3 * 2048 * 4 + 2 * 5 * 2 * 4
    assert lib.csa2_compress_bwd_workspace_bytes(1, 8192, 512, 4, 1) > 0
    assert lib.csa2_compress_bwd_workspace_bytes(0, 8192, 512, 4, 1) == 0


@pytest.mark.parametrize("dt", [C.F32, C.BF16])
@pytest.mark.parametrize("B,Q,H,k,window", [(1, 4, 64, 512, 128), (2, 96, 40, 301, 100), (1, 8192, 128, 512, 128)])
def test_attention_backward_workspace_may_begin_at_any_16_bytes(lib, ctx, dt, B, Q, H, k, window):
    """The kernels store up to 32 bytes at once, so the buffers (whole 256-byte pieces) begin at a
    256-byte boundary; a base 16 bytes behind one is 240 away from the next."""
    assert lib.csa2_attn_bwd_workspace_bytes(ctx, dt, dt, dt, dt, B, Q, H, k, window, 2048, 128, 7) % 256 == 240


@pytest.mark.parametrize("c,m,overlap,entries,slabs", [
    # the launch takes one CTA, and one slab, an entry up to the count that follows from the threads
    (128, 5, 0, 4000, 4000), (128, 5, 1, 4000, 2000), (128, 12, 0, 1217, 1217), (128, 16, 0, 1217, 609),
    (256, 7, 0, 2000, 2000), (256, 8, 1, 1217, 406), (384, 5, 0, 1600, 1600), (512, 5, 0, 1217, 609),
    (1024, 7, 0, 608, 608), (512, 128, 0, 152, 152), (512, 128, 0, 153, 77), (128, 4, 0, 1217, 406), (128, 2, 0, 1217, 609),
])
def test_bias_slabs_match_the_launch(lib, c, m, overlap, entries, slabs):
    """csa2_compress_bwd's workspace has a slab of bias sums for every CTA of the launch: windows that
    are not compiled for their size run 1,216 CTAs of 128 threads, or as many more or fewer as
    their CTAs are smaller or larger."""
    table = (2 if overlap else 1) * m * c * 4
    assert lib.csa2_compress_bwd_workspace_bytes(1, entries * m, c, m, overlap) == slabs * table


def test_binding_checks_shapes_before_the_library():
    t = torch.zeros(2, 5)
    with pytest.raises(ValueError):
        C._want("x", t, (2, 4), torch.float32, t.device)
    with pytest.raises(ValueError):
        C._want("x", t.t(), (5, 2), torch.float32, t.device)
    with pytest.raises(ValueError):
        C._want("x", t, (2, 5), torch.float64, t.device)
    assert C._given("x", t, (2, 5), torch.float32, t.device) is t
    with pytest.raises(ValueError):
        C.csa2_attn_mass(torch.zeros(1, 1, 1, 512), torch.zeros(1, 4, 512), None, None)
