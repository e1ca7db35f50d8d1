"""Drafted trees on the tensor cores with queries that lie along the rows they read: logits up to their bound,
sqrt(512) = 22.6, a few of them nearly equal, the rest of the slots without weight.

Tolerances, per node and head, from the inputs.  A slot's logit z = q^ . k^ / sqrt(512) is off by
  a   the bf16 rounding of q^'s 64 rotated dims, at most half a step each (2^-8 relative), independent: five
      deviations are 5 * 2^-8 / sqrt(3) * sqrt(sum (q^_i k^_i)^2) / sqrt(512) over those dims;
  b   the half of it that crosses between the two CTAs, a multiple of 1/992 in base 2: ln 2 / 1984;
  c   sums and exponentials in fp32: 2e-4 (22.6 * 2^-23 for each of the 32 products' additions is 9e-5).
dz = the largest a + b + c of a node's slots bounds the log-sum-exp's error.  An output sum w_s k^_s is off by
at most (2 dz + 2^-8) sum w_s |k^_s|, the second term p in bf16; a rotated dim gets its pair's too."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_06_gb300 import csa2 as C
from oracle import csa2_oracle as O
from oracle import csa2_oracle_draft as D
from tests.helpers import to_np
from tests.test_gpu_tree import DEV, Case

pytestmark = pytest.mark.gpu
CLUSTERS = 50


def _peaked(seed, B, T, H, N, k, kind, energy, dense, window=20):
    """A case whose rows are near copies of 50 vectors and whose heads' queries lie along those."""
    c = Case(seed, B, T, H, N, k, kind, window=window, dense=dense, page=16)
    rng = np.random.default_rng(seed)
    size = np.ones(512)
    if energy != "all":
        size[slice(256, None) if energy == "low" else slice(None, 256)] = 0.02
    g = rng.standard_normal((CLUSTERS, 512)) * size

    def rows(n):
        x = g[np.arange(n) % CLUSTERS] + 0.15 * rng.standard_normal((n, 512)) * size
        return torch.tensor(x * np.exp(0.3 * rng.standard_normal((n, 1))), dtype=torch.float32, device=DEV)

    c.swa = rows(c.swa.shape[0] * c.swa.shape[1]).view(c.swa.shape).to(torch.bfloat16)
    c.draft = rows(B * T).view(c.draft.shape).to(torch.bfloat16)
    n_pages = c.kv.shape[0]
    x = rows(n_pages * 16).view(n_pages, 16, 512)
    c.kv = C.csa2_fp4_pack(x) if kind == "fp4" else x.to(torch.bfloat16)
    v = O.nvfp4_unpack(to_np(c.kv).reshape(-1, 288)).reshape(n_pages, 16, 512) if kind == "fp4" else to_np(c.kv)
    c.entries = [v[to_np(t)].reshape(-1, 512)[:N] for t in c.table]
    q = np.zeros((B, T, H, 512))
    for b in range(B):
        pos, _ = D.tree_plan(to_np(c.parent[b]), int(c.len[b]))
        for i in range(T):
            q[b, i] = O.rope(g[(np.arange(H) + 7 * i) % CLUSTERS], int(pos[i]), inverse=True)
    c.q = torch.tensor(q, dtype=torch.float32, device=DEV).to(torch.bfloat16)
    return c


def _check(c, out, lse):
    """Returns the largest logit."""
    top = 0.0
    out, lse = to_np(out), to_np(lse)
    for b in range(c.q.shape[0]):
        parent, n = to_np(c.parent[b]), int(c.len[b])
        pos, path = D.tree_plan(parent, n)
        want, wl = D.tree_attn(to_np(c.q[b]), c.entries[b], c.sel[b], to_np(c.swa[b]), c.kw["swa_pos0"], to_np(c.draft[b]), parent, n,
                               to_np(c.sink), c.kw["window"])
        for i in range(len(parent)):
            K = O.rms_norm(D.tree_keys(c.entries[b], c.sel[b][i], to_np(c.swa[b]), c.kw["swa_pos0"], to_np(c.draft[b]), pos, path, n, i,
                                       c.kw["window"]))
            q = O.rope(O.rms_norm(to_np(c.q[b, i])), int(pos[i]))
            z = q @ K.T / np.sqrt(512)
            top = max(top, z.max())
            a = 5 * 2.0 ** -8 / np.sqrt(3) * np.sqrt(q[:, 448:] ** 2 @ (K[:, 448:] ** 2).T / 512)
            # (slots without weight move nothing: those ten below the largest count e^-10 of their error)
            dz = np.max(np.where(z > z.max(1, keepdims=True) - 10, a, 0), 1) + np.log(2) / 1984 + 2e-4
            bad = np.abs(lse[b, i] - wl[i]) > dz
            assert not bad.any(), f"lse of node {i}: off by {np.abs(lse[b, i] - wl[i])[bad]}, allowed {dz[bad]}"
            w = np.exp(z - wl[i][:, None])
            size = w @ np.abs(K)
            size[:, 448:] = np.repeat(size[:, 448::2] + size[:, 449::2], 2, axis=1)
            bound = (2 * dz[:, None] + 2.0 ** -8) * size + 1e-6
            err = np.abs(out[b, i] - want[i])
            assert (err <= bound).all(), f"out of node {i}: off by {err.max()}, {(err / bound).max()} of what is allowed"
    return top


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("energy", ["all", "low", "high"])
@pytest.mark.parametrize("B,T,H,N,k,dense", [(2, 6, 40, 300, 128, False), (1, 1, 64, 700, 250, False), (1, 13, 128, 256, 100, False),
                                             (2, 9, 24, 100, 0, True), (1, 5, 50, 1700, 0, True)])
def test_queries_along_rows(kind, energy, B, T, H, N, k, dense):
    c = _peaked(7 * T + H, B, T, H, N, k, kind, energy, dense)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    assert _check(c, out, lse) > 20


@pytest.mark.parametrize("energy", ["all", "low", "high"])
def test_queries_that_are_rows(energy):
    """Queries equal to a row, turned back by the position: the bound itself, and its negative."""
    c = _peaked(5, 1, 4, 16, 60, 30, "bf16", energy, False)
    pos, _ = D.tree_plan(to_np(c.parent[0]), int(c.len[0]))
    q = np.stack([O.rope(c.entries[0][c.sel[0][i][:16]] * (-1.0) ** np.arange(16)[:, None], int(pos[i]), inverse=True) for i in range(4)])
    c.q = torch.tensor(q[None], dtype=torch.float32, device=DEV).to(torch.bfloat16)
    out, lse = c.run(out_dtype=torch.float32)
    C.csa2_ctx_check()
    assert _check(c, out, lse) > 22.5
