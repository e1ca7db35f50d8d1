"""The gradient oracle against central differences of the forward oracle, and the eviction
and weight definitions against brute force, on tiny inputs (CPU)."""
import numpy as np
import pytest

from oracle import csa2_oracle as O
from oracle import csa2_oracle_grad as G

STEP = 1e-5
# central differences in f64: truncation about STEP^2 = 1e-10 of the third derivative, rounding
# 2^-53 * |loss| / STEP with |loss| of a few tens: 1e-15 * 30 / 1e-5 = 3e-9; 1e-6 covers both
TOL = 1e-6


def _differences(loss, x, picks):
    out = []
    for i in picks:
        hi, lo = x.copy(), x.copy()
        hi.flat[i] += STEP
        lo.flat[i] -= STEP
        out.append((loss(hi) - loss(lo)) / (2 * STEP))
    return np.array(out)


def _picks(rng, x, n=24):
    return rng.choice(x.size, size=min(n, x.size), replace=False)


@pytest.mark.parametrize("flags", [O.QNORM | O.KVNORM | O.ROPE, 0, O.ROPE, O.KVNORM])
@pytest.mark.parametrize("sink", [True, False])
def test_attention_gradients_match_differences(flags, sink):
    rng = np.random.default_rng(5 + flags)
    Q, H, c, N, cap, window = 3, 2, 64, 9, 5, 4
    # unnormalised rows keep the logits small: values of about 1/4
    q, kv, swa = (0.5 * rng.standard_normal(s) for s in ((Q, H, c), (N, c), (cap, c)))
    sel = np.array([[0, 3, 3, 7], [2, -1, 8, -1], [-1, -1, -1, -1]])
    pos = [6, 2, 11]
    z = rng.standard_normal(H) if sink else None
    dout = rng.standard_normal((Q, H, c))

    def run(q, kv, swa, z):
        r = [O.sparse_attn(q[i], kv, sel[i], swa, 1, pos[i], z, window, flags) for i in range(Q)]
        return np.array([x[0] for x in r]), np.array([x[1] for x in r])

    def loss(q, kv, swa, z):
        return float((run(q, kv, swa, z)[0] * dout).sum())

    out, lse = run(q, kv, swa, z)
    (dq, dkv, dswa, dsink), _ = G.attn_bwd(q, kv, sel, swa, 1, pos, z, window, out, lse, dout, flags)
    cases = [(dq, q, lambda x: loss(x, kv, swa, z)), (dkv, kv, lambda x: loss(q, x, swa, z)),
             (dswa, swa, lambda x: loss(q, kv, x, z))]
    if sink:
        cases.append((dsink, z, lambda x: loss(q, kv, swa, x)))
    else:
        assert not dsink.any()
    for got, x, f in cases:
        at = _picks(rng, x)
        np.testing.assert_allclose(got.flat[at], _differences(f, x, at), rtol=TOL, atol=TOL)
    assert not dkv[[1, 4, 5, 6]].any()            # entries that no query attends to


def test_query_without_keys_has_no_gradient():
    rng = np.random.default_rng(3)
    q, out = rng.standard_normal((1, 2, 64)), np.zeros((1, 2, 64))
    for lse in (np.full((1, 2), -np.inf), np.zeros((1, 2))):
        g, _ = G.attn_bwd(q, rng.standard_normal((4, 64)), np.array([[-1, -1]]), rng.standard_normal((3, 64)), 0, [-1], None,
                       2, out, lse, rng.standard_normal((1, 2, 64)))
        assert all(not x.any() for x in g)


@pytest.mark.parametrize("overlap,prev", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("flags", [0, O.NORM_W, O.NORM_W | O.ROPE_W])
def test_compressor_gradients_match_differences(overlap, prev, flags):
    rng = np.random.default_rng(17 + flags)
    n, m, c = 12, 3, 64
    names = ["Ca", "Za", "Ba"] + (["Cb", "Zb", "Bb"] if overlap else []) + (["prev_Cb", "prev_Zb"] if prev else [])
    x = {k: rng.standard_normal((n, c) if k in ("Ca", "Za", "Cb", "Zb") else (m, c)) for k in names}
    dout = rng.standard_normal((n // m, c))

    def loss(v):
        return float((O.compress_write(O.compress(m=m, **v), flags, m, 40) * dout).sum())

    g = G.compress_bwd(m=m, dout=dout, flags=flags, pos0=40, **x)
    for k in names:
        at = _picks(rng, x[k])
        want = _differences(lambda y, k=k: loss({**x, k: y}), x[k], at)
        np.testing.assert_allclose(g[k].flat[at], want, rtol=TOL, atol=TOL, err_msg=k)


def test_mass_is_the_forward_probability():
    rng = np.random.default_rng(8)
    q, kv = rng.standard_normal((1, 3, 64)), rng.standard_normal((6, 64))
    sel = np.array([[4, 1, 4, -1]])
    o, lse, mass = O.sparse_attn(q[0], kv, sel[0], None, 0, 9, None, 0)
    w, total = G.attn_mass(q, kv, sel, [9], lse[None])
    assert w[0, 3] == 0 and w[0, 0] == w[0, 2]
    np.testing.assert_allclose(total[4], w[0, 0] + w[0, 2])
    np.testing.assert_allclose(total.sum(), mass.sum(), rtol=1e-12)
    assert not total[[0, 2, 3, 5]].any()


@pytest.mark.parametrize("n,keep,recent", [(10, 4, 2), (10, 4, 0), (10, 4, 4), (3, 4, 2), (4, 4, 1), (0, 4, 0)])
def test_evict_keep_by_brute_force(n, keep, recent):
    rng = np.random.default_rng(n + keep + recent)
    acc = rng.integers(0, 3, 10).astype(float)
    ids = G.evict_keep(acc, n, keep, recent)
    kept = [i for i in ids if i >= 0]
    assert kept == sorted(set(kept)) and len(kept) == min(n, keep) and len(ids) == keep
    if n > keep:
        assert set(range(n - recent, n)) <= set(kept)
        for i in set(range(n - recent)) & set(kept):
            for j in set(range(n - recent)) - set(kept):
                assert acc[i] > acc[j] or (acc[i] == acc[j] and i < j)
