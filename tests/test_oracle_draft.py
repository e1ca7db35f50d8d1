"""Pins of the oracle of drafted trees and paged caches: a chain is the sparse attention over a ring
that holds the drafts, branches do not see each other, and the pages' bookkeeping adds up."""
import numpy as np
import pytest

from oracle import csa2_oracle as O
from oracle import csa2_oracle_draft as D


def test_plan_of_a_small_tree():
    pos, path = D.tree_plan([-1, 0, 0, 2, -1, -2, 5, 7], 10)
    assert pos.tolist() == [10, 11, 11, 12, 10, -1, -1, -1]          # below an unused node, and its own parent
    assert path[3].tolist() == [0, 2, 3] + [-1] * 5 and path[4, 0] == 4 and (path[5:] == -1).all()


@pytest.mark.parametrize("window,L,T", [(128, 5, 3), (4, 9, 6), (1, 0, 2), (0, 7, 3)])
def test_chain_is_the_sparse_attention(window, L, T):
    rng = np.random.default_rng(1)
    kv, swa, draft = rng.normal(size=(20, 128)), rng.normal(size=(160, 128)), rng.normal(size=(T, 128))
    q, sink = rng.normal(size=(T, 3, 128)), rng.normal(size=3)
    sel = [rng.permutation(20)[:5] for _ in range(T)]
    out, lse = D.tree_attn(q, kv, sel, swa, 3, draft, np.arange(T) - 1, L, sink, window)
    ring = swa.copy()
    for i in range(T):
        ring[(L + i - 3) % 160] = draft[i]
        o, l, _ = O.sparse_attn(q[i], kv, sel[i], ring, 3, L + i, sink, window)
        assert np.allclose(out[i], o, atol=1e-13) and np.allclose(lse[i], l, atol=1e-13)


def test_branches_do_not_see_each_other():
    rng = np.random.default_rng(2)
    swa, draft, q = rng.normal(size=(8, 128)), rng.normal(size=(5, 128)), rng.normal(size=(5, 2, 128))
    parent = [-1, 0, 0, 1, 2]
    a = D.tree_attn(q, None, [[]] * 5, swa, 0, draft, parent, 3, None, 8)[0]
    draft[[1, 3]] += 1.0
    b = D.tree_attn(q, None, [[]] * 5, swa, 0, draft, parent, 3, None, 8)[0]
    assert np.array_equal(a[[0, 2, 4]], b[[0, 2, 4]]) and not np.allclose(a[[1, 3]], b[[1, 3]])


def _holds(p):
    return np.array_equal(p.refs, np.bincount(p.table[p.table >= 0], minlength=len(p.refs)))


def test_pages_add_up():
    p = D.Pages(np.zeros(40, int), np.full((3, 12), -1), 4)
    granted, copies = p.reserve([0, 0, 0], [10, 0, 17])
    assert granted.tolist() == [10, 0, 17] and (copies == -1).all() and _holds(p)
    assert p.table[0, :4].tolist() == [0, 1, 2, -1] and p.table[2, :5].tolist() == [3, 4, 5, 6, 7]
    table = np.concatenate([p.table, p.fork([0, 0, 2, -1])])
    p.table = table
    assert _holds(p) and p.refs[:8].tolist() == [3, 3, 3, 2, 2, 2, 2, 2]
    granted, copies = p.reserve([10] * 2 + [17] * 5, [1, 0, 4, 3, 0, 1, 1])
    # sequence 0 and its copies write into the third page, 2 and its copy into the fifth; an empty one at 17
    assert granted.tolist() == [1, 0, 4, 3, 0, 1, 1] and copies[0].tolist() == [2, 8] and copies[3].tolist()[0] == -1
    assert _holds(p)
    p.free(np.array([0, -1, 6, 0, 100, 0, 0]))
    assert _holds(p)
    before = {(b, j): p.table[b, j] for b in range(7) for j in range(12) if p.table[b, j] >= 0}
    moves, cut = p.compact()
    assert _holds(p) and cut == (p.refs > 0).sum() and (p.refs[:cut] > 0).all()
    to = dict(m for m in moves.tolist() if m[0] >= 0)
    assert all(p.table[k] == to.get(v, v) for k, v in before.items())


def test_pages_run_out_in_order():
    p = D.Pages(np.zeros(5, int), np.full((3, 4), -1), 2)
    granted, _ = p.reserve([0, 0, 1], [5, 3, 9])
    assert granted.tolist() == [5, 3, 0] and p.table.tolist()[1] == [3, 4, -1, -1] and _holds(p)
