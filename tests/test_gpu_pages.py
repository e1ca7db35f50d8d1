"""Caches in pages against the oracle's bookkeeping, bit for bit: shared pages, copy on write, pools that
run out, compaction, and rows written and read through the table."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_06_gb300 import csa2 as C
from compressed_sparse_attention_06_gb300 import pipeline as P
from oracle import csa2_oracle_draft as D
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _i64(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int64, device=DEV)


def _state(o):
    return _i32(o.refs), _i32(o.table)


def _same(o, refs, table):
    assert np.array_equal(to_np(refs), o.refs) and np.array_equal(to_np(table), o.table)


def _random(seed, n_pages, B, P_, page, fill=0.6):
    """A state with pages dealt out, some shared."""
    rng = np.random.default_rng(seed)
    o = D.Pages(np.zeros(n_pages, int), np.full((B, P_), -1), page)
    for b in range(B):
        for j in range(int(P_ * fill)):
            u = rng.random()
            if u < 0.2 and b > 0 and o.table[b - 1, j] >= 0:
                t = o.table[b - 1, j]
            elif u < 0.9 and (o.refs == 0).any():
                t = rng.choice(np.flatnonzero(o.refs == 0))
            else:
                continue
            o.table[b, j] = t
            o.refs[t] += 1
    return o, rng


@pytest.mark.parametrize("n_pages,B,P_,page", [(1, 1, 1, 1), (40, 3, 7, 4), (300, 33, 40, 17), (5000, 2, 1200, 64), (9001, 300, 33, 16),
                                               (200, 1, 150, 3)])
def test_state_follows_the_oracle(n_pages, B, P_, page):
    """Rounds of fork, reserve, free and compact on one state, the table of every sequence in one block."""
    o, rng = _random(n_pages + B, n_pages, B, P_, page)
    refs, table = _state(o)
    for _ in range(4):
        first = rng.integers(0, P_ * page + 1, B)
        count = np.minimum(rng.integers(0, 4 * page + 2, B), P_ * page - first)
        if rng.random() < 0.5:
            first[rng.integers(0, B)] = -3
        g, c = o.reserve(first, count)
        granted, copies = C.csa2_pages_reserve(refs, table, _i64(first), _i64(count), page)
        _same(o, refs, table)
        assert np.array_equal(to_np(granted), g) and np.array_equal(to_np(copies), c)
        parent = rng.integers(-1, B, 5)
        out = o.fork(parent)
        forked = C.csa2_pages_fork(refs, table, _i32(parent))
        assert np.array_equal(to_np(forked), out)
        _same(o, refs, table)
        C.csa2_pages_free(refs, forked, page)
        assert (forked == -1).all()
        for t in out[out >= 0]:
            o.refs[t] -= 1
        keep = rng.integers(-1, P_ * page + 2, B)
        o.free(keep)
        C.csa2_pages_free(refs, table, page, _i64(keep))
        _same(o, refs, table)
        moves, cut = o.compact()
        m, n_used = C.csa2_pages_compact(refs, table)
        _same(o, refs, table)
        assert np.array_equal(to_np(m), moves) and int(n_used) == cut
    C.csa2_pages_free(refs, table, page)
    C.csa2_ctx_check()
    assert not refs.any() and (table == -1).all()


def test_reserve_a_long_range_and_run_out():
    """More words of pages than a pass of the block takes, and a pool that ends inside them."""
    o = D.Pages(np.zeros(3500, int), np.full((3, 2000), -1), 2)
    o.refs[::7] = 1                                       # held by somebody else's table
    refs, table = _state(o)
    first, count = np.array([5, 0, 3]), np.array([3990, 1, 3000])
    g, c = o.reserve(first, count)
    granted, copies = C.csa2_pages_reserve(refs, table, _i64(first), _i64(count), 2)
    C.csa2_ctx_check()
    _same(o, refs, table)
    assert np.array_equal(to_np(granted), g) and np.array_equal(to_np(copies), c) and 0 < g[2] < 3000
    again, none = C.csa2_pages_reserve(refs, table, _i64(first), _i64(g), 2)      # all of it is there
    _same(o, refs, table)
    assert np.array_equal(to_np(again), g) and (none == -1).all()


def test_the_longest_table():
    """The last pages of a row of 2^31 - 1: what lies behind it is neither looked at nor written."""
    P_ = 2 ** 31 - 1
    flat = torch.full((P_ + 1,), -1, dtype=torch.int32, device=DEV)
    table, refs = flat[:P_].view(1, P_), _i32(np.zeros(50))
    ws = torch.empty(C.load().csa2_pages_reserve_workspace_bytes(50, 1, P_), dtype=torch.uint8, device=DEV)
    for first, count, got in ((P_ - 1, 1, 1), (P_ - 3, 2, 2), (P_ - 40, 40, 40)):
        granted, copies = C.csa2_pages_reserve(refs, table, _i64([first]), _i64([count]), 1, ws=ws)
        C.csa2_ctx_check()
        assert granted.tolist() == [got] and copies.tolist() == [[-1, -1]]
    assert table[0, P_ - 40:].tolist() == [*range(3, 40), 1, 2, 0] and int(flat[P_]) == -1 and int(refs.sum()) == 40
    granted, _ = C.csa2_pages_reserve(refs, table, _i64([P_ - 2]), _i64([3]), 1, ws=ws)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()                                # (the row ends)
    assert granted.tolist() == [2]
    pool = torch.zeros(50, 1, 4, device=DEV)
    C.csa2_page_write(pool, table, torch.ones(1, 2, 4, device=DEV), _i64([P_ - 2]), granted)
    C.csa2_ctx_check()
    assert pool.sum((1, 2)).nonzero().flatten().tolist() == [0, 2]
    C.csa2_pages_free(refs, table, 1, _i64([P_ - 1]))
    C.csa2_ctx_check()
    assert int(flat[P_ - 1]) == -1 and int(refs.sum()) == 39
    C.csa2_pages_free(refs, table, 1)
    C.csa2_ctx_check()
    assert not refs.any() and bool((flat[P_ - 64:] == -1).all())


def test_what_does_not_fit_is_flagged():
    refs, table = _i32(np.zeros(4)), _i32(np.full((2, 3), -1))
    granted, _ = C.csa2_pages_reserve(refs, table, _i64([5, 9]), _i64([3, 2 ** 62]), 2)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()                                # the table's row ends at entry 6
    assert granted.tolist() == [1, 0] and table.tolist() == [[-1, -1, 0], [-1, -1, -1]] and refs.tolist() == [1, 0, 0, 0]
    for bad in (4, -2):
        t = _i32([[bad, 0, -1], [-1, -1, -1]])
        granted, copies = C.csa2_pages_reserve(refs, t, _i64([0, 0]), _i64([4, 2]), 2)
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        assert granted.tolist() == [0, 2]                 # nothing of a sequence whose first page is none
        C.csa2_pages_free(refs, t, 2, _i64([-1, 0]))
        out = C.csa2_pages_fork(refs, t, _i32([0, 2]))
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        assert out.tolist() == [[-1, 0, -1], [-1, -1, -1]] and refs.tolist() == [2, 0, 0, 0]
        C.csa2_pages_free(refs, out, 2)
        C.csa2_ctx_check()
        C.csa2_pages_compact(refs, t)
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        assert refs.tolist() == [1, 0, 0, 0]
    t = _i32([[1, 0, -1]])                                # page 1 has no uses: its count stays at 0
    C.csa2_pages_free(refs, t, 2)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert refs.tolist() == [0, 0, 0, 0] and (t == -1).all()


@pytest.mark.parametrize("row", [((288,), torch.uint8), ((68,), torch.uint8), ((512,), torch.bfloat16), ((1,), torch.float32),
                                 ((6, 50), torch.float32)])
@pytest.mark.parametrize("page,B,n", [(1, 1, 1), (16, 5, 37), (17, 3, 300)])
def test_rows_and_pages(row, page, B, n):
    shape, dt = row
    gen = torch.Generator(DEV).manual_seed(page + n)

    def noise(*lead):
        return torch.randint(0, 256, (*lead, *shape), generator=gen, device=DEV).to(dt)

    cache = P.alloc_pages(B, (n // page + 3) * B + 2, page, n // page + 3, {"x": row}, DEV)
    pool = cache.pools["x"].copy_(noise(*cache.pools["x"].shape[:2]))
    first = torch.arange(B, device=DEV) % (page + 2)
    count = torch.full((B,), n, device=DEV)
    count[-1] = n // 2
    rows, old = noise(B, n), pool.clone()
    granted, _ = C.csa2_pages_reserve(cache.refs, cache.table, first, count, page)
    C.csa2_page_write(pool, cache.table, rows, first, granted)
    C.csa2_ctx_check()
    assert torch.equal(granted, count)
    o = D.Pages(to_np(cache.refs), to_np(cache.table), page)
    want = old.clone()
    for b in range(B):
        for i in range(int(count[b])):
            want[o.place(b, int(first[b]) + i)] = rows[b, i]
    assert torch.equal(pool, want)                        # and nothing else of the pool
    idx = torch.full((B, n + 2), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        idx[b, 1:1 + int(count[b])] = (first[b] + torch.randperm(int(count[b]), generator=gen, device=DEV)).int()
    dst = noise(B, n + 2)
    got = C.csa2_page_read(pool, cache.table, idx, out=dst.clone())
    C.csa2_ctx_check()
    for b in range(B):
        live = idx[b] >= 0
        assert torch.equal(got[b][live], rows[b][(idx[b][live] - first[b]).long()]) and torch.equal(got[b][~live], dst[b][~live])
    pairs = _i32([[0, 1], [-1, -1], [-1, 0]])
    before = pool.clone()
    C.csa2_page_copy(pool, pairs)
    C.csa2_ctx_check()
    before[1] = before[0]
    assert torch.equal(pool, before)


def test_rows_that_have_no_page_are_flagged_and_left():
    pool = torch.arange(4 * 2 * 4, device=DEV, dtype=torch.float32).view(4, 2, 4)
    table, old = _i32([[2, -1], [7, 0]]), pool.clone()
    out = torch.full((2, 5, 4), -7.0, device=DEV)
    C.csa2_page_read(pool, table, _i32([[0, 1, 2, 4, -1], [0, 1, 2, -5, 3]]), out=out)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert torch.equal(out[0, :2], pool[2]) and torch.equal(out[1, 2], pool[0, 0]) and torch.equal(out[1, 4], pool[0, 1])
    assert (out[0, 2:] == -7).all() and (out[1, [0, 1, 3]] == -7).all()
    C.csa2_page_write(pool, table, torch.zeros(2, 3, 4, device=DEV), _i64([1, 4]), _i64([3, 1]))
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    old[2, 1] = 0
    assert torch.equal(pool, old)
    C.csa2_page_write(pool, table, torch.ones(2, 3, 4, device=DEV), _i64([-1, 0]), _i64([2, -4]))
    C.csa2_ctx_check()                                    # nothing to write is no error
    assert torch.equal(pool, old)
    for pair in ([4, 0], [0, 4], [-2, 0]):
        C.csa2_page_copy(pool, _i32([pair]))
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
    assert torch.equal(pool, old)


def test_long_pages_and_unaligned_pools():
    """Pages of several chunks, and a pool at 4 bytes past a 16-byte boundary."""
    flat = torch.arange(3 * 70000 * 4 + 1, device=DEV, dtype=torch.int32)
    for pool in (flat[:-1].view(3, 70000, 4), flat[1:].view(3, 70000, 4)):
        want = pool.clone()
        want[2] = want[0]
        C.csa2_page_copy(pool, _i32([[0, 2]]))
        C.csa2_ctx_check()
        assert torch.equal(pool, want)


def test_forked_sequences_append_apart():
    """Continuations of a prompt: entries that were there are shared, the ones appended are not, in every pool."""
    gen = torch.Generator(DEV).manual_seed(9)
    rows = {"kv": ((288,), torch.uint8), "ki": ((68,), torch.uint8)}

    def noise(B, n):
        return {k: torch.randint(0, 256, (B, n, *s), generator=gen, device=DEV, dtype=d) for k, (s, d) in rows.items()}

    base = P.alloc_pages(2, 64, 8, 20, rows, DEV)
    first = noise(2, 43)
    P.pages_append(base, first, _i64([43, 30]))
    beams = P.pages_fork(base, _i32([0, 0, 1, -1, 0]))
    used = int((base.refs > 0).sum())
    assert used == 6 + 4 and beams.n_entries.tolist() == [43, 43, 30, 0, 43]
    more = noise(5, 10)
    granted = P.pages_append(beams, more, _i64([10, 1, 0, 10, 6]))
    C.csa2_ctx_check()
    assert granted.tolist() == [10, 1, 0, 10, 6] and beams.n_entries.tolist() == [53, 44, 30, 10, 49]
    want = {k: [torch.cat([first[k][p, :n], more[k][i, :m]]) for i, (p, n, m) in
                enumerate([(0, 43, 10), (0, 43, 1), (1, 30, 0), (0, 0, 10), (0, 43, 6)])] for k in rows}

    def check(cache, want):
        for k, seqs in want.items():
            for b, w in enumerate(seqs):
                idx = torch.full((cache.table.shape[0], len(w)), -1, dtype=torch.int32, device=DEV)
                idx[b] = torch.arange(len(w), device=DEV)
                assert torch.equal(C.csa2_page_read(cache.pools[k], cache.table, idx)[b], w)

    check(beams, want)
    check(base, {k: [first[k][0, :43], first[k][1, :30]] for k in rows})
    P.pages_cut(base)                                     # the prompts end, their continuations stay
    P.pages_cut(beams, _i64([53, 0, -1, 4, 17]))
    assert beams.n_entries.tolist() == [53, 0, 30, 4, 17]
    n_used = P.pages_compact(beams)
    C.csa2_ctx_check()
    assert int(n_used) == int((beams.refs > 0).sum()) and int(beams.table.max()) == int(n_used) - 1
    check(beams, {k: [want[k][0], want[k][1][:0], want[k][2], want[k][3][:4], want[k][4][:17]] for k in rows})


def test_fork_of_what_is_no_sequence():
    """A parent past the sequences is flagged and gives an empty continuation, of no sequences at all too."""
    cache = P.alloc_pages(2, 20, 4, 4, {"x": ((4,), torch.float32)}, DEV)
    P.pages_append(cache, {"x": torch.rand(2, 9, 4, device=DEV)}, _i64([9, 6]))
    refs = cache.refs.tolist()
    out = P.pages_fork(cache, _i32([1, 2, -1, 2 ** 31 - 1, -2 ** 31]))
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert out.n_entries.tolist() == [6, 0, 0, 0, 0]
    assert torch.equal(out.table[0], cache.table[1]) and (out.table[1:] == -1).all()
    assert sum(out.refs.tolist()) == sum(refs) + 2
    P.pages_append(out, {"x": torch.rand(5, 2, 4, device=DEV)}, _i64([2] * 5))
    C.csa2_ctx_check()
    assert out.n_entries.tolist() == [8, 2, 2, 2, 2] and cache.n_entries.tolist() == [9, 6]
    none = P.alloc_pages(0, 20, 4, 4, {"x": ((4,), torch.float32)}, DEV)
    for parent, bad in (([-1, -1], False), ([0, -1], True), ([], False)):
        out = P.pages_fork(none, _i32(parent))
        if bad:
            with pytest.raises(C.Csa2Error):
                C.csa2_ctx_check()
        C.csa2_ctx_check()
        assert out.n_entries.tolist() == [0] * len(parent) and out.table.shape == (len(parent), 4) and (out.table == -1).all()


def test_append_takes_no_more_than_the_rows():
    """A count above the rows given appends those, so that every entry counted has been written; pools that are
    given different numbers of rows are refused before anything is reserved."""
    rows = {"kv": ((16,), torch.float32), "ki": ((4,), torch.float32)}
    cache = P.alloc_pages(3, 30, 4, 8, rows, DEV)
    for pool in cache.pools.values():
        pool.fill_(-7.0)                                  # what a page held before
    gen = torch.Generator(DEV).manual_seed(13)
    want = {k: [] for k in rows}
    for n, count, got in ((5, [9, 2, -1], [5, 2, 0]), (0, [3, 0, 1], [0, 0, 0]), (3, [3, 2 ** 40, 4], [3, 3, 3])):
        x = {k: torch.rand(3, n, *shape, generator=gen, device=DEV) for k, (shape, _) in rows.items()}
        counts = _i64(count)
        assert P.pages_append(cache, x, counts).tolist() == got
        assert counts.tolist() == count                   # the caller's tensor stays
        for k in rows:
            want[k].append([x[k][b, :m] for b, m in enumerate(got)])
    C.csa2_ctx_check()
    assert cache.n_entries.tolist() == [8, 5, 3]
    for k in rows:
        for b, m in enumerate([8, 5, 3]):
            idx = torch.full((3, m), -1, dtype=torch.int32, device=DEV)
            idx[b] = torch.arange(m, device=DEV)
            assert torch.equal(C.csa2_page_read(cache.pools[k], cache.table, idx)[b], torch.cat([w[b] for w in want[k]]))
    state = [x.clone() for x in (cache.refs, cache.table, cache.n_entries)]
    x = {k: torch.rand(3, 6, *shape, device=DEV) for k, (shape, _) in rows.items()}
    for bad in ({**x, "ki": x["ki"][:, :4].contiguous()}, {"kv": x["kv"]}, {}):
        with pytest.raises(ValueError, match="as many rows"):
            P.pages_append(cache, bad, _i64([6, 6, 6]))
    for a, b in zip(state, (cache.refs, cache.table, cache.n_entries)):
        assert torch.equal(a, b)


def test_captured_step_of_a_branch():
    """Fork, reserve, copy and write recorded once and replayed: the state moves on as by eager calls."""
    gen = torch.Generator(DEV).manual_seed(11)
    cache = P.alloc_pages(2, 40, 4, 8, {"x": ((16,), torch.float32)}, DEV)
    P.pages_append(cache, {"x": torch.rand(2, 9, 16, generator=gen, device=DEV)}, _i64([9, 6]))
    pool, parent, rows = cache.pools["x"], _i32([0, 1, 1]), torch.rand(3, 5, 16, generator=gen, device=DEV)
    first, count = cache.n_entries[parent.long()].contiguous(), _i64([5, 1, 5])
    work, granted, copies = torch.full_like(cache.table[:1].expand(3, -1), -1), _i64([0] * 3), _i32(np.zeros((3, 2)))
    work = work.contiguous()
    ws = torch.empty(C.load().csa2_pages_reserve_workspace_bytes(40, 3, 8), dtype=torch.uint8, device=DEV)

    def step():
        C.csa2_pages_free(cache.refs, work, 4)
        C.csa2_pages_fork(cache.refs, cache.table, parent, out=work)
        C.csa2_pages_reserve(cache.refs, work, first, count, 4, granted=granted, copies=copies, ws=ws)
        C.csa2_page_copy(pool, copies)
        C.csa2_page_write(pool, work, rows, first, granted)

    step()
    want = [x.clone() for x in (cache.refs, work, granted, copies, pool)]
    graph = torch.cuda.CUDAGraph()
    check, C._check = C._check, lambda fn, st: None if st == C.OK else pytest.fail(fn)
    try:
        with torch.cuda.graph(graph):
            step()
    finally:
        C._check = check
    rows.mul_(2.0)
    for _ in range(3):
        graph.replay()
    C.csa2_ctx_check()
    for x, w in zip((cache.refs, work, granted, copies), want):
        assert torch.equal(x, w)
    idx = torch.arange(14, dtype=torch.int32, device=DEV).expand(3, 14)
    idx = torch.where(idx < (first + count).unsqueeze(-1), idx, -1).to(torch.int32).contiguous()
    got = C.csa2_page_read(pool, work, idx)
    for i in range(3):
        f, n = int(first[i]), int(count[i])
        assert torch.equal(got[i, f:f + n], rows[i, :n])


@pytest.mark.parametrize("n_pages,B,P_", [(9, 2, 3), (300, 7, 30), (3000, 33, 41), (5000, 3, 20001), (2, 1, 1), (1, 1, 1)])
@pytest.mark.parametrize("off", [0, 1])
def test_compaction_without_all_tables_moves_nothing(n_pages, B, P_, off):
    """Pages that a table outside the call holds would move away under it: flagged, and everything stays."""
    o, rng = _random(n_pages + 1, n_pages, B, P_, 4, fill=min(1.0, 0.7 * n_pages / (B * P_)))
    free = np.flatnonzero(o.refs == 0)
    o.refs[rng.permutation(free)[:len(free) // 2]] = 0
    if not o.refs.any():
        o.refs[0], o.table[0, 0] = 1, 0
    refs, _ = _state(o)
    flat = torch.full((B * P_ + 1,), -1, dtype=torch.int32, device=DEV)
    table = flat[off:off + B * P_].view(B, P_).copy_(_i32(o.table))    # (off: not on a 16-byte boundary)
    held = int(rng.choice(np.flatnonzero(o.refs)))
    for page, d in ((held, 1), (held, -1), (int(np.argmin(o.refs)), 1)):
        r = refs.clone()
        r[page] += d
        before, t = r.clone(), table.clone()
        moves, n_used = C.csa2_pages_compact(r, table)
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        assert torch.equal(r, before) and torch.equal(table, t) and (moves == -1).all() and int(n_used) == n_pages
    moves, n_used = C.csa2_pages_compact(refs, table)
    C.csa2_ctx_check()
    want, cut = o.compact()
    _same(o, refs, table)
    assert np.array_equal(to_np(moves), want) and int(n_used) == cut


@pytest.mark.parametrize("P_", [12, 9000])
def test_compaction_of_prompts_and_continuations(P_):
    """The caches of prompts and of their continuations, each with its table, over one pool: alone either one's
    compaction is refused, together both find their entries again."""
    gen = torch.Generator(DEV).manual_seed(19)
    base = P.alloc_pages(3, 60, 4, P_, {"x": ((4,), torch.float32), "y": ((3,), torch.float32)}, DEV)

    def rows(B, n):
        return {k: torch.rand(B, n, w, generator=gen, device=DEV) for k, w in (("x", 4), ("y", 3))}

    x = rows(3, 20)
    P.pages_append(base, x, _i64([20, 9, 15]))
    beams = P.pages_fork(base, _i32([0, 0, 2, 1]))
    y = rows(4, 6)
    P.pages_append(beams, y, _i64([6, 1, 3, 0]))
    wide = P.PagedCache(base.pools, base.refs, torch.full((1, 2), -1, dtype=torch.int32, device=DEV), _i64([0]))
    z = rows(1, 5)
    P.pages_append(wide, z, _i64([5]))                    # a table of another width over the same pools
    P.pages_cut(base, _i64([-1, 0, 6]))
    C.csa2_ctx_check()
    first = {"base": (20, 0, 6), "beams": ((0, 20, 6), (0, 20, 1), (2, 15, 3), (1, 9, 0))}

    def check():
        for k in ("x", "y"):
            want = [(base, [x[k][b, :n] for b, n in enumerate(first["base"])]), (wide, [z[k][0]]),
                    (beams, [torch.cat([x[k][p, :n], y[k][i, :m]]) for i, (p, n, m) in enumerate(first["beams"])])]
            for cache, seqs in want:
                for b, w in enumerate(seqs):
                    idx = torch.full((len(seqs), len(w)), -1, dtype=torch.int32, device=DEV)
                    idx[b] = torch.arange(len(w), device=DEV)
                    assert torch.equal(C.csa2_page_read(cache.pools[k], cache.table, idx)[b], w)
        C.csa2_ctx_check()

    check()
    used = int((base.refs > 0).sum())
    for some in ((base,), (beams,), (base, beams), (wide, beams)):
        assert int(P.pages_compact(*some)) == 60
        with pytest.raises(C.Csa2Error):
            C.csa2_ctx_check()
        check()
    assert int(base.refs[used:].sum()) > 0                # (there is something to move)
    assert int(P.pages_compact(beams, wide, base)) == used
    C.csa2_ctx_check()
    assert not base.refs[used:].any() and max(int(c.table.max()) for c in (base, beams, wide)) == used - 1
    check()
    other = P.alloc_pages(1, 60, 4, 4, {"x": ((4,), torch.float32)}, DEV)
    with pytest.raises(ValueError, match="same pools"):
        P.pages_compact(base, other)


def test_captured_appends_go_on(monkeypatch):
    """pages_append and pages_cut recorded once: every replay appends behind the entries of the one before."""
    monkeypatch.setattr(C, "alloc", lambda shape, dtype, device: torch.empty(shape, dtype=dtype, device=device))
    gen = torch.Generator(DEV).manual_seed(17)
    cache = P.alloc_pages(2, 40, 4, 12, {"x": ((16,), torch.float32)}, DEV)
    rows, count, keep = torch.zeros(2, 5, 16, device=DEV), _i64([5, 2]), _i64([-1, -1])
    want = [torch.zeros(0, 16, device=DEV)] * 2

    def step():
        P.pages_cut(cache, keep)
        return P.pages_append(cache, {"x": rows}, count)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()                                            # (warm-up: five and two entries of zeros)
        P.pages_cut(cache)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        granted = step()
    assert cache.n_entries.tolist() == [0, 0]             # recorded, not run
    for cut in ([-1, -1], [-1, -1], [3, -1], [100, 1], [0, 4]):
        x = torch.rand(2, 5, 16, generator=gen, device=DEV)
        rows.copy_(x)
        keep.copy_(_i64(cut))
        graph.replay()
        C.csa2_ctx_check()
        assert granted.tolist() == [5, 2]
        want = [torch.cat([w if k < 0 else w[:k], x[b, :n]]) for b, (w, k, n) in enumerate(zip(want, cut, (5, 2)))]
        assert cache.n_entries.tolist() == [len(w) for w in want]
        for b, w in enumerate(want):
            idx = torch.full((2, len(w)), -1, dtype=torch.int32, device=DEV)
            idx[b] = torch.arange(len(w), device=DEV)
            assert torch.equal(C.csa2_page_read(cache.pools["x"], cache.table, idx)[b], w)
    assert int(cache.refs.sum()) == int((cache.table >= 0).sum())


def test_empty_calls():
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    t0 = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    C.csa2_pages_free(none, t0, 4)
    m, n = C.csa2_pages_compact(none, t0)
    assert m.shape == (0, 2) and int(n) == 0
    refs, t = _i32(np.zeros(3)), _i32(np.zeros((2, 0)))
    assert C.csa2_pages_fork(refs, t, _i32([0])).shape == (1, 0)
    granted, copies = C.csa2_pages_reserve(refs, t, _i64([0, 0]), _i64([0, 1]), 4)
    with pytest.raises(C.Csa2Error):
        C.csa2_ctx_check()
    assert granted.tolist() == [0, 0] and (copies == -1).all()
    granted, _ = C.csa2_pages_reserve(none, _i32([[-1, -1]]), _i64([0]), _i64([2]), 4)
    C.csa2_ctx_check()
    assert granted.tolist() == [0]
    C.csa2_page_write(torch.zeros(3, 4, 5, device=DEV), t, torch.zeros(2, 0, 5, device=DEV), _i64([0, 0]), _i64([0, 0]))
    C.csa2_page_copy(torch.zeros(3, 4, 5, device=DEV), _i32(np.zeros((0, 2))))
    C.csa2_ctx_check()
