"""Cases of the operators for drafting and for shared caches: attention for a tree of drafted tokens
over a cache (its rows one block a sequence, or in pages), and the pages themselves: continuations
that share a prompt's pages and then append to them, a pool whose used pages are moved together,
and rows read through the page table.

Every case runs in plain torch (`own` false) or through the framework's entry points."""
import math

import torch

own = False
DEV = "cuda"
C = 512          # channels of a main cache row
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # ordinary decode through the same call: one token of one sequence, nothing drafted beside it
        dict(name="tree bf16 1x1", op="tree", dtype="bf16", form="sparse", B=1, T=1, H=64, N=16384, k=512, m=4,
             window=128, page=0, ragged=False),
        # a small fp32 layer with odd sizes and unused nodes, as a check of a model runs it
        dict(name="tree f32 2x13 odd", op="tree", dtype="f32", form="sparse", B=2, T=13, H=16, N=997, k=301, m=2,
             window=100, page=16, ragged=True),
        # eight sequences of a 256K context, 32 drafted tokens each, FP4 rows in pages, each node's own selection
        dict(name="tree fp4 8x32 paged", op="tree", dtype="fp4", form="sparse", B=8, T=32, H=64, N=65536, k=512, m=4,
             window=128, page=64, ragged=False),
        # four sequences, wide trees over the heavily compressed cache of a 512K context, rows shared by the nodes
        dict(name="tree bf16 4x64 dense paged", op="tree", dtype="bf16", form="dense", B=4, T=64, H=64, N=4096, k=4096,
             m=128, window=128, page=64, ragged=False),
        # the wide configuration: 128 heads, top-1024, eight sequences of ragged lengths
        dict(name="tree bf16 8x24 h128 top1024", op="tree", dtype="bf16", form="sparse", B=8, T=24, H=128, N=16384, k=1024,
             m=4, window=128, page=32, ragged=True),
        # one prompt continued eight ways, two new entries each
        dict(name="branch fp4 1 to 8", op="branch", dtype="fp4", B=8, prompts=1, N=1000, n=2, page=64),
        # beams of 16 prompts that each append an odd piece
        dict(name="branch bf16 16 to 64", op="branch", dtype="bf16", B=64, prompts=16, N=4093, n=77, page=32),
        # eight prompts of 64K entries that get a long document each, in eight ways
        dict(name="branch bf16 8 to 64 long", op="branch", dtype="bf16", B=64, prompts=8, N=8191, n=4096, page=64),
        # a small pool after a few requests ended
        dict(name="compact bf16 300 pages", op="compact", dtype="bf16", B=9, pages=300, page=16, used=0.6),
        # a large FP4 pool, half of it given back in pieces
        dict(name="compact fp4 40000 pages", op="compact", dtype="fp4", B=128, pages=40000, page=64, used=0.5),
        # the rows of one selection, to be kept together
        dict(name="read fp4 1x512", op="read", dtype="fp4", B=1, N=65536, keep=512, page=64),
        # a cut of many ragged sequences, rows read out of their pages
        dict(name="read bf16 32x4001", op="read", dtype="bf16", B=32, N=9001, keep=4001, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "branch", "compact", "read"])
    page = rng.choice([1, 16, 17, 32, 64, 64, 128])
    if op == "tree":
        form = rng.choice(["sparse", "sparse", "dense"])
        dtype = rng.choice(["bf16", "bf16", "fp4", "fp4", "f32"])
        H = rng.choice([8, 16, 40, 64, 64, 100, 128])
        window = rng.choice([1, 100, 128, 128, 200])
        B = _log(rng, 1, 16)
        k = _log(rng, 1, 4096 if form == "dense" else 1024)
        # slots x heads: at most a quarter of the largest case's (an eighth of that in fp32)
        budget = 4 * 64 * 64 * 4096 // (32 if dtype == "f32" else 4)
        T = max(1, min(_log(rng, 1, 128), budget // (B * H * (k + window))))
        N = k if form == "dense" else k + _log(rng, 1, 65536 // B)
        return dict(op=op, dtype=dtype, form=form, B=B, T=T, H=H, N=N, k=k, m=128 if form == "dense" else rng.choice([1, 2, 4]),
                    window=window, page=rng.choice([0, page, page]), ragged=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp4"])
    row = 1280 if dtype == "bf16" else 356
    if op == "branch":
        B = _log(rng, 1, 64)
        n = max(1, min(_log(rng, 1, 4096), (1 << 28) // (row * B)))
        prompts = rng.randint(1, B)
        N = max(1, min(_log(rng, 1, 16384), (1 << 28) // (row * prompts)))
        return dict(op=op, dtype=dtype, B=B, prompts=prompts, N=N, n=n, page=page)
    if op == "compact":
        pages = max(2, min(_log(rng, 2, 60000), (1 << 29) // (row * page)))
        return dict(op=op, dtype=dtype, B=rng.randint(1, 100), pages=pages, page=page, used=rng.uniform(0.05, 0.95))
    B = _log(rng, 1, 32)
    N = max(1, min(_log(rng, 1, 65536), (1 << 28) // (row * B)))
    return dict(op=op, dtype=dtype, B=B, N=N, keep=max(1, int(N * rng.uniform(0.02, 1.0))), page=page)


# ------------------------------------------------------------------ pieces of the plain forms (32 bits)
def _rope(x, pos, sign):
    """Rotates the last 64 of x's 512 channels by sign * pos (pos broadcasts over x's leading axes);
    angles in 64 bits."""
    j = torch.arange(32, dtype=torch.float64, device=x.device)
    turns = pos.double().unsqueeze(-1) * (10000.0 ** (-2.0 * j / 64.0) / (2.0 * math.pi))
    ang = (turns - turns.floor()) * (2.0 * math.pi)
    cs, sn = ang.cos().to(x.dtype), (sign * ang.sin()).to(x.dtype)
    a, b = x[..., C - 64::2], x[..., C - 63::2]
    return torch.cat([x[..., :C - 64], torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)], -1)


def _rms(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(rows, dtype):
    """Rows as values: fp32 or bf16 rows, or FP4 rows [..., 288] (256 code bytes, low nibble first,
    then 32 E4M3 scales)."""
    if rows.dtype != torch.uint8:
        return rows.to(dtype)
    table = torch.tensor(_E2M1, dtype=dtype, device=rows.device)
    b = rows[..., :256].long()
    v = torch.stack([table[b & 15], table[b >> 4]], -1).flatten(-2)
    s = rows[..., 256:].contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (v.unflatten(-1, (32, 16)) * s.unsqueeze(-1)).flatten(-2)


def _plan(s):
    """Who is on whose path [B, T, T], the nodes' positions (-1: unused) and their paths by depth."""
    par = s["parent"].long()
    B, T = par.shape
    j = torch.arange(T, device=DEV)
    reach = ((par.unsqueeze(-1) == j) | (j.unsqueeze(-1) == j)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    unused = ((reach @ (par < -1).float().unsqueeze(-1)) > 0).squeeze(-1)
    on = (reach > 0) & ~unused.unsqueeze(-1)
    depth = on.sum(-1) - 1
    pos = torch.where(unused, -1, s["ctx_len"].unsqueeze(-1) + depth)
    at = torch.where(on, depth.unsqueeze(1), T).clamp(min=0)             # path slot of every node on the path
    path = torch.full((B, T, T + 1), -1, dtype=torch.int64, device=DEV)
    path.scatter_(2, at, j.expand(B, T, T))
    return on, pos, path[..., :T].to(torch.int16)


def _tree(s):
    on, pos, path = _plan(s)
    B, T, H, _ = s["q"].shape
    W, k = s["window"], s["k"]
    outs = []
    for b in range(B):
        L, t = s["ctx_len"][b], pos[b]
        qh = _rope(_rms(s["q"][b].float()), t.unsqueeze(-1), 1.0)                        # [T, H, C]
        p = L - W + 1 + torch.arange(W - 1, device=DEV)
        near = torch.cat([s["swa"][b][(p - s["swa_pos0"]) % s["swa"].shape[1]], s["draft"][b]])
        okn = torch.cat([((p >= 0) & (p > (t - W).unsqueeze(-1))) & (t >= 0).unsqueeze(-1),
                         on[b] & (t > (t - W).unsqueeze(-1))], -1)                      # [T, W - 1 + T]
        if s["idx"] is not None:
            e = s["idx"][b].long()
            ok = (e >= 0) & (t >= 0).unsqueeze(-1)
            far = _rms(_values(_entries(s, b, e.clamp(min=0)), torch.float32))          # [T, k, C]
        else:
            e = torch.arange(k, device=DEV)
            ok = (e < s["n_visible"][b].unsqueeze(-1)) & (t >= 0).unsqueeze(-1)
            e = torch.minimum(e, s["n_visible"][b].max().clamp(min=1) - 1)
            far = _rms(_values(_entries(s, b, e), torch.float32))                       # [k, C]
        near = _rms(near.float())
        z = torch.cat([qh @ far.transpose(-1, -2), qh @ near.t()], -1) / math.sqrt(C)
        z.masked_fill_(~torch.cat([ok, okn], -1).unsqueeze(1), -math.inf)
        top = z.amax(-1, keepdim=True)
        if s["sink"] is not None:
            top = torch.maximum(top, s["sink"].view(1, H, 1))
        top = top.masked_fill(top == -math.inf, 0.0)
        z = torch.exp(z - top)
        den = z.sum(-1, keepdim=True)
        if s["sink"] is not None:
            den = den + torch.exp(s["sink"].view(1, H, 1) - top)
        z = z / torch.where(den > 0, den, torch.ones_like(den))
        outs.append(_rope(z[..., :k] @ far + z[..., k:] @ near, t.unsqueeze(-1), -1.0))
    return pos, path, torch.stack(outs).to(s["q"].dtype)


def _entries(s, b, e):
    """Rows of entries e of sequence b."""
    if s["table"] is None:
        return s["kv"][b][e]
    page = s["kv"].shape[1]
    return s["kv"].flatten(0, 1)[s["table"][b].long()[e // page] * page + e % page]


def _uses(refs, pages, add):
    """refs += add for every page of `pages` that is one."""
    live = pages >= 0
    refs.scatter_add_(0, pages.clamp(min=0).flatten().long(), torch.where(live, add, 0).flatten().to(refs.dtype))


def _branch(s):
    refs, page = s["refs"], s["page"]
    # the last round's continuations are given up, the prompts' pages shared out again
    _uses(refs, s["work"], torch.full_like(s["work"], -1))
    work = s["table"][s["parent"].long()]
    _uses(refs, work, torch.ones_like(work))
    # pages of the entries to come: missing or shared ones are replaced by the lowest free ones
    B, P = work.shape
    first, n = s["first"].unsqueeze(-1), s["count"].unsqueeze(-1)
    j = torch.arange(P, device=DEV)
    need = (n > 0) & (j >= first // page) & (j < (first + n + page - 1) // page)
    shared = (work >= 0) & (refs[work.clamp(min=0).long()] > 1)
    want = need & ((work < 0) | shared)
    rank = torch.cumsum(want.flatten().long(), 0).view(B, P) - 1
    free = torch.sort((refs > 0).to(torch.int8), stable=True).indices
    ok = want & (rank < (refs == 0).sum())
    new = torch.where(ok, free[rank.clamp(min=0, max=free.numel() - 1)].to(torch.int32), work)
    lacks = torch.where(want & ~ok, j, P + 1).amin(-1, keepdim=True)
    granted = torch.minimum(n, lacks * page - first).clamp(min=0).squeeze(-1)
    cow = ok & shared & (j == first // page) & (first % page != 0)
    copies = torch.stack([torch.where(cow, x, -1).amax(-1) for x in (work, new)], -1)
    _uses(refs, torch.where(ok, work, -1), torch.full_like(work, -1))
    _uses(refs, torch.where(ok, new, -1), torch.ones_like(work))
    s["work"].copy_(new)
    # shared beginnings copied, rows written
    i = torch.arange(s["rows"][0].shape[1], device=DEV)
    e = first + i
    b, r = torch.nonzero(i < granted.unsqueeze(-1), as_tuple=True)
    at = new[b, e[b, r] // page].long() * page + e[b, r] % page
    moved = copies[copies[:, 0] >= 0].long()
    for pool, rows in zip(s["pools"], s["rows"]):
        pool[moved[:, 1]] = pool[moved[:, 0]]
        pool.flatten(0, 1)[at] = rows[b, r]
    return [s["work"], refs, granted, copies, *s["pools"]]


def _compact(s):
    table, refs = s["table"].copy_(s["table0"]), s["refs"].copy_(s["refs0"])
    n = refs.numel()
    ids = torch.arange(n, device=DEV)
    used = refs > 0
    n_used = used.sum()
    src, dst = used & (ids >= n_used), ~used & (ids < n_used)
    half = n // 2
    live = torch.arange(half, device=DEV) < src.sum()
    pairs = [torch.sort((~x).to(torch.int8), stable=True).indices[:half] for x in (src, dst)]
    moves = torch.where(live.unsqueeze(-1), torch.stack(pairs, -1), -1).to(torch.int32)
    moved = moves[moves[:, 0] >= 0].long()
    to = ids.clone()
    to[moved[:, 0]] = moved[:, 1]
    refs[moved[:, 1]] = refs[moved[:, 0]]
    refs[moved[:, 0]] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    for pool in s["pools"]:
        pool[moved[:, 1]] = pool[moved[:, 0]]
    return [table, refs, moves, n_used.view(1), *s["pools"]]


def _read(s):
    page = s["page"]
    e = s["idx"].long().clamp(min=0)
    at = torch.gather(s["table"].long(), 1, e // page) * page + e % page
    live = (s["idx"] >= 0).unsqueeze(-1)
    for pool, out in zip(s["pools"], s["outs"]):
        out.copy_(torch.where(live, pool.flatten(0, 1)[at], out))
    return s["outs"]


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from compressed_sparse_attention_06_gb300 import csa2

    op = s["op"]
    if op == "tree":
        pos, path = csa2.csa2_tree_plan(s["parent"], s["ctx_len"])
        out, _ = csa2.csa2_tree_attn(s["q"], s["kv"], pos, path, s["ctx_len"], s["swa"], s["draft"], idx=s["idx"],
                                     n_visible=s["n_visible"], k_max=s["k"], table=s["table"], sink=s["sink"],
                                     window=s["window"], swa_pos0=s["swa_pos0"])
        return pos, path, out
    if op == "branch":
        work, refs, page = s["work"], s["refs"], s["page"]
        csa2.csa2_pages_free(refs, work, page)
        csa2.csa2_pages_fork(refs, s["table"], s["parent"], out=work)
        granted, copies = csa2.csa2_pages_reserve(refs, work, s["first"], s["count"], page)
        for pool, rows in zip(s["pools"], s["rows"]):
            csa2.csa2_page_copy(pool, copies)
            csa2.csa2_page_write(pool, work, rows, s["first"], granted)
        return [work, refs, granted, copies, *s["pools"]]
    if op == "compact":
        table, refs = s["table"].copy_(s["table0"]), s["refs"].copy_(s["refs0"])
        moves, n_used = csa2.csa2_pages_compact(refs, table)
        for pool in s["pools"]:
            csa2.csa2_page_copy(pool, moves)
        return [table, refs, moves, n_used, *s["pools"]]
    for pool, out in zip(s["pools"], s["outs"]):
        csa2.csa2_page_read(pool, s["table"], s["idx"], out=out)
    return s["outs"]


def run(state):
    if own:
        return _own(state)
    return {"tree": _tree, "branch": _branch, "compact": _compact, "read": _read}[state["op"]](state)


# ------------------------------------------------------------------ inputs
def _fp4_rows(gen, rows):
    """FP4 rows of normal values with a log-normal size per row."""
    x = torch.randn(rows, C, generator=gen, device=DEV)
    x = x * torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=DEV))
    g = x.view(rows, 32, 16)
    s = (g.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = (g / s.float().clamp(min=2.0 ** -9).unsqueeze(-1)).view(rows, C)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(y.abs(), edges) + 8 * (y < 0)
    return torch.cat([(code[:, ::2] + 16 * code[:, 1::2]).to(torch.uint8), s.view(torch.uint8)], 1)


def _cache_rows(gen, dtype, *shape):
    n = math.prod(shape)
    if dtype == "fp4":
        some = _fp4_rows(gen, min(n, 1 << 14))
        return some[torch.randint(0, some.shape[0], shape, generator=gen, device=DEV)]
    return torch.randn(*shape, C, generator=gen, device=DEV).to(torch.float32 if dtype == "f32" else torch.bfloat16)


def _byte_pools(gen, dtype, pages, page):
    """Main rows and indexer keys of a pool: pages are moved as they are, whatever they hold."""
    def noise(*shape):
        return torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.uint8)
    if dtype == "fp4":
        return [noise(pages, page, 288), noise(pages, page, 68)]
    return [torch.randn(pages, page, n, generator=gen, device=DEV, dtype=torch.bfloat16) for n in (C, 128)]


def _selection(gen, v, k, T):
    """A selection as an indexer makes it for the T nodes of a tree: distinct ascending entries of the
    v[b] visible ones, neighbours sharing much of theirs, all of them where there are no more than k."""
    B = v.shape[0]
    base = torch.rand(B, 1, k, generator=gen, device=DEV)
    u = torch.where(torch.rand(B, T, k, generator=gen, device=DEV) < 0.6, base,
                    torch.rand(B, T, k, generator=gen, device=DEV)).double()
    j = torch.arange(k, device=DEV, dtype=torch.float64)
    v = v.view(B, 1, 1).double()
    lo, hi = torch.floor(j * v / k), torch.floor((j + 1) * v / k)
    ids = torch.minimum(lo + torch.floor(u * (hi - lo)), hi - 1)
    return torch.where(v <= k, torch.where(j < v, j.expand_as(ids), -torch.ones_like(ids)), ids).to(torch.int32)


def _prepare_tree(case, gen):
    B, T, H, N, k, W = (case[x] for x in ("B", "T", "H", "N", "k", "window"))
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    s = dict(op="tree", window=W, k=k)
    # entries a sequence has; the drafted tokens have none yet
    n = torch.full((B,), N, dtype=torch.int64, device=DEV)
    if case["ragged"]:
        n = torch.randint(0, N + 1, (B,), generator=gen, device=DEV)
    s["ctx_len"] = n * case["m"] + torch.randint(0, case["m"], (B,), generator=gen, device=DEV)
    # the tree: early nodes have more children, a tenth of the nodes are alternatives for the first token
    u = torch.rand(B, T, generator=gen, device=DEV)
    i = torch.arange(T, device=DEV)
    par = torch.floor(u * u * i).long().clamp(max=T)
    par = torch.where((i == 0) | (torch.rand(B, T, generator=gen, device=DEV) < 0.1), -1, torch.minimum(par, i - 1))
    if case["ragged"]:
        nodes = torch.randint(max(1, T // 2), T + 1, (B, 1), generator=gen, device=DEV)
        par = torch.where(i < nodes, par, -2)
    s["parent"] = par.to(torch.int32)
    page = case["page"]
    if page:
        # the sequences continue one prompt: the first half of their pages is the same
        P = (N + page - 1) // page
        common = P // 2
        perm = torch.randperm(common + B * (P - common) + 3, generator=gen, device=DEV).to(torch.int32)
        rest = perm[common:common + B * (P - common)].view(B, P - common)
        s["table"] = torch.cat([perm[:common].expand(B, common), rest], 1).contiguous()
        s["kv"] = _cache_rows(gen, case["dtype"], perm.numel(), page)
    else:
        s["table"] = None
        s["kv"] = _cache_rows(gen, case["dtype"], B, N)
    s["q"], s["draft"] = normal(B, T, H, C, dtype=dt), normal(B, T, C, dtype=dt)
    s["swa_pos0"] = int(torch.randint(0, 1000, (1,), generator=torch.Generator().manual_seed(N + T)))
    s["swa"] = normal(B, W + T, C, dtype=dt)
    s["sink"] = normal(H)
    if case["form"] == "dense":
        s["idx"], s["n_visible"] = None, n.unsqueeze(-1).expand(B, T).contiguous()
    else:
        s["idx"], s["n_visible"] = _selection(gen, n, k, T), None
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=DEV)

    op, page = case["op"], case.get("page")
    if op == "tree":
        return _prepare_tree(case, gen)
    s = dict(op=op, page=page)
    B = case["B"]
    if op == "branch":
        prompts, N, n = case["prompts"], case["N"], case["n"]
        length = ints(max(1, N // 2), N + 1, prompts)
        have, P = (N + page - 1) // page, (N + n + page - 1) // page
        total = prompts * have + B * (P - N // (2 * page) + 1)
        perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
        table = torch.full((prompts, P), -1, dtype=torch.int32, device=DEV)
        table[:, :have] = perm[:prompts * have].view(prompts, have)
        table[torch.arange(P, device=DEV) * page >= length.unsqueeze(-1)] = -1
        refs = torch.zeros(total, dtype=torch.int32, device=DEV)
        _uses(refs, table, torch.ones_like(table))
        s["parent"] = torch.cat([torch.arange(prompts, device=DEV), ints(0, prompts, B - prompts)]).to(torch.int32)
        s["first"] = length[s["parent"].long()].contiguous()
        s["count"] = ints(max(1, n // 2), n + 1, B)
        s.update(table=table, refs=refs, work=torch.full((B, P), -1, dtype=torch.int32, device=DEV))
        s["pools"] = _byte_pools(gen, case["dtype"], total, page)
        s["rows"] = [x.view(B, n, -1) for x in _byte_pools(gen, case["dtype"], B, n)]
        return s
    if op == "compact":
        pages = case["pages"]
        used = torch.rand(pages, generator=gen, device=DEV) < case["used"]
        # the used pages dealt out to the sequences, every tenth shared by a second one
        P = (pages + B - 1) // B
        perm = torch.randperm(pages, generator=gen, device=DEV)
        table = torch.full((B, P + P // 10 + 1), -1, dtype=torch.int32, device=DEV)
        mine = torch.full((B * P,), -1, dtype=torch.int64, device=DEV)
        mine[:pages] = torch.where(used[perm], perm, -1)
        table[:, :P] = mine.view(B, P).to(torch.int32)
        table[:, P:P + P // 10] = table[:, :P // 10].roll(1, 0)
        refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        _uses(refs, table, torch.ones_like(table))
        s.update(table0=table, refs0=refs, table=table.clone(), refs=refs.clone())
        s["pools"] = _byte_pools(gen, case["dtype"], pages, page)
        return s
    N, keep = case["N"], case["keep"]
    P = (N + page - 1) // page
    s["table"] = torch.randperm(B * P, generator=gen, device=DEV).to(torch.int32).view(B, P)
    s["pools"] = _byte_pools(gen, case["dtype"], B * P, page)
    # a cut's entries: ascending, and -1 behind those of a shorter sequence
    j = torch.arange(keep, device=DEV, dtype=torch.float64)
    u = torch.rand(B, keep, generator=gen, device=DEV).double()
    lo, hi = torch.floor(j * N / keep), torch.floor((j + 1) * N / keep)
    idx = torch.minimum(lo + torch.floor(u * (hi - lo)), hi - 1).to(torch.int32)
    kept = torch.full((B, 1), keep, device=DEV) if B == 1 else ints(keep // 2, keep + 1, B, 1)
    s["idx"] = torch.where(torch.arange(keep, device=DEV) < kept, idx, -1).to(torch.int32)
    s["outs"] = [torch.zeros(B, keep, x.shape[-1], dtype=x.dtype, device=DEV) for x in s["pools"]]
    return s


# ------------------------------------------------------------------ work and the 64-bit answers
def work(case):
    op, B = case["op"], case["B"]
    if op == "tree":
        T, H, N, k, W = (case[x] for x in ("T", "H", "N", "k", "window"))
        e = 4 if case["dtype"] == "f32" else 2
        row = 288 if case["dtype"] == "fp4" else C * e
        few = 0.5 if case["ragged"] else 1.0                  # half of the entries on average
        # paged sequences share the first half of their pages
        most = N * (1 + B) / 2 if case["page"] and N > 2 * case["page"] else B * N
        picked = min(few * most, B * T * k)
        ids = B * T * 4 * k if case["form"] == "sparse" else B * T * 8
        near = B * (min(W, N * case["m"]) + T) * C * e
        nodes = B * T * (0.75 if case["ragged"] else 1.0)
        slots = k if case["form"] == "sparse" else k * few
        return {"bytes": int(2 * B * T * H * C * e + picked * row + near + ids + B * T * (4 + 8 + 2 * T) + 4 * H),
                "flops": int(4 * nodes * H * (slots + W) * C)}
    row = 288 + 68 if case["dtype"] == "fp4" else 2 * (C + 128)
    page = case["page"]
    if op == "branch":
        P = (case["N"] + case["n"] + page - 1) // page
        rows = B * case["n"] * 0.75 + (B * page * 0.5 if page > 1 else 0)
        return {"bytes": int(2 * rows * row + (2 * B + case["prompts"]) * P * 4 + B * P * 4), "flops": 0}
    if op == "compact":
        moved = case["pages"] * case["used"] * (1 - case["used"])
        return {"bytes": int(2 * moved * page * row + case["pages"] * 16), "flops": 0}
    kept = B * case["keep"] * (0.75 if B > 1 else 1.0)
    return {"bytes": int(2 * kept * row + B * case["keep"] * 4), "flops": 0}


def _spin(x, pos, sign):
    """x with its last 64 channels as 32 complex numbers turned by sign * pos * base^(-j/32)."""
    j = torch.arange(32, dtype=torch.float64, device=x.device)
    ang = sign * float(pos) * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device), -j / 32)
    z = torch.view_as_complex(x[..., -64:].contiguous().unflatten(-1, (32, 2))) * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([x[..., :-64], torch.view_as_real(z).flatten(-2)], -1)


def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def exact(case, seed):
    """Node by node, each walking up its own path; pages are moved, not computed."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    B, T, H, _ = s["q"].shape
    W, cap = s["window"], s["swa"].shape[1]
    out = torch.zeros(B, T, H, C, dtype=torch.float64, device=DEV)
    parent, ctx = s["parent"].tolist(), s["ctx_len"].tolist()
    for b in range(B):
        shared = None
        if s["idx"] is None:
            count = s["n_visible"][b].tolist()
            shared = _unit(_values(_entries(s, b, torch.arange(max(count), device=DEV)), torch.float64)) if max(count) else None
        ring, draft = _unit(s["swa"][b].double()), _unit(s["draft"][b].double())
        for i in range(T):
            up, j = [], i
            while j >= 0:
                up.append(j)
                j = parent[b][j]
            if j < -1:
                continue
            t = ctx[b] + len(up) - 1
            older = [(p - s["swa_pos0"]) % cap for p in range(max(0, t - W + 1), ctx[b])]
            if s["idx"] is None:
                rows = [shared[:count[i]]] if count[i] else []
            else:
                e = s["idx"][b, i].long()
                rows = [_unit(_values(_entries(s, b, e[e >= 0]), torch.float64))]
            rows = torch.cat(rows + [ring[older], draft[up[:W]]])
            z = _spin(_unit(s["q"][b, i].double()), t, 1.0) @ rows.t() / C ** 0.5
            if s["sink"] is not None:
                z = torch.cat([z, s["sink"].double().unsqueeze(-1)], -1)
            out[b, i] = _spin(torch.softmax(z, -1)[:, :rows.shape[0]] @ rows, t, -1.0)
    return None, None, out
