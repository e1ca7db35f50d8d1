"""Cases of the operators that stand behind the attention's forward pass: its backward pass
(sparse and dense form), the accumulated attention weight of the cache entries with the
eviction that goes by it, and the compressor's backward pass.

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
        # gradient check of one small fp32 layer (four decode queries, 2,048 entries)
        dict(name="attn_bwd f32 tiny layer", op="attn_bwd", dtype="f32", form="sparse", B=1, Q=4, H=16, N=2048, k=512,
             window=128, m=2, t0=4092),
        # a short fine-tuning sequence pair with odd sizes
        dict(name="attn_bwd bf16 2x96 odd", op="attn_bwd", dtype="bf16", form="sparse", B=2, Q=96, H=40, N=997, k=301,
             window=100, m=4, t0=3897),
        # a training chunk over a 128K-token context
        dict(name="attn_bwd bf16 1x2048", op="attn_bwd", dtype="bf16", form="sparse", B=1, Q=2048, H=64, N=33280,
             k=512, window=128, m=4, t0=131072),
        # the prefill chunk's own size: 8,192 queries, 34,816 entries
        dict(name="attn_bwd bf16 1x8192", op="attn_bwd", dtype="bf16", form="sparse", B=1, Q=8192, H=64, N=34816,
             k=512, window=128, m=4, t0=131072),
        # the wide configuration: 128 heads, top-1024
        dict(name="attn_bwd bf16 h128 top1024", op="attn_bwd", dtype="bf16", form="sparse", B=1, Q=333, H=128, N=16384,
             k=1024, window=128, m=4, t0=65203),
        # dense attention over the heavily compressed cache (128 tokens an entry)
        dict(name="attn_bwd bf16 dense", op="attn_bwd", dtype="bf16", form="dense", B=1, Q=1000, H=64, N=1032, k=1032,
             window=128, m=128, t0=131072),
        # accounting after a decode step: 8 sequences of 1M FP4 entries
        dict(name="mass fp4 decode 8x1M", op="mass", dtype="fp4", form="sparse", B=8, Q=1, H=64, N=1 << 20, k=512, m=1,
             t0=(1 << 20) - 1),
        # accounting over a prefill chunk
        dict(name="mass bf16 prefill 4096", op="mass", dtype="bf16", form="sparse", B=1, Q=4096, H=64, N=33792, k=512,
             m=4, t0=131072),
        # a batch of middling caches of different lengths, bf16 rows
        dict(name="evict bf16 32x9001 ragged", op="evict", dtype="bf16", B=32, N=9001, keep=4001, recent=128, ragged=True),
        # eight 1M-entry FP4 caches cut to half
        dict(name="evict fp4 8x1M", op="evict", dtype="fp4", B=8, N=1 << 20, keep=1 << 19, recent=4096, ragged=False),
        # the prefill chunk's overlapped compressor
        dict(name="compress_bwd bf16 8192 overlap", op="compress_bwd", dtype="bf16", B=1, n=8192, m=4, overlap=True,
             norm=True, rope=True, bias=True),
        # the encoder's non-overlapping compressor over four long sequences
        dict(name="compress_bwd bf16 4x131072", op="compress_bwd", dtype="bf16", B=4, n=131072, m=2, overlap=False,
             norm=True, rope=True, bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_bwd", "attn_bwd", "attn_bwd", "mass", "mass", "evict", "evict", "compress_bwd"])
    if op in ("attn_bwd", "mass"):
        form = rng.choice(["sparse", "sparse", "dense"])
        dtype = rng.choice(["bf16", "bf16", "f32"] if op == "attn_bwd" else ["bf16", "fp4", "fp4", "f32"])
        H = rng.choice([16, 40, 64, 64, 100, 128])
        window = rng.choice([0, 1, 100, 128, 128, 200]) if op == "attn_bwd" else 0
        B = rng.randint(1, 4)
        k = _log(rng, 5, 1024)
        m = 128 if form == "dense" else rng.choice([1, 2, 4])
        # queries: at most a quarter of the largest case's products (an eighth of that in fp32)
        budget = 8192 * 64 * 640 // (32 if dtype == "f32" else 4)
        Q = max(1, min(_log(rng, 1, 4096), budget // (B * H * (k + window + 1))))
        N = k if form == "dense" else k + _log(rng, 1, 40000)
        if dtype == "fp4":
            N = min(N * 8, 1 << 18) if form == "sparse" else N
        t0 = max(0, N * m - rng.choice([0, 0, Q // 2, Q]))
        c = dict(op=op, dtype=dtype, form=form, B=B, Q=Q, H=H, N=N, k=k, m=m, t0=t0)
        if op == "attn_bwd":
            c["window"] = window
        return c
    if op == "evict":
        dtype = rng.choice(["bf16", "fp4"])
        N = _log(rng, 17, 1 << 20 if dtype == "fp4" else 1 << 17)
        B = max(1, min(_log(rng, 1, 64), (1 << 23 if dtype == "fp4" else 1 << 20) // N))
        keep = max(1, int(N * rng.uniform(0.05, 1.0)))
        return dict(op=op, dtype=dtype, B=B, N=N, keep=keep, recent=rng.randint(0, min(keep, 4096)),
                    ragged=rng.random() < 0.6)
    m = rng.choice([1, 2, 3, 4, 8, 128])
    n = max(1, _log(rng, 16, 131072) // m) * m
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=rng.randint(1, 3), n=n, m=m,
                overlap=m <= 8 and rng.random() < 0.5, norm=rng.random() < 0.7, rope=rng.random() < 0.7,
                bias=rng.random() < 0.5)


# ------------------------------------------------------------------ pieces of the plain forms (32 bits)
def _rope(x, pos, sign, c0):
    """Rotates the last 64 of c0 channels of x [..., c0] by sign * pos (pos broadcasts over
    x's leading axes); angles in 64 bits."""
    j = torch.arange(32, dtype=torch.float64, device=x.device)
    turns = pos.double().unsqueeze(-1) * (10000.0 ** (-2.0 * j / 64.0) / (2.0 * math.pi))
    ang = (turns - turns.floor()) * (2.0 * math.pi)
    cs, sn = ang.cos().to(x.dtype), (sign * ang.sin()).to(x.dtype)
    a, b = x[..., c0 - 64::2], x[..., c0 - 63::2]
    return torch.cat([x[..., :c0 - 64], torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)], -1)


def _rms_factor(x):
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _fp4_values(rows, dtype):
    """Values of FP4 rows [..., 288] (256 code bytes, low nibble first, 32 E4M3 scales)."""
    table = torch.tensor(_E2M1, dtype=dtype, device=rows.device)
    b = rows[..., :256].long()
    v = torch.stack([table[b & 15], table[b >> 4]], -1).flatten(-2)
    s = rows[..., 256:].contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (v.unflatten(-1, (32, 16)) * s.unsqueeze(-1)).flatten(-2)


def _rows_of(cache, b, ids, dtype):
    """cache[b, ids] as values: cache [B, N, 512] or FP4 rows, ids [B, Q, S] (clamped)."""
    r = cache[b, ids]
    return _fp4_values(r, dtype) if cache.dtype == torch.uint8 else r.to(dtype)


def _slots(s):
    """Entry id and validity of every cache slot of every query, [B, Q, k]."""
    if s["idx"] is not None:
        return s["idx"].long().clamp(min=0), s["idx"] >= 0
    ids = torch.arange(s["k"], device=DEV).expand(*s["q_pos"].shape, s["k"])
    return ids, ids < s["n_visible"].unsqueeze(-1)


def _window(s):
    """Window slot and validity of every query's window, [B, Q, window]."""
    p = s["q_pos"].unsqueeze(-1) - s["window"] + 1 + torch.arange(s["window"], device=DEV)
    return (p - s["swa_pos0"]) % s["swa"].shape[1], p >= 0


def _queries(s, dtype):
    q = s["q"].to(dtype)
    rq = _rms_factor(q)
    qn = q * rq
    return rq, qn, _rope(qn, s["q_pos"].unsqueeze(-1), 1.0, C)


def _forward(s):
    """out and lse of the attention, as the training step's forward pass leaves them."""
    rows, ok = _attended(s)
    khat = rows * _rms_factor(rows)
    z = (_queries(s, torch.float32)[2] @ khat.transpose(-1, -2)) / math.sqrt(C)
    z.masked_fill_(~ok.unsqueeze(-2), -math.inf)
    if s["sink"] is not None:
        z = torch.cat([z, s["sink"].view(1, 1, -1, 1).expand(*z.shape[:3], 1)], -1)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z[..., :rows.shape[-2]] - lse.unsqueeze(-1))
    o = _rope(p @ khat, s["q_pos"].unsqueeze(-1), -1.0, C)
    return o.to(s["q"].dtype), lse


def _attended(s):
    b = torch.arange(s["q"].shape[0], device=DEV).view(-1, 1, 1)
    ids, ok = _slots(s)
    rows = _rows_of(s["kv"], b, ids, torch.float32)
    if s["window"]:
        slot, okw = _window(s)
        rows = torch.cat([rows, s["swa"][b, slot].float()], -2)
        ok = torch.cat([ok, okw], -1)
    return rows, ok


def _row_grad(grad, stored):
    """Gradient of stored rows from that of their normalised form."""
    x = stored.float()
    r = _rms_factor(x)
    xh = x * r
    return (r * (grad - xh * (xh * grad).mean(-1, keepdim=True))).to(stored.dtype)


def _attn_bwd(s):
    B, Q, H, _ = s["q"].shape
    rq, qn, qh = _queries(s, torch.float32)
    rows, ok = _attended(s)
    khat = rows * _rms_factor(rows)
    kt = khat.transpose(-1, -2)
    p = torch.exp((qh @ kt) / math.sqrt(C) - s["lse"].unsqueeze(-1)).masked_fill(~ok.unsqueeze(-2), 0.0)
    dout = s["dout"].float()
    D = (dout * s["out"].float()).sum(-1)
    do = _rope(dout, s["q_pos"].unsqueeze(-1), 1.0, C)
    ds = p * (do @ kt - D.unsqueeze(-1)) / math.sqrt(C)
    dqn = _rope(ds @ khat, s["q_pos"].unsqueeze(-1), -1.0, C)
    dq = (rq * (dqn - qn * (qn * dqn).mean(-1, keepdim=True))).to(s["q"].dtype)
    dk = ds.transpose(-1, -2) @ qh + p.transpose(-1, -2) @ do
    off = torch.arange(B, device=DEV).view(-1, 1, 1)
    k, N, cap = s["k"], s["kv"].shape[1], s["swa"].shape[1]
    g = torch.zeros(B * N, C, device=DEV)
    g.index_add_(0, (_slots(s)[0] + off * N).flatten(), dk[..., :k, :].reshape(-1, C))
    dkv = _row_grad(g.view(B, N, C), s["kv"])
    g = torch.zeros(B * cap, C, device=DEV)
    if s["window"]:
        g.index_add_(0, (_window(s)[0] + off * cap).flatten(), dk[..., k:, :].reshape(-1, C))
    dswa = _row_grad(g.view(B, cap, C), s["swa"])
    dsink = -(torch.exp(s["sink"] - s["lse"]) * D).sum((0, 1))
    return dq, dkv, dswa, dsink


def _mass(s):
    B, Q, H, _ = s["q"].shape
    rows, ok = _attended(s)
    khat = rows * _rms_factor(rows)
    z = (_queries(s, torch.float32)[2] @ khat.transpose(-1, -2)) / math.sqrt(C)
    w = torch.exp(z - s["lse"].unsqueeze(-1)).sum(2).masked_fill(~ok, 0.0)
    N = s["kv"].shape[1]
    at = _slots(s)[0] + torch.arange(B, device=DEV).view(-1, 1, 1) * N
    s["acc"].view(-1).index_add_(0, at.flatten(), w.flatten())
    return w, s["acc"]


def _evict(s):
    B, N = s["acc"].shape
    e = torch.arange(N, device=DEV)
    n = s["n_entries"].unsqueeze(-1)
    rank = s["acc"].masked_fill(e >= n - s["recent"], math.inf).masked_fill(e >= n, -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :s["keep"]]
    kept = best.masked_fill(best >= n, N).sort(-1).values
    full = kept < N
    idx = kept.masked_fill(~full, -1).to(torch.int32)
    at = kept.clamp(max=N - 1)
    b = torch.arange(B, device=DEV).unsqueeze(-1)
    for src, dst in (("kv", "kv_dst"), ("ki", "ki_dst"), ("acc", "acc_dst")):
        mask = full if s[src].dim() == 2 else full.unsqueeze(-1)
        s[dst].copy_(torch.where(mask, s[src][b, at], s[dst]))
    return idx, s["kv_dst"], s["ki_dst"], s["acc_dst"]


def _compress_rows(s, name):
    return s[name].float().unflatten(1, (-1, s["m"])) if s[name] is not None else None


def _compress_bwd(s):
    m, c = s["m"], C
    val, gate = _compress_rows(s, "ca"), _compress_rows(s, "za")
    if s["ba"] is not None:
        gate = gate + s["ba"]
    if s["cb"] is not None:
        vb, gb = _compress_rows(s, "cb"), _compress_rows(s, "zb")
        vb = torch.cat([s["prev_cb"].float().unsqueeze(1), vb[:, :-1]], 1)
        gb = torch.cat([s["prev_zb"].float().unsqueeze(1), gb[:, :-1]], 1)
        if s["bb"] is not None:
            gb = gb + s["bb"]
        val, gate = torch.cat([val, vb], 2), torch.cat([gate, gb], 2)
    w = torch.exp(gate - gate.amax(2, keepdim=True))
    w = w / w.sum(2, keepdim=True)
    e = (w * val).sum(2)
    g = s["dout"].float()
    if s["rope"]:
        pos = s["pos0"].unsqueeze(-1) + m * torch.arange(e.shape[1], device=DEV)
        g = _rope(g, pos, -1.0, c)
    if s["norm"]:
        r = _rms_factor(e)
        eh = e * r
        g = r * (g - eh * (eh * g).mean(-1, keepdim=True))
    dval = w * g.unsqueeze(2)
    dgate = dval * (val - e.unsqueeze(2))
    dt = s["ca"].dtype
    outs = [dval[:, :, :m].flatten(1, 2).to(dt), dgate[:, :, :m].flatten(1, 2).to(dt)]
    if s["cb"] is not None:
        last = torch.zeros_like(dval[:, :1, m:])
        for x in (dval, dgate):
            outs.append(torch.cat([x[:, 1:, m:], last], 1).flatten(1, 2).to(dt))
        outs += [dval[:, 0, m:].to(dt), dgate[:, 0, m:].to(dt)]
    if s["ba"] is not None:
        outs.append(dgate[:, :, :m].sum((0, 1)))
        if s["cb"] is not None:
            outs.append(dgate[:, :, m:].sum((0, 1)))
    return outs


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from compressed_sparse_attention_06_gb300 import csa2

    op = s["op"]
    if op == "attn_bwd":
        kw = dict(window=s["window"], swa_pos0=s["swa_pos0"])
        if s["idx"] is not None:
            return csa2.csa2_sparse_attn_bwd(s["q"], s["kv"], s["idx"], s["swa"], s["q_pos"], s["sink"], s["out"],
                                             s["lse"], s["dout"], **kw)
        return csa2.csa2_dense_attn_bwd(s["q"], s["kv"], s["n_visible"], s["k"], s["swa"], s["q_pos"], s["sink"],
                                        s["out"], s["lse"], s["dout"], **kw)
    if op == "mass":
        return csa2.csa2_attn_mass(s["q"], s["kv"], s["q_pos"], s["lse"], idx=s["idx"], n_visible=s["n_visible"],
                                   k_max=s["k"], acc=s["acc"], want_weights=True)
    if op == "evict":
        idx = csa2.csa2_evict_select(s["acc"], s["n_entries"], s["keep"], recent=s["recent"])
        return (idx, csa2.csa2_cache_gather(s["kv"], idx, out=s["kv_dst"]),
                csa2.csa2_cache_gather(s["ki"], idx, out=s["ki_dst"]),
                csa2.csa2_cache_gather(s["acc"], idx, out=s["acc_dst"]))
    flags = (csa2.W_NORM if s["norm"] else 0) | (csa2.W_ROPE if s["rope"] else 0)
    g = csa2.csa2_compress_bwd(s["ca"], s["za"], s["m"], s["dout"], cb=s["cb"], zb=s["zb"], ba=s["ba"], bb=s["bb"],
                               prev_cb=s["prev_cb"], prev_zb=s["prev_zb"], pos0=s["pos0"], flags=flags)
    return [x for x in (g.dca, g.dza, g.dcb, g.dzb, g.dprev_cb, g.dprev_zb, g.dba, g.dbb) if x is not None]


def run(state):
    if own:
        return _own(state)
    return {"attn_bwd": _attn_bwd, "mass": _mass, "evict": _evict, "compress_bwd": _compress_bwd}[state["op"]](state)


# ------------------------------------------------------------------ inputs
def _fp4_pool(gen, rows):
    """FP4 rows of normal values with a log-normal size per row."""
    x = torch.randn(rows, C, generator=gen, device=DEV)
    x = x * torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=DEV))
    g = x.view(rows, 32, 16)
    s = (g.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = (g / s.float().clamp(min=2.0 ** -9).unsqueeze(-1)).view(rows, C)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(y.abs(), edges) + 8 * (y < 0)
    return torch.cat([(code[:, ::2] + 16 * code[:, 1::2]).to(torch.uint8), s.view(torch.uint8)], 1)


def _cache(gen, dtype, B, N):
    if dtype == "fp4":
        pool = _fp4_pool(gen, min(B * N, 1 << 16))
        if B * N <= 1 << 16:
            return pool.view(B, N, -1)
        return pool[torch.randint(0, 1 << 16, (B, N), generator=gen, device=DEV)]
    return torch.randn(B, N, C, generator=gen, device=DEV).to(torch.float32 if dtype == "f32" else torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    op, B = case["op"], case["B"]
    s = dict(op=op)
    if op == "evict":
        N = case["N"]
        s.update(keep=case["keep"], recent=case["recent"], kv=_cache(gen, case["dtype"], B, N))
        if case["dtype"] == "fp4":
            s["ki"] = torch.randint(0, 256, (B, N, 68), generator=gen, device=DEV, dtype=torch.uint8)
        else:
            s["ki"] = normal(B, N, 128, dtype=torch.bfloat16)
        # weights as a long decode leaves them: a few heavy entries, many that were never picked (ties at 0)
        u = torch.rand(B, N, generator=gen, device=DEV)
        s["acc"] = torch.where(u < 0.35, torch.zeros_like(u), torch.exp(2.0 * normal(B, N)) * u ** 4)
        n = torch.full((B,), N, dtype=torch.int64, device=DEV)
        if case["ragged"]:
            n = torch.randint(0, N + 1, (B,), generator=gen, device=DEV)
        s["n_entries"] = n
        for name in ("kv", "ki", "acc"):
            s[name + "_dst"] = torch.zeros(B, case["keep"], *s[name].shape[2:], dtype=s[name].dtype, device=DEV)
        return s
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    if op == "compress_bwd":
        n, m = case["n"], case["m"]
        two = case["overlap"]
        s.update(m=m, norm=case["norm"], rope=case["rope"])
        s["ca"], s["za"] = normal(B, n, C, dtype=dt), normal(B, n, C, dtype=dt)
        s["cb"], s["zb"] = (normal(B, n, C, dtype=dt), normal(B, n, C, dtype=dt)) if two else (None, None)
        s["prev_cb"], s["prev_zb"] = (normal(B, m, C, dtype=dt), normal(B, m, C, dtype=dt)) if two else (None, None)
        s["ba"] = 0.1 * normal(m, C) if case["bias"] else None
        s["bb"] = 0.1 * normal(m, C) if case["bias"] and two else None
        s["pos0"] = torch.randint(0, 1 << 17, (B,), generator=gen, device=DEV) // m * m
        s["dout"] = normal(B, n // m, C, dtype=dt)
        return s
    Q, H, N, k, m = case["Q"], case["H"], case["N"], case["k"], case["m"]
    s.update(k=k, window=case.get("window", 0), swa_pos0=0)
    s["q"] = normal(B, Q, H, C, dtype=dt)
    s["kv"] = _cache(gen, case["dtype"], B, N)
    s["q_pos"] = (case["t0"] + torch.arange(Q, device=DEV)).expand(B, Q).contiguous()
    seen = (s["q_pos"] // m).clamp(max=N)                      # entries a query sees
    if case["form"] == "dense":
        s["idx"], s["n_visible"] = None, seen
    else:
        # a selection as an indexer makes it: distinct ascending entries, neighbours in time
        # sharing much of theirs, all visible entries where there are no more than k
        s["n_visible"] = None
        base = torch.rand(B, (Q + 15) // 16, k, generator=gen, device=DEV).repeat_interleave(16, 1)[:, :Q]
        own_u = torch.rand(B, Q, k, generator=gen, device=DEV)
        u = torch.where(torch.rand(B, Q, k, generator=gen, device=DEV) < 0.6, base, own_u).double()
        j = torch.arange(k, device=DEV, dtype=torch.float64)
        v = seen.unsqueeze(-1)
        lo, hi = torch.floor(j * v / k), torch.floor((j + 1) * v / k)
        ids = torch.minimum(lo + torch.floor(u * (hi - lo)), hi - 1)
        ids = torch.where(v <= k, torch.where(j < v, j.expand_as(ids), -torch.ones_like(ids)), ids)
        s["idx"] = ids.to(torch.int32)
    if op == "mass":
        s["sink"] = None
        s["lse"] = _forward(s)[1]
        s["acc"] = torch.rand(B, N, generator=gen, device=DEV)
        return s
    s["swa_pos0"] = max(0, case["t0"] - s["window"] + 1)
    s["swa"] = normal(B, max(1, case["t0"] + Q - s["swa_pos0"]), C, dtype=dt)
    s["sink"] = normal(H)
    s["out"], s["lse"] = _forward(s)
    s["dout"] = normal(B, Q, H, C, dtype=dt)
    return s


# ------------------------------------------------------------------ work and the 64-bit answers
def work(case):
    op, B = case["op"], case["B"]
    e = 4 if case["dtype"] == "f32" else 2
    row = 288 if case["dtype"] == "fp4" else C * e
    if op in ("attn_bwd", "mass"):
        Q, H, N, k, w = case["Q"], case["H"], case["N"], case["k"], case.get("window", 0)
        heads = B * Q * H * C * e
        picked = min(B * N, B * Q * k) * row
        ids = B * Q * k * 4 if case["form"] == "sparse" else B * Q * 8
        pairs = B * Q * H * (k + w)
        if op == "mass":
            return {"bytes": heads + picked + ids + B * Q * (H * 4 + 8 + k * 4) + min(B * N, B * Q * k) * 8,
                    "flops": 2 * pairs * C}
        swa = B * (case["t0"] + Q - max(0, case["t0"] - w + 1)) * C * e
        return {"bytes": 4 * heads + picked + B * N * row + 2 * swa + ids + B * Q * (H * 4 + 8) + 8 * H,
                "flops": 10 * pairs * C}
    if op == "evict":
        N, keep = case["N"], case["keep"]
        rows = row + (68 if case["dtype"] == "fp4" else 256) + 4
        return {"bytes": B * (N * 4 + keep * 4 + 2 * keep * rows), "flops": 0}
    n, m = case["n"], case["m"]
    tensors = 4 if case["overlap"] else 2
    extra = tensors * m * C * e * B if case["overlap"] else 0
    return {"bytes": B * n * C * e * 2 * tensors + B * (n // m) * C * e + extra, "flops": B * n * C * 5 * tensors}


def _spin(x, pos, sign):
    """x with its last 64 channels as 32 complex numbers turned by sign * pos * base^(-j/32)."""
    j = torch.arange(32, dtype=torch.float64, device=x.device)
    ang = sign * pos.double().unsqueeze(-1) * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device), -j / 32)
    z = torch.view_as_complex(x[..., -64:].contiguous().unflatten(-1, (32, 2))) * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([x[..., :-64], torch.view_as_real(z).flatten(-2)], -1)


def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _unit_grad(x, g):
    """Gradient through _unit, by the quotient rule on the norm."""
    n2 = x.square().mean(-1, keepdim=True) + EPS
    return g * n2.rsqrt() - x * (x * g).mean(-1, keepdim=True) * n2.pow(-1.5)


def _exact_attention(s, grads):
    """One sequence at a time, its queries in blocks; definition sums in 64 bits."""
    B, Q, H, _ = s["q"].shape
    N, k, W = s["kv"].shape[1], s["k"], s["window"]
    f64 = torch.float64
    step = max(1, (1 << 27) // ((k + W) * C))
    if grads:
        cap = s["swa"].shape[1]
        dq = torch.empty(B, Q, H, C, dtype=f64, device=DEV)
        dkh, dwh = torch.zeros(B, N, C, dtype=f64, device=DEV), torch.zeros(B, cap, C, dtype=f64, device=DEV)
        dsink = torch.zeros(H, dtype=f64, device=DEV)
    else:
        weights = torch.zeros(B, Q, k, dtype=f64, device=DEV)
        acc = s["acc"].double()
    for b in range(B):
        for q0 in range(0, Q, step):
            sl = slice(q0, min(Q, q0 + step))
            t = s["q_pos"][b, sl]
            if s["idx"] is not None:
                ids = s["idx"][b, sl].long()
            else:
                ids = torch.arange(k, device=DEV).repeat(t.numel(), 1)
                ids[ids >= s["n_visible"][b, sl, None]] = -1
            real = ids >= 0
            x = s["kv"][b][ids.clamp(min=0)]
            x = _fp4_values(x, f64) if x.dtype == torch.uint8 else x.double()
            if W:
                p = t[:, None] + torch.arange(1 - W, 1, device=DEV)
                ws = torch.remainder(p - s["swa_pos0"], s["swa"].shape[1])
                x = torch.cat([x, s["swa"][b][ws].double()], 1)
                real = torch.cat([real, p >= 0], 1)
            kh = _unit(x)
            qraw = s["q"][b, sl].double()
            qh = _spin(_unit(qraw), t[:, None], 1.0)
            prob = torch.exp(torch.einsum("qhc,qsc->qhs", qh, kh) / C ** 0.5 - s["lse"][b, sl].double()[..., None])
            prob = prob * real[:, None, :]
            if not grads:
                wgt = prob.sum(1)
                weights[b, sl] = wgt
                acc[b].index_put_((ids.clamp(min=0).flatten(),), wgt.flatten(), accumulate=True)
                continue
            go = s["dout"][b, sl].double()
            D = torch.einsum("qhc,qhc->qh", go, s["out"][b, sl].double())
            gh = _spin(go, t[:, None], 1.0)
            score = prob * (torch.einsum("qhc,qsc->qhs", gh, kh) - D[..., None]) / C ** 0.5
            dq[b, sl] = _unit_grad(qraw, _spin(torch.einsum("qhs,qsc->qhc", score, kh), t[:, None], -1.0))
            rows = torch.einsum("qhs,qhc->qsc", score, qh) + torch.einsum("qhs,qhc->qsc", prob, gh)
            dkh[b].index_put_((ids.clamp(min=0).flatten(),), rows[:, :k].reshape(-1, C), accumulate=True)
            if W:
                dwh[b].index_put_((ws.flatten(),), rows[:, k:].reshape(-1, C), accumulate=True)
            dsink -= (torch.exp(s["sink"].double() - s["lse"][b, sl].double()) * D).sum(0)
    if not grads:
        return weights, acc
    return dq, _unit_grad(s["kv"].double(), dkh), _unit_grad(s["swa"].double(), dwh), dsink


def _exact_evict(s):
    kept = torch.zeros(s["acc"].shape[0], s["keep"], dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["n_entries"].tolist()):
        a = s["acc"][b, :n].double()
        lo = max(0, n - s["recent"])
        take = min(s["keep"], n) - (n - lo)
        order = torch.sort(-a[:lo], stable=True).indices[:max(0, take)]
        ids = torch.cat([order.sort().values, torch.arange(lo, n, device=DEV)])
        kept[b, :ids.numel()] = a[ids]
    return None, None, None, kept


def _exact_compress(s):
    """The forward definition in 64 bits, differentiated by torch."""
    names = [x for x in ("ca", "za", "cb", "zb", "prev_cb", "prev_zb", "ba", "bb") if s[x] is not None]
    v = {x: s[x].double().requires_grad_() for x in names}
    m, n = s["m"], s["ca"].shape[1]
    total = 0.0
    for b in range(s["ca"].shape[0]):
        value, logit = v["ca"][b].view(n // m, m, C), v["za"][b].view(n // m, m, C)
        logit = logit + v["ba"] if "ba" in v else logit
        if "cb" in v:
            pv = torch.cat([v["prev_cb"][b], v["cb"][b]])[:n].view(n // m, m, C)
            pl = torch.cat([v["prev_zb"][b], v["zb"][b]])[:n].view(n // m, m, C)
            pl = pl + v["bb"] if "bb" in v else pl
            value, logit = torch.cat([value, pv], 1), torch.cat([logit, pl], 1)
        y = (torch.softmax(logit, 1) * value).sum(1)
        y = _unit(y) if s["norm"] else y
        if s["rope"]:
            y = _spin(y, s["pos0"][b] + m * torch.arange(n // m, device=DEV), 1.0)
        total = total + (y * s["dout"][b].double()).sum()
    return list(torch.autograd.grad(total, [v[x] for x in names]))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("attn_bwd", "mass"):
        return _exact_attention(s, s["op"] == "attn_bwd")
    return _exact_evict(s) if s["op"] == "evict" else _exact_compress(s)
