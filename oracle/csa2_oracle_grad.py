"""CPU oracle of the operators behind the attention's forward pass: the backward passes of
the attention and of the compressor, the accumulated attention weight, and the eviction.

TEST INFRASTRUCTURE, like csa2_oracle.py: plain numpy in float64, the definitions written
out, no code shared with the CUDA sources.  tests/test_oracle_grad.py holds the gradients to
central differences of the forward oracle.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import csa2_oracle as O


def rms_norm_bwd(x, g):
    """Gradient of x from that of x / sqrt(mean(x^2) + eps)."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(g, dtype=np.float64)
    s = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + O.RMS_EPS)
    return g / s - x * np.mean(x * g, axis=-1, keepdims=True) / s ** 3


def key_rows(n_entries: int, idx, swa_cap: int, swa_pos0: int, t: int, window: int):
    """The rows gather_keys takes, as ("kv", entry) / ("swa", slot), in its order."""
    rows = [("kv", int(s)) for s in np.asarray(idx) if 0 <= s < n_entries]
    for p in range(max(0, t - window + 1), t + 1) if window > 0 else ():
        rows.append(("swa", (p - swa_pos0) % swa_cap))
    return rows


def probabilities(q, keys, t: int, lse, flags, base=O.ROPE_BASE):
    """(q^ [H, c], k^ [nk, c], p [H, nk]) with p = exp(z - lse); an lse of -inf gives 0."""
    q, K = np.asarray(q, dtype=np.float64), np.asarray(keys, dtype=np.float64)
    c = q.shape[1]
    if flags & O.KVNORM and K.shape[0]:
        K = O.rms_norm(K)
    qh = O.rms_norm(q) if flags & O.QNORM else q
    if flags & O.ROPE:
        qh = O.rope(qh, t, base=base)
    lse = np.asarray(lse, dtype=np.float64)
    live = lse > O.NEG_INF
    p = np.zeros((q.shape[0], K.shape[0]))
    p[live] = np.exp(qh[live] @ K.T / math.sqrt(c) - lse[live, None])
    return qh, K, p


def attn_bwd(q, kv, sel, swa, swa_pos0: int, q_pos, sink, window: int, out, lse, dout,
             flags: int = O.QNORM | O.KVNORM | O.ROPE, base=O.ROPE_BASE):
    """Gradients of one sequence: q, out, dout [Q, H, c], kv [N, c], sel: per query the entry
    ids (-1 = none), swa [cap, c], q_pos [Q], sink [H] or None, lse [Q, H].  Returns
    (dq, dkv, dswa, dsink), and the root sums of squares of the terms that dq, dkv and dswa
    are sums of (what independent relative errors of the terms add up by)."""
    q, dout, out = (np.asarray(x, dtype=np.float64) for x in (q, dout, out))
    kv, swa = np.asarray(kv, dtype=np.float64), np.asarray(swa, dtype=np.float64)
    Q, H, c = q.shape
    dq = np.zeros_like(q)
    gk, gw = np.zeros_like(kv), np.zeros_like(swa)          # of the normalised rows
    dsink = np.zeros(H)
    tq, tk, tw = np.zeros_like(q), np.zeros_like(kv), np.zeros_like(swa)
    for i in range(Q):
        t = int(q_pos[i])
        rows = key_rows(kv.shape[0], sel[i], swa.shape[0], swa_pos0, t, window)
        keys = np.array([kv[j] if w == "kv" else swa[j] for w, j in rows]).reshape(len(rows), c)
        D = np.sum(dout[i] * out[i], axis=1)
        if sink is not None:
            live = np.asarray(lse[i]) > O.NEG_INF
            dsink[live] -= (np.exp(np.asarray(sink, dtype=np.float64) - lse[i]) * D)[live]
        if not rows:
            continue
        qh, K, p = probabilities(q[i], keys, t, lse[i], flags, base)
        do = O.rope(dout[i], t, base=base) if flags & O.ROPE else dout[i]
        dS = p * (do @ K.T - D[:, None]) / math.sqrt(c)
        g = dS @ K
        if flags & O.ROPE:
            g = O.rope(g, t, inverse=True, base=base)
        dq[i] = rms_norm_bwd(q[i], g) if flags & O.QNORM else g
        # dP is itself a sum whose rotated channels may be rounded: p times its root sum of squares
        # there counts with dS (dS is small where dP comes close to D, that rounding is not)
        d2 = dS ** 2 + p ** 2 * (do[:, -O.ROPE_DIMS:] ** 2 @ (K[:, -O.ROPE_DIMS:] ** 2).T) / c
        # (a norm's projection takes the same errors along its direction from every channel)
        along_q, along_do = (qh @ K.T / c) ** 2, (do @ K.T / c) ** 2
        # (and the rotation back mixes the two channels of a pair)
        tq[i] = d2 @ K ** 2
        if flags & O.ROPE:
            pair = tq[i][:, -O.ROPE_DIMS::2] + tq[i][:, -O.ROPE_DIMS + 1::2]
            tq[i][:, -O.ROPE_DIMS::2] = tq[i][:, -O.ROPE_DIMS + 1::2] = pair
        if flags & O.QNORM:
            tq[i] += O.rms_norm(q[i]) ** 2 * (d2 * along_q).sum(axis=1, keepdims=True)
            tq[i] /= np.mean(q[i] ** 2, axis=-1, keepdims=True) + O.RMS_EPS
        squares = d2.T @ qh ** 2 + (p ** 2).T @ do ** 2
        if flags & O.KVNORM:
            squares += K ** 2 * (d2 * along_q + p ** 2 * along_do).sum(axis=0)[:, None]
        for (w, j), r, r2 in zip(rows, dS.T @ qh + p.T @ do, squares):
            (gk if w == "kv" else gw)[j] += r
            (tk if w == "kv" else tw)[j] += r2
    tq, tk, tw = np.sqrt(tq), np.sqrt(tk), np.sqrt(tw)
    if flags & O.KVNORM:
        gk, gw = rms_norm_bwd(kv, gk), rms_norm_bwd(swa, gw)
        tk, tw = (t / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + O.RMS_EPS) for t, x in ((tk, kv), (tw, swa)))
    return (dq, gk, gw, dsink), (tq, tk, tw)


def attn_mass(q, kv, sel, q_pos, lse, flags: int = O.QNORM | O.KVNORM | O.ROPE, base=O.ROPE_BASE):
    """(weights [Q, k], mass [N]) of one sequence: the sum over heads of every slot's
    probability, and its sum per entry."""
    kv = np.asarray(kv, dtype=np.float64)
    sel = np.asarray(sel)
    weights, mass = np.zeros(sel.shape), np.zeros(kv.shape[0])
    for i in range(sel.shape[0]):
        at = np.flatnonzero((sel[i] >= 0) & (sel[i] < kv.shape[0]))
        if at.size:
            weights[i, at] = probabilities(q[i], kv[sel[i][at]], int(q_pos[i]), lse[i], flags, base)[2].sum(0)
            np.add.at(mass, sel[i][at], weights[i, at])
    return weights, mass


def evict_keep(acc, n: int, keep: int, recent: int):
    """Entries of one row that stay, ascending, -1 padded to keep."""
    n = int(n)
    if n <= keep:
        ids = list(range(max(n, 0)))
    else:
        old = n - recent

        def rank(e):
            a = float(acc[e])
            return (0, 0.0, e) if math.isnan(a) else (1, -a, e)

        ids = sorted(sorted(range(old), key=rank)[:keep - recent]) + list(range(old, n))
    return np.array(ids + [-1] * (keep - len(ids)), dtype=np.int32)


def compress_bwd(Ca, Za, m: int, dout, Ba=None, Cb=None, Zb=None, Bb=None, prev_Cb=None, prev_Zb=None,
                 flags: int = 0, pos0: int = 0, base=O.ROPE_BASE):
    """Gradients of one stream's compressor inputs from dout [n/m, c]: a dict with the keys
    Ca, Za, Ba and, overlapping, Cb, Zb, Bb, prev_Cb, prev_Zb (0 where there is no input)."""
    Ca, Za, dout = (np.asarray(x, dtype=np.float64) for x in (Ca, Za, dout))
    n, c = Ca.shape
    two = Cb is not None
    zero = np.zeros((m, c))
    g = {k: np.zeros_like(Ca) for k in ("Ca", "Za", "Cb", "Zb")}
    g.update({k: np.zeros((m, c)) for k in ("Ba", "Bb", "prev_Cb", "prev_Zb")})
    for i in range(n // m):
        cur = slice(m * i, m * (i + 1))
        value, logit = Ca[cur], Za[cur] + (zero if Ba is None else Ba)
        hist = None
        if two and i > 0:
            old = slice(m * (i - 1), m * i)
            hist = (np.asarray(Cb[old], dtype=np.float64), np.asarray(Zb[old], dtype=np.float64), g["Cb"][old], g["Zb"][old])
        elif two and prev_Cb is not None:
            hist = (np.asarray(prev_Cb, dtype=np.float64), np.asarray(prev_Zb, dtype=np.float64), g["prev_Cb"], g["prev_Zb"])
        if hist is not None:
            value = np.concatenate([value, hist[0]])
            logit = np.concatenate([logit, hist[1] + (zero if Bb is None else Bb)])
        s = np.exp(logit - logit.max(axis=0))
        s /= s.sum(axis=0)
        E = (s * value).sum(axis=0)
        dE = dout[i]
        if flags & O.ROPE_W:
            dE = O.rope(dE, pos0 + m * i, inverse=True, base=base)
        if flags & O.NORM_W:
            dE = rms_norm_bwd(E, dE)
        dC = s * dE
        dZ = dC * (value - E)
        g["Ca"][cur], g["Za"][cur] = dC[:m], dZ[:m]
        g["Ba"] += dZ[:m]
        if hist is not None:
            hist[2][:], hist[3][:] = dC[m:], dZ[m:]
            g["Bb"] += dZ[m:]
    return g
