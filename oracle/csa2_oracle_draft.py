"""CPU oracle of the drafted trees and of the caches in pages.

TEST INFRASTRUCTURE, like csa2_oracle.py: plain numpy and Python, the definitions written out one
node, one page and one entry at a time, no code shared with the CUDA sources.
"""
from __future__ import annotations

import numpy as np

from oracle import csa2_oracle as O


def tree_plan(parent, ctx_len: int):
    """(pos [T], path [T, T]) of one sequence's nodes."""
    T = len(parent)
    pos, path = np.full(T, -1, dtype=np.int64), np.full((T, T), -1, dtype=np.int16)
    for i in range(T):
        up, j = [], i
        while j >= 0:
            up.append(j)
            j = -2 if parent[j] >= j or ctx_len < 0 else int(parent[j])
        if j == -1:
            pos[i] = ctx_len + len(up) - 1
            path[i, :len(up)] = up[::-1]
    return pos, path


def tree_keys(entries, sel, swa, swa_pos0: int, draft, pos, path, ctx_len: int, i: int, window: int):
    """The rows node i attends to: entries[sel], its window's committed rows, its path's drafts."""
    c = entries.shape[-1] if entries is not None else draft.shape[-1]
    if pos[i] < 0:
        return np.zeros((0, c))
    rows = [entries[s] for s in sel if s >= 0]
    for p in range(max(0, int(pos[i]) - window + 1), int(pos[i]) + 1) if window > 0 else ():
        rows.append(swa[(p - swa_pos0) % swa.shape[0]] if p < ctx_len else draft[path[i, p - ctx_len]])
    return np.asarray(rows, dtype=np.float64).reshape(-1, c)


def tree_attn(q, entries, sel, swa, swa_pos0: int, draft, parent, ctx_len: int, sink, window: int,
              flags: int = O.QNORM | O.KVNORM | O.ROPE, base=O.ROPE_BASE):
    """One sequence: q [T, H, c], entries [N, c], sel: entry ids per node, swa [cap, c], draft [T, c],
    parent [T].  Returns (out [T, H, c], lse [T, H])."""
    T, H, c = q.shape
    pos, path = tree_plan(parent, ctx_len)
    out, lse = np.zeros((T, H, c)), np.full((T, H), -np.inf)
    for i in range(T):
        K = tree_keys(entries, sel[i], swa, swa_pos0, draft, pos, path, ctx_len, i, window)
        if K.shape[0] == 0:
            if sink is not None:
                lse[i] = sink
            continue
        out[i], lse[i] = O.attend(q[i], K, int(pos[i]), sink, flags, base)[:2]
    return out, lse


class Pages:
    """The state of a paged cache: refs [n_pages], table [B, P]; calls in the order of their effects."""

    def __init__(self, refs, table, page: int):
        self.refs, self.table, self.page = np.array(refs, dtype=np.int64), np.array(table, dtype=np.int64), page

    def fork(self, parent):
        out = np.array([self.table[p] if p >= 0 else np.full(self.table.shape[1], -1) for p in parent])
        for t in out.flatten():
            if t >= 0:
                self.refs[t] += 1
        return out.reshape(len(parent), self.table.shape[1])

    def free(self, keep=None):
        for b in range(self.table.shape[0]):
            k = 0 if keep is None else int(keep[b])
            for j in range(self.table.shape[1]):
                if k >= 0 and j * self.page >= k and self.table[b, j] >= 0:
                    self.refs[self.table[b, j]] -= 1
                    self.table[b, j] = -1

    def reserve(self, first, count):
        B, P = self.table.shape
        uses, free = self.refs.copy(), [p for p in range(len(self.refs)) if self.refs[p] == 0]
        granted, copies = np.zeros(B, dtype=np.int64), np.full((B, 2), -1, dtype=np.int64)
        for b in range(B):
            f, n = int(first[b]), int(count[b])
            if f < 0 or n <= 0:
                continue
            end, ok = min(f + n, P * self.page), True
            granted[b] = max(0, end - f)
            for j in range(f // self.page, -(-end // self.page) if end > f else 0):
                t = self.table[b, j]
                if t >= 0 and uses[t] == 1:
                    continue
                if not free:
                    granted[b] = min(granted[b], max(0, j * self.page - f))
                    continue
                new = free.pop(0)
                self.refs[new] = 1
                self.table[b, j] = new
                if t >= 0:
                    self.refs[t] -= 1
                    if j == f // self.page and f % self.page:
                        copies[b] = t, new
        return granted, copies

    def compact(self):
        n = len(self.refs)
        cut = int((self.refs > 0).sum())
        src = [p for p in range(cut, n) if self.refs[p] > 0]
        dst = [p for p in range(cut) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = np.vectorize(lambda t: to.get(t, t), otypes=[np.int64])(self.table)
        moves = np.full((n // 2, 2), -1, dtype=np.int64)
        for i, m in enumerate(to.items()):
            moves[i] = m
        return moves, cut

    def place(self, b: int, e: int):
        """(page, slot) of entry e of sequence b, or None."""
        j = e // self.page
        t = self.table[b, j] if 0 <= e and j < self.table.shape[1] else -1
        return None if t < 0 else (int(t), e % self.page)
