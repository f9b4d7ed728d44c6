"""CPU oracle of the operators around the verification attention: drafted
tokens accepted or rejected, cache compaction, shared pages, attention of a
batch that shares a prefix.

TEST INFRASTRUCTURE ONLY, under the rules of ``dustin_oracle``: plain and
sequential, float64, no code shared with the CUDA library.  Pinned by
``tests/test_serving_oracle.py`` (closed forms, enumeration, invariants).
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------- drafted tokens

def _mass(row: np.ndarray) -> np.ndarray:
    return np.where(np.isfinite(row) & (row > 0), row, 0.0)


def draw(mass: np.ndarray, u: float) -> int:
    """First j with C_j > u * C_last; -1 if there is no mass."""
    c = np.cumsum(mass)
    if not c[-1] > 0:
        return -1
    t = u * c[-1] if u > 0 else 0.0
    hit = np.nonzero((c > t) & (mass > 0))[0]
    return int(hit[0]) if len(hit) else int(np.nonzero(mass > 0)[0][-1])


def verify_tokens(p, q, draft, n_draft, u_accept, u_sample):
    """p [b][w][V]; q [b][w-1][V] or None; draft, u_accept [b][w-1]; n_draft
    [b] or None; u_sample [b].  Returns tokens [b][w] and n_accepted [b]."""
    b, w, vocab = p.shape
    tokens = np.full((b, w), -1, dtype=np.int32)
    accepted = np.zeros(b, dtype=np.int32)
    for i in range(b):
        g = w - 1 if n_draft is None else min(max(int(n_draft[i]), 0), w - 1)
        a = 0
        while a < g:
            x = int(draft[i, a])
            if not 0 <= x < vocab:
                break
            qx = 1.0 if q is None else _mass(q[i, a, x])
            if not u_accept[i, a] * qx < _mass(p[i, a, x]):
                break
            tokens[i, a] = x
            a += 1
        mass = _mass(p[i, a])
        if a < g:
            if q is None:
                rest = mass.copy()
                if 0 <= draft[i, a] < vocab:
                    rest[draft[i, a]] = 0.0
            else:
                rest = np.maximum(mass - _mass(q[i, a]), 0.0)
            if rest.sum() > 0:
                mass = rest
        tokens[i, a] = draw(mass, float(u_sample[i]))
        accepted[i] = a
    return tokens, accepted


# ------------------------------------------------------------ cache and pages

def compact(rows: np.ndarray, idx, k_len, out: np.ndarray) -> np.ndarray:
    """rows [b][h][n][d]; out [b][h][>= k][d] is filled and returned."""
    for i in range(idx.shape[0]):
        k = idx.shape[1] if k_len is None else min(max(int(k_len[i]), 0), idx.shape[1])
        taken = [rows[i, :, j].copy() if 0 <= j < rows.shape[2] else None
                 for j in idx[i, :k]]
        for at, row in enumerate(taken):
            if row is not None:
                out[i, :, at] = row
    return out


class PageBook:
    """Page table, lengths and counts as plain lists, one operation at a time."""

    def __init__(self, table, seq_len, refcount, page_size):
        self.table = [[int(x) for x in row] for row in table]
        self.seq_len = [int(x) for x in seq_len]
        self.refcount = [int(x) for x in refcount]
        self.page = page_size

    def pages(self, length):
        return -(-length // self.page)

    def fork(self, parents, children):
        done = set()
        skipped = []
        for f, (p, c) in enumerate(zip(parents, children)):
            n = len(self.table)
            if not (0 <= p < n and 0 <= c < n) or p == c or c in done or p in set(children) \
                    or self.seq_len[c] != 0:
                skipped.append(f)
                if 0 <= c < n:
                    done.add(c)
                continue
            done.add(c)
            for s in range(self.pages(self.seq_len[p])):
                self.table[c][s] = self.table[p][s]
                self.refcount[self.table[p][s]] += 1
            self.seq_len[c] = self.seq_len[p]
        return skipped

    def resize(self, seqs, new_len):
        """Returns copies [n][2] and the list entries left out for lack of
        pages."""
        cap = len(self.table[0]) * self.page
        valid = [0 <= s < len(self.table) and 0 <= m <= cap and s not in seqs[:i]
                 for i, (s, m) in enumerate(zip(seqs, new_len))]
        old = {s: self.seq_len[s] for s, ok in zip(seqs, valid) if ok}
        for s, m, ok in zip(seqs, new_len, valid):
            if ok and m < old[s]:
                for x in range(self.pages(m), self.pages(old[s])):
                    self.refcount[self.table[s][x]] -= 1
                    self.table[s][x] = -1
                self.seq_len[s] = m
        free = [p for p, c in enumerate(self.refcount) if c == 0]
        counts = list(self.refcount)           # as the releases left them
        copies, starved, taken = [], [], 0
        short = False
        for i, (s, m, ok) in enumerate(zip(seqs, new_len, valid)):
            copies.append([-1, -1])
            if not ok or m <= old[s]:
                continue
            had, have = self.pages(old[s]), self.pages(m)
            cow = old[s] % self.page > 0 and counts[self.table[s][had - 1]] > 1
            need = have - had + cow
            if need == 0:
                self.seq_len[s] = m
                continue
            short = short or taken + need > len(free)
            if short:
                starved.append(i)
                continue
            fresh = free[taken:taken + need]
            taken += need
            if cow:
                page = fresh.pop(0)
                copies[-1] = [self.table[s][had - 1], page]
                self.refcount[self.table[s][had - 1]] -= 1
                self.table[s][had - 1] = page
                self.refcount[page] = 1
            for x, page in zip(range(had, have), fresh):
                self.table[s][x] = page
                self.refcount[page] = 1
            self.seq_len[s] = m
        return copies, starved

    def consistent(self):
        """Counts equal the number of entries that name each page."""
        seen = [0] * len(self.refcount)
        for row, n in zip(self.table, self.seq_len):
            for page in row[:self.pages(n)]:
                seen[page] += 1
        return seen == self.refcount


# --------------------------------------------------------------- shared prefix

def prefix_attention(q, k_prefix, v_prefix, k_own, v_own, groups, scale,
                     prefix_len=None, own_len=None, k_win=None, v_win=None):
    """q [b][h_q][w][d]; prefix caches [groups][h_kv][n][d]; own caches
    [b][h_kv][n][d]; window [b][h_kv][w][d] (causal).  Each sequence's keys are
    laid end to end, then attention is its definition.  Returns o, lse."""
    b, hq, w, d = q.shape
    hkv, per = k_prefix.shape[1], b // groups
    o = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    for i in range(b):
        g = i // per
        n_p = k_prefix.shape[2] if prefix_len is None else min(max(int(prefix_len[g]), 0),
                                                               k_prefix.shape[2])
        n_o = k_own.shape[2] if own_len is None else min(max(int(own_len[i]), 0),
                                                         k_own.shape[2])
        for h in range(hq):
            kv = h // (hq // hkv)
            k = [k_prefix[g, kv, :n_p], k_own[i, kv, :n_o]]
            v = [v_prefix[g, kv, :n_p], v_own[i, kv, :n_o]]
            for t in range(w):
                kk = k + ([k_win[i, kv, :t + 1]] if k_win is not None else [])
                vv = v + ([v_win[i, kv, :t + 1]] if v_win is not None else [])
                kk, vv = np.concatenate(kk), np.concatenate(vv)
                if not len(kk):
                    continue
                s = scale * (kk @ q[i, h, t])
                m = s.max()
                e = np.exp(s - m)
                o[i, h, t] = e @ vv / e.sum()
                lse[i, h, t] = m + np.log(e.sum())
    return o, lse
