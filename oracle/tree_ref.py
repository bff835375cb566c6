"""CPU oracle of the operators around a drafted token tree -- TEST INFRASTRUCTURE ONLY.

Plain definitions in float64 (numpy) and Python integers: masks and positions of
trees, attention under a mask over the chunk's own keys, shaped distributions
and draws, the confirmed branch, and the pages' bookkeeping.
"""
from __future__ import annotations

import numpy as np

from .dflash_ref import f64

PAGE = 128


def branch(parents, i: int) -> list[int]:
    """Node i and its ancestors, from the node up."""
    got = []
    while i >= 0:
        got.append(i)
        i = parents[i]
    return got


def sees(parents) -> np.ndarray:
    """[n, n]: whether j is i or an ancestor of it."""
    m = np.zeros((len(parents), len(parents)), dtype=bool)
    for i in range(len(parents)):
        m[i, branch(parents, i)] = True
    return m


def bits(m: np.ndarray, words: int) -> np.ndarray:
    """Rows of truth values as int32 words, bit j % 32 of word j / 32."""
    wide = np.zeros((m.shape[0], words * 32), dtype=np.uint32)
    wide[:, :m.shape[1]] = m[:, :words * 32]
    w = (wide.reshape(-1, words, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
    return w.view(np.int32)


def attention(q, k, v, ctx: int, mask, scale: float = 0.0):
    """Row i of q [n, Hq, Dh] over the keys below ctx and the keys ctx + j with
    mask[i, j], of k, v [Hkv, ctx + n, Dh]; zeros for a row that sees none.
    Returns (out, sum_s p_s |v_s|, the largest sum_d |q_d k_d| * scale), the last
    two for error bounds."""
    q, k, v = f64(q), f64(k), f64(v)
    n, hq, dh = q.shape
    grp = hq // k.shape[0]
    scale = scale or 1.0 / np.sqrt(dh)
    out, mass, big = np.zeros((n, hq, dh)), np.zeros((n, hq, dh)), np.zeros((n, hq))
    for i in range(n):
        own = ctx + np.nonzero(mask[i])[0]
        at = np.concatenate([np.arange(max(ctx, 0)), own[own >= 0]])
        if at.size == 0:
            continue
        for h in range(hq):
            kk, vv = k[h // grp][at], v[h // grp][at]
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h], mass[i, h] = p @ vv, p @ np.abs(vv)
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, mass, big


def shape(x, T=1.0, k=0, p=1.0, m=0.0) -> np.ndarray:
    """The shaped distribution of one row of logits (float64 [V]); largest: what
    +inf counts as is put in by the caller. None where nothing has weight."""
    x = np.where(np.isnan(x), -np.inf, x)
    if not (x > -np.inf).any() or not T >= 0:
        return None
    order = np.argsort(-x, kind="stable")
    if T == 0:
        T, k = 1.0, 1
    z = np.exp((x[order] - x[order[0]]) / T)
    z[x[order] == -np.inf] = 0.0
    n = len(x) if k < 1 else min(k, len(x))
    w = z[:n]
    before = np.cumsum(w) - w
    keep = before < p * w.sum() if p < 1 else np.ones(n, dtype=bool)
    if m > 0:
        keep &= x[order[:n]] >= x[order[0]] + T * np.log(min(m, 1.0))
    keep[0] = True
    out = np.zeros(len(x))
    out[order[:n][keep]] = w[keep]
    return out / out.sum()


def draw(probs, u: float) -> int:
    """The first v with probs_0 + .. + probs_v > u * sum."""
    c = np.cumsum(probs)
    return min(len(probs) - 1, int(np.searchsorted(c, u * c[-1], side="right")))


def verify_tree(tokens, parents, drawn, max_path: int):
    """(tau, committed, path, next_anchor) of one tree; no rows: (0, -1.., -1.., -1)."""
    n = len(tokens)
    if n == 0:
        return 0, [-1] * max_path, [-1] * max_path, -1
    path = [0]
    while len(path) < max_path:
        at = path[-1]
        nxt = [c for c in range(at + 1, n) if parents[c] == at and tokens[c] == drawn[at]]
        if not nxt:
            break
        path.append(nxt[0])
    last = drawn[path[-1]]
    com = [tokens[i] for i in path[1:]] + [last]
    return len(path), com + [-1] * (max_path - len(com)), path + [-1] * (max_path - len(path)), last


class Pages:
    """Table, counts and lengths, changed step by step in the order of sequences."""

    def __init__(self, table, refs, length=None):
        self.table, self.refs = [list(map(int, r)) for r in table], [int(x) for x in refs]
        self.length = None if length is None else [int(x) for x in length]
        self.copies = []           # (from page, to page, rows)
        self.full = False          # whether something did not fit

    def free(self):
        return next((i for i, c in enumerate(self.refs) if c <= 0), None)

    def drop(self, b, keep):
        for j in range(-(-max(keep, 0) // PAGE), len(self.table[b])):
            if 0 <= self.table[b][j] < len(self.refs):
                self.refs[self.table[b][j]] -= 1
            self.table[b][j] = -1

    def release(self, keep):
        for b, n in enumerate(keep):
            self.drop(b, n)

    def reserve(self, want):
        for b, n in enumerate(want):
            need = -(-max(n, 0) // PAGE)
            self.full |= need > len(self.table[b])
            for j in range(min(need, len(self.table[b]))):
                if not 0 <= self.table[b][j] < len(self.refs):
                    p = self.free()
                    if p is None:
                        self.full = True
                        continue
                    self.table[b][j] = p
                    self.refs[p] = 1

    def fork(self, src, dst):
        """Returns whether a pair was left out."""
        B, per = len(self.table), len(self.table[0])
        ok = [0 <= s < B and 0 <= d < B and d not in src and d not in dst[:i] and 0 <= self.length[s] <= per * PAGE
              for i, (s, d) in enumerate(zip(src, dst))]
        pairs = [(s, d) for s, d, good in zip(src, dst, ok) if good]
        for _, d in pairs:
            self.drop(d, 0)
        own = []
        for s, _ in pairs:
            n = self.length[s]
            whole = all(0 <= e < len(self.refs) for e in self.table[s][: -(-n // PAGE)])
            p = None
            if whole and n % PAGE:
                p = self.free()
                if p is not None:
                    self.refs[p] = 1
            own.append((whole and (n % PAGE == 0 or p is not None), p))
        for (s, d), (good, p) in zip(pairs, own):
            n = self.length[s]
            if not good:
                self.full, self.length[d] = True, 0
                continue
            for j in range(n // PAGE):
                self.table[d][j] = self.table[s][j]
                self.refs[self.table[s][j]] += 1
            if n % PAGE:
                self.table[d][n // PAGE] = p
                self.copies.append((self.table[s][n // PAGE], p, n % PAGE))
            self.length[d] = n
        return not all(ok)
