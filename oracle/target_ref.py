"""CPU oracle of the target-side operators -- TEST INFRASTRUCTURE ONLY.

Plain definitions in float64 (numpy): per-head norms with rotary positions,
causal attention of a chunk behind a cached context, and verification of
drafts against given probabilities from given random numbers.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .dflash_ref import f64, rms_norm, rope


def qk_norm_rope(x, gain, pos, eps: float, theta: float) -> np.ndarray:
    """R_p(gain * x / sqrt(mean x^2 + eps)) of x [T, H, Dh]; gain None: no norm."""
    y = f64(x)
    if gain is not None:
        y = rms_norm(y, f64(gain), eps)
    return rope(y, np.asarray(pos), theta)


def chunk_attention(q, k, v, ctx: int, causal: bool = True, scale: float = 0.0):
    """Row i of q [n, Hq, Dh] over keys 0 .. ctx + i (causal) or all of
    k, v [Hkv, ctx + n, Dh]; a row that sees no key gives zeros. Returns
    (out [n, Hq, Dh], sum_s p_s |v_s| of the same shape, the largest
    sum_d |q_d k_d| * scale of a row [n, Hq]) -- the last two for error bounds."""
    q, k, v = f64(q), f64(k), f64(v)
    n, hq, dh = q.shape
    grp = hq // k.shape[0]
    scale = scale or 1.0 / np.sqrt(dh)
    out, mass, big = np.zeros((n, hq, dh)), np.zeros((n, hq, dh)), np.zeros((n, hq))
    for i in range(n):
        seen = min(max(ctx + i + 1, 0) if causal else max(ctx + n, 0), k.shape[1])
        if seen == 0:
            continue
        for h in range(hq):
            g = h // grp
            s = k[g, :seen] @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ v[g, :seen]
            mass[i, h] = p @ np.abs(v[g, :seen])
            big[i, h] = (np.abs(k[g, :seen]) @ np.abs(q[i, h])).max() * scale
    return out, mass, big


def probability(p) -> np.ndarray:
    """Entries as probabilities: NaN and negative ones are 0, larger ones 1."""
    x = f64(p)
    return np.where(np.isnan(x), 0.0, np.clip(x, 0.0, 1.0))


def fixed62(p) -> np.ndarray:
    """Probabilities as whole multiples of 2^-62 (uint64), truncated."""
    return np.floor(probability(p) * 2.0 ** 62).astype(np.uint64)


def first_above(w: np.ndarray, u: float) -> int:
    """The first v with w_0 + .. + w_v > u * sum(w), in exact arithmetic."""
    c = np.cumsum(w, dtype=np.uint64)
    thr = Fraction(float(u)) * int(c[-1])
    return int(np.searchsorted(c, np.uint64(int(thr)), side="right"))   # c > floor(thr) <=> c > thr


def verify_probs(p, q, draft, u_accept, u_draw):
    """One sequence: p [gamma+1, V], q [gamma, V] or None (drafts taken without
    a draw), draft [gamma], u_accept [gamma], u_draw. Returns (tau, committed
    [gamma+1] padded with -1, next_anchor)."""
    p = probability(p)
    q = None if q is None else probability(q)
    gamma, V = len(draft), p.shape[-1]
    a = 0
    while a < gamma:
        x = int(draft[a])
        if not 0 <= x < V:
            break
        if not float(u_accept[a]) * (1.0 if q is None else q[a, x]) < p[a, x]:
            break
        a += 1
    whole = fixed62(p[a])
    w = whole
    if a < gamma:
        if q is None:
            w = whole.copy()
            if 0 <= int(draft[a]) < V:
                w[int(draft[a])] = 0
        else:
            f = fixed62(q[a])
            w = np.where(whole > f, whole - f, np.uint64(0))
        if not w.any():
            w = whole
    # without mass, and with more than a probability could have (4 and up), there is nothing to draw from
    y = first_above(w, u_draw) if 0 < int(w.sum(dtype=object)) < 1 << 64 else 0
    com = np.full(gamma + 1, -1, dtype=np.int64)
    com[:a] = np.asarray(draft)[:a]
    com[a] = y
    return a + 1, com, y
