"""Pins of the target-side oracle against facts fixed outside it: attention
against torch's own on the visible keys, the norm and rotation against complex
numbers, the verification rule against exact enumeration. CPU only."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import dflash_ref as ref
from oracle import target_ref as tr


def test_norm_rope_is_a_complex_rotation_of_the_unit_rms_head():
    g = np.random.default_rng(0)
    x, gain, pos = g.normal(size=(5, 3, 64)), 1 + 0.1 * g.normal(size=64), np.array([0, 1, 7, 500, 32767])
    y = tr.qk_norm_rope(x, gain, pos, 0.0, 1e6)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True)) * gain
    z = (n[..., :32] + 1j * n[..., 32:]) * np.exp(1j * pos[:, None, None] * 1e6 ** (-np.arange(32) / 32.0))
    np.testing.assert_allclose(y, np.concatenate([z.real, z.imag], -1), atol=1e-11)
    np.testing.assert_allclose(tr.qk_norm_rope(x, None, pos, 1e-6, 0.0), x)


@pytest.mark.parametrize("ctx,n,causal", [(0, 1, True), (0, 4, True), (9, 3, True), (9, 3, False), (0, 5, False)])
def test_chunk_attention_against_torch(ctx, n, causal):
    g = torch.Generator().manual_seed(ctx + n)
    q = torch.randn((n, 4, 64), generator=g, dtype=torch.float64)
    k, v = (torch.randn((2, ctx + n, 64), generator=g, dtype=torch.float64) for _ in range(2))
    mask = torch.ones((n, ctx + n), dtype=torch.bool)
    if causal:
        mask = mask.tril(ctx)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 0), v.repeat_interleave(2, 0), attn_mask=mask).transpose(0, 1)
    got, mass, _ = tr.chunk_attention(q.numpy(), k.numpy(), v.numpy(), ctx, causal)
    np.testing.assert_allclose(got, want.numpy(), atol=1e-12)
    assert (np.abs(got) <= mass + 1e-12).all()


def test_full_chunk_attention_is_the_drafters_block_attention():
    g = np.random.default_rng(3)
    c = ref.Cfg(1, 64, 1, 64, 4, 2, 64, 64, 100, 4, 99)
    q, k, v = g.normal(size=(5, 4, 64)), g.normal(size=(2, 12, 64)), g.normal(size=(2, 12, 64))
    np.testing.assert_allclose(tr.chunk_attention(q, k, v, 7, causal=False)[0], ref.attention(c, q, k, v), atol=1e-12)


def test_a_row_without_keys_gives_zeros():
    out, _, _ = tr.chunk_attention(np.ones((3, 2, 64)), np.ones((1, 2, 64)), np.ones((1, 2, 64)), -1)
    assert not out[0].any() and out[1:].all()


def test_the_draw_is_the_inverse_of_the_distribution_function():
    w = tr.fixed62([0.25, 0.0, 0.5, 0.25])
    for u, want in [(0.0, 0), (0.2499, 0), (0.25, 2), (0.7499, 2), (0.75, 3), (1 - 2.0 ** -24, 3)]:
        assert tr.first_above(w, u) == want, u
    assert tr.first_above(tr.fixed62([0.0, 0.0, 2.0 ** -30, 0.0]), 0.9) == 2


def test_fixed_point_values():
    x = np.array([1.0, 0.5, 2.0 ** -38 * (1 + 2.0 ** -23), 2.0 ** -62, 2.0 ** -63, 0.0, -1.0, np.nan, 3.0], np.float32)
    want = [1 << 62, 1 << 61, int(Fraction(float(x[2])) * 2 ** 62) , 1, 0, 0, 0, 0, 1 << 62]
    assert [int(v) for v in tr.fixed62(x)] == want


@pytest.mark.parametrize("greedy", [False, True])
def test_committed_token_follows_the_target_exactly(greedy):
    """Sum over drafts and over a grid of both uniforms: the first committed token is distributed as p_0."""
    V, N = 4, 64
    p = np.array([[24, 8, 20, 12], [16, 16, 16, 16]]) / 64.0
    q = np.array([[8, 8, 32, 16]]) / 64.0
    mass = np.zeros(V)
    for x in range(V):
        px = (1.0 if x == 2 else 0.0) if greedy else q[0, x]
        for i in range(N):
            for j in range(N):
                t, com, _ = tr.verify_probs(p, None if greedy else q, [x], [(i + 0.5) / N], (j + 0.5) / N)
                mass[com[0]] += px / (N * N)
                assert t == 1 or com[0] == x
    # u * q < p has its border inside a grid cell at most; a cell weighs 1 / N of one draft
    np.testing.assert_allclose(mass, p[0], atol=1.0 / N)


def test_verification_corner_cases():
    p = np.zeros((3, 5))
    p[:, 1] = 1.0
    assert tr.verify_probs(p, None, [1, 1], [0.9, 0.9], 0.5)[0] == 3             # all kept, bonus
    assert tr.verify_probs(p, None, [1, 0], [0.9, 0.0], 0.5)[1].tolist() == [1, 1, -1]   # 0 < 0 is false
    assert tr.verify_probs(p, None, [7, 1], [0.0, 0.0], 0.5)[0] == 1             # not a token
    same = np.full((2, 4), 0.25)
    t, com, y = tr.verify_probs(same, same[:1], [3], [1.0], 0.6)                 # p == q: drawn from p
    assert (t, com.tolist(), y) == (1, [2, -1], 2)
    assert tr.verify_probs(np.zeros((2, 4)), None, [0], [0.1], 0.3)[2] == 0      # no mass at all


# Entries that are no probabilities, (u, q_j(x_j), p_j(x_j), kept): NaN and negative ones count as 0, larger ones as 1.
ODD_ENTRIES = [(0.6, 2.0, 1.0, True), (0.6, float("nan"), 0.25, True), (0.6, -0.5, 0.0, False), (0.3, -2.0, -0.5, False),
               (0.0, float("inf"), 0.25, True), (0.5, float("inf"), 0.75, True), (0.5, float("inf"), 0.25, False),
               (0.0, float("nan"), 0.0, False), (0.9, 0.5, float("nan"), False), (0.9, 0.5, -1.0, False), (0.9, 1.0, 2.0, True),
               (0.9, 1.0, float("inf"), True), (0.5, float("-inf"), float("nan"), False), (0.5, 0.5, 0.75, True)]


@pytest.mark.parametrize("u,q,p,kept", ODD_ENTRIES)
def test_acceptance_clamps_entries_to_probabilities(u, q, p, kept):
    P, Q = np.zeros((2, 12)), np.zeros((1, 12))
    P[0, 5], P[1, 9] = 0.3, 1.0
    P[0, 3], Q[0, 3] = p, q
    t, com, _ = tr.verify_probs(P, Q, [3], [u], 0.25)
    assert t == (2 if kept else 1) and (com[0] == 3) >= kept
    # a drafter that draws nothing: q is one
    t, _, _ = tr.verify_probs(P, None, [3], [u], 0.25)
    assert t == (2 if not np.isnan(p) and u < min(p, 1.0) else 1)
