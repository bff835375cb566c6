"""GPU: verification of drafts against given probabilities from given random
numbers (dflash_verify_probs) against the oracle's exact arithmetic. Results
are whole numbers and must be equal."""
import numpy as np
import pytest
import torch

import synth
from oracle import target_ref as tr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def config(dfl, V, gamma, B):
    return dfl.make_config(1, 256, 1, 256, 4, 4, 64, 512, V, gamma, V - 1, B, 128)


def run(dfl, p, q, draft, ua, ud, gamma_b=None, stream=None):
    B, R, V = p.shape
    dev = lambda t: None if t is None else torch.as_tensor(t).cuda().contiguous()  # noqa: E731
    tau, nxt = (torch.full((B + 1,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    com = torch.full((B + 1, R), 77, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfl.dflash_verify_probs(config(dfl, V, R - 1, B), dev(p), dev(q), dev(draft), dev(ua), dev(ud), tau, com, nxt, st,
                            gamma_b=dev(gamma_b), stream=stream)
    torch.cuda.synchronize()
    assert (tau[B] == 77) and (nxt[B] == 77) and (com[B] == 77).all()       # nothing behind the last sequence
    return tau[:B].cpu().numpy(), com[:B].cpu().numpy(), nxt[:B].cpu().numpy(), int(st)


def check(got, p, q, draft, ua, ud, gamma_b=None):
    tau, com, nxt, _ = got
    R = p.shape[1]
    for b in range(p.shape[0]):
        g = R - 1 if gamma_b is None else min(max(int(gamma_b[b]), 1), R - 1)
        t, c, y = tr.verify_probs(p[b, :g + 1], None if q is None else q[b, :g], draft[b, :g].numpy(), ua[b].numpy(), float(ud[b]))
        assert (tau[b], nxt[b]) == (t, y), (b, tau[b], t, nxt[b], y)
        assert com[b].tolist() == c.tolist() + [-1] * (R - 1 - g)
    return tau


def inputs(B, gamma, V, seed, greedy=False, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn((B, gamma + 1, V), generator=g) * 2.5
    q = torch.softmax(lg[:, :gamma], -1)
    p = torch.softmax(lg + 0.6 * torch.randn((B, gamma + 1, V), generator=g), -1)
    if greedy:
        draft = q.argmax(-1)
        p[:, :gamma] = 0.25 * p[:, :gamma] + 0.75 * torch.nn.functional.one_hot(draft, V)
        q = None
    else:
        draft = torch.multinomial(q.view(-1, V), 1, generator=g).view(B, gamma)
    return (p.to(dtype), q, draft.to(torch.int32), torch.rand((B, gamma), generator=g), torch.rand((B,), generator=g))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,gamma,V", [(1, 16, 151936), (5, 16, 1003), (3, 7, 4103), (40, 1, 2), (2, 16, 200003), (9, 4, 131),
                                       (130, 3, 127), (30, 5, 20011)])
def test_matches_the_oracle(dfl, dtype, greedy, B, gamma, V):
    x = inputs(B, gamma, V, B + V, greedy, dtype)
    got = run(dfl, *x)
    tau = check(got, *x)
    assert got[3] == 0
    if B * gamma > 40:
        assert tau.max() > 1 and tau.min() < gamma + 1


def test_per_sequence_blocks(dfl):
    x = inputs(6, 16, 1003, 4)
    gb = torch.tensor([16, 1, 7, 0, 99, 3], dtype=torch.int32)
    got = run(dfl, *x, gamma_b=gb)
    check(got, *x, gamma_b=gb.numpy())
    assert all(np.array_equal(a, b) for a, b in zip(run(dfl, *x)[:3], run(dfl, *x, gamma_b=torch.full((6,), 16, dtype=torch.int32))[:3]))


@pytest.mark.parametrize("V", [1000, 4096, 151936])
def test_draws_at_the_borders_of_the_distribution(dfl, V):
    """Equal weights 2^-20: border v is exactly v 2^-20 of the total's scale, and u times the total lands on it."""
    n = 256
    at = torch.linspace(0, V - 1, n).long()                   # the tokens with mass
    p = torch.zeros((n, 2, V))
    p[:, :, at] = 2.0 ** -8
    ud = torch.arange(n) / n                                  # u * total = i / 256: the border of token i
    draft = torch.full((n, 1), int(at[0]), dtype=torch.int32)
    ua = torch.zeros((n, 1))                                  # kept: the bonus row is drawn from
    x = (p, None, draft, ua, ud)
    got = run(dfl, *x)
    assert got[2].tolist() == at.tolist() and (got[0] == 2).all()
    eps = 2.0 ** -24
    got = run(dfl, p, None, draft, ua, (ud - eps).clamp(min=0.0))   # just below: the token before
    assert got[2].tolist() == [int(at[max(i - 1, 0)]) for i in range(n)]
    check(got, p, None, draft, ua, (ud - eps).clamp(min=0.0))


def test_acceptance_is_decided_in_exact_arithmetic(dfl):
    """u q = p exactly is a rejection, the next u below an acceptance; fp32 would round both products to p."""
    V = 64
    p, q = torch.zeros((2, 2, V)), torch.zeros((2, 1, V))
    q[:, 0, 3] = 0.75
    u = torch.tensor([0.7, np.nextafter(np.float32(0.7), np.float32(0))], dtype=torch.float32)
    p[:, 0, 3] = float(np.float32(float(u[0]) * 0.75))        # the rounded product
    p[:, 0, 5] = 0.3
    p[:, 1, 9] = 1.0
    x = (p, q, torch.full((2, 1), 3, dtype=torch.int32), u[:, None], torch.tensor([0.4, 0.4]))
    check(run(dfl, *x), *x)
    p[0, 0, 3] = 0.375                                        # an exact product: 0.5 * 0.75
    x = (p, q, x[2], torch.tensor([[0.5], [0.5 - 2.0 ** -25]]), x[4])
    p[1, 0, 3] = 0.375
    got = run(dfl, *x)
    check(got, *x)
    assert got[0].tolist() == [1, 2]


def test_odd_values(dfl):
    """NaN, infinities, negative values and values above one in the rows; drafts that are no tokens; uniforms at the ends."""
    B, V = 6, 517
    p, q, draft, ua, ud = inputs(B, 3, V, 12)
    p[0, :, 5], p[0, :, 7] = float("nan"), -0.5
    q[1, :, 9], q[1, :, 11] = float("nan"), float("inf")
    p[2, :, 500] = 2.0
    draft[3] = torch.tensor([-1, V, 2 ** 31 - 1])
    ud[4], ud[5] = 0.0, 1.0 - 2.0 ** -24
    ua[4] = 1.0 - 2.0 ** -24
    x = (p, q, draft, ua, ud)
    got = run(dfl, *x)
    check(got, *x)
    assert got[3] == 0 and got[0][3] == 1
    for u in (1.0, 2.0, -1.0, float("nan")):                  # outside the range: still a token
        y = run(dfl, p, q, draft, ua, torch.full((B,), u))[2]
        assert ((y >= 0) & (y < V)).all()


@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,V", [(4, 5003), (24, 1999), (48, 1001)])
@pytest.mark.parametrize("low,high", [(-72, 0), (-72, -11), (-66, -40), (-63, -58)])
def test_weights_of_every_size_are_summed_exactly(dfl, greedy, B, V, low, high):
    """Rows whose whole mass lies in the last bits that are kept, as well as in the first, for each number of CTAs."""
    g = torch.Generator().manual_seed(B + V + low)
    draw = lambda *n: torch.ldexp(1 + torch.rand(n, generator=g), torch.randint(low, high, n, generator=g))  # noqa: E731
    p, q = draw(B, 3, V), draw(B, 2, V)
    p[:, :, 1::7] = torch.ldexp(torch.ones(()), torch.randint(low, high, (B, 3, p[:, :, 1::7].shape[2]), generator=g))
    q[:, :, ::5] = p[:, :2, ::5]                              # equal: no weight
    q[:, :, 2::5] = 0.0
    p[:, :, 3::11], q[:, :, 4::11] = 1e-42, 1e-42             # subnormal
    draft = torch.randint(0, V, (B, 2), generator=g, dtype=torch.int32)
    x = (p.clamp(max=1.0), None if greedy else q, draft, torch.rand((B, 2), generator=g) * (0.01 if low == -72 else 1.0),
         torch.rand((B,), generator=g))
    got = run(dfl, *x)
    check(got, *x)
    assert got[3] == (dfl.ERR_INVALID_ARG if high == 0 else 0)   # those rows' weights sum to 100 and more


@pytest.mark.parametrize("B", [2, 24, 48])
def test_sums_that_are_no_probabilities(dfl, B):
    """Weights that sum to 4 or more give token 0 and an error, below that a token; in one lane or spread over all."""
    V = 4001
    p, q, draft, ua, ud = inputs(B, 1, V, 17, greedy=True)
    p[:] = 0.0
    ua[:] = 0.5                                               # the only draft is rejected
    draft[:] = V - 1
    for where, over in ((torch.arange(4) * 32, True), (torch.arange(3) * 32, False), (torch.arange(4) * 1000 + 9, True),
                        (torch.arange(3) * 1000 + 9, False), (torch.arange(64) * 32, True), (torch.arange(128), True)):
        p[:, 0, :] = 0.0
        p[:, 0, where] = 1.0
        x = (p, q, draft, ua, ud)
        got = run(dfl, *x)
        check(got, *x)
        assert got[3] == (dfl.ERR_INVALID_ARG if over else 0)
        assert not over or (got[2] == 0).all()


def test_rows_without_mass(dfl):
    V = 300
    p, q, draft, ua, ud = inputs(3, 2, V, 13)
    q[0] = p[0, :2]                                           # no residual: drawn from p itself
    ua[0] = 1.0 - 2.0 ** -24
    p[1] = 0.0                                                # no target mass at all
    x = (p, q, draft, ua, ud)
    got = run(dfl, *x)
    check(got, *x)
    assert got[3] == dfl.ERR_INVALID_ARG and got[2][1] == 0 and got[0][1] == 1
    p[2, :, 1:] = 0.0                                         # one token holds all mass
    p[2, :, 0] = 2.0 ** -40
    x = (p, q, draft, ua, ud)
    check(run(dfl, *x), *x)


def test_greedy_drafts_of_a_rejected_only_token(dfl):
    """p has its whole mass on the rejected draft: the residual is empty and p itself is drawn from."""
    V = 50
    p = torch.zeros((1, 2, V))
    p[:, :, 7] = 0.5
    x = (p, None, torch.full((1, 1), 7, dtype=torch.int32), torch.tensor([[0.75]]), torch.tensor([0.3]))
    got = run(dfl, *x)
    assert got[0].tolist() == [1] and got[2].tolist() == [7]
    check(got, *x)


def test_frequencies_follow_the_target(dfl):
    """Drafts from q and even grids of both uniforms: the first committed token has the target's frequencies."""
    V, N, B = 6, 64, 64 * 64
    g = torch.Generator().manual_seed(3)
    p1, q1 = torch.softmax(torch.randn(V, generator=g), 0), torch.softmax(torch.randn(V, generator=g), 0)
    p = p1.expand(B, 2, V).contiguous()
    q = q1.expand(B, 1, V).contiguous()
    ua = ((torch.arange(B) % N + 0.5) / N)[:, None]
    ud = (torch.arange(B) // N + 0.5) / N
    mass = np.zeros(V)
    for x in range(V):
        got = run(dfl, p, q, torch.full((B, 1), x, dtype=torch.int32), ua, ud)
        mass += float(q1[x]) * np.bincount(got[1][:, 0], minlength=V) / B
    # the acceptance border falls inside one of 64 cells of a draft, a draw's border inside one of 64
    np.testing.assert_allclose(mass, p1.numpy(), atol=2.0 / N)


def test_same_answer_every_time_on_a_stream_and_from_a_graph(dfl):
    B, gamma, V = 4, 16, 20011
    p, q, draft, ua, ud = (t.cuda() for t in inputs(B, gamma, V, 31))
    cfg, st = config(dfl, V, gamma, B), torch.zeros(1, dtype=torch.int32, device="cuda")
    tau, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    com = torch.empty((B, gamma + 1), dtype=torch.int32, device="cuda")

    def call():
        dfl.dflash_verify_probs(cfg, p, q, draft, ua, ud, tau, com, nxt, st)

    call()
    torch.cuda.synchronize()
    want = com.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        com.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(com, want)
    ud.copy_(torch.rand(B, generator=torch.Generator().manual_seed(8)))
    graph.replay()
    torch.cuda.synchronize()
    check((tau.cpu().numpy(), com.cpu().numpy(), nxt.cpu().numpy(), 0), p.cpu(), q.cpu(), draft.cpu(), ua.cpu(), ud.cpu())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0, 3])
def test_acceptance_clamps_entries_to_probabilities(dfl, dtype, at):
    """The drafted token itself lies on a NaN, negative, infinite or larger entry of q, of p or of both, first or behind kept ones."""
    from tests.test_oracle_target import ODD_ENTRIES
    B, V, gamma = len(ODD_ENTRIES), 517, at + 2
    p, q = torch.zeros((B, gamma + 1, V)), torch.full((B, gamma, V), 2.0 ** -12)
    p[:, :, 300] = 1.0                                        # the drafts beside the odd one are kept
    p[:, at, 300], p[:, at, 5] = 0.0, 0.3125
    draft = torch.full((B, gamma), 300, dtype=torch.int32)
    draft[:, at] = 500
    ua = torch.full((B, gamma), 0.5)
    for b, (u, qx, px, _) in enumerate(ODD_ENTRIES):
        ua[b, at], q[b, at, 500], p[b, at, 500] = u, qx, px
    x = (p.to(dtype), q, draft, ua, torch.linspace(0, 0.99, B))
    got = run(dfl, *x)
    assert got[0].tolist() == [gamma + 1 if kept else at + 1 for _, _, _, kept in ODD_ENTRIES]
    assert got[3] == 0
    check(got, *x)
    got = run(dfl, x[0], None, *x[2:])
    assert got[0].tolist() == [gamma + 1 if u < min(px, 1.0) else at + 1 for u, _, px, _ in ODD_ENTRIES]
    check(got, x[0], None, *x[2:])
