"""GPU: shaped distributions and draws (dflash_sample) against the float64 oracle.

Which entries have weight has to be equal, and tokens: weights are off by at most
2^-27 of themselves, so that every prefix of their sum is, and a token can be
the neighbour of the oracle's only where the draw lies within 2^-27 of the border
between the two (even weights at a very high temperature, where a draw of 1/2
meets a border to the last bit). A probability is off by 2^-27 (its weight) and
four roundings of 2^-24 at most, and by 2^-43 of the largest weight that the
integer cuts off; a row's sum is at least that weight."""
import numpy as np
import pytest
import torch

from oracle import tree_ref as tt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def dev(v, dt=torch.float32):
    return None if v is None else torch.tensor(v, dtype=dt, device="cuda")


def run(dfl, x, u, T=None, k=None, p=None, m=None, probs=True, tokens=True, **kw):
    N, V = x.shape
    tok = torch.full((N + 1,), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((N, V), 9.0, device="cuda") if probs else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfl.dflash_sample(x, dev(u) if tokens else None, tok if tokens else None, st, temperature=dev(T), top_k=dev(k, torch.int32),
                      top_p=dev(p), min_p=dev(m), probs=pr, **kw)
    torch.cuda.synchronize()
    assert int(tok[N]) == -7
    return tok[:N].tolist(), None if pr is None else pr.double().cpu().numpy(), int(st)


def check(dfl, x, u, T=None, k=None, p=None, m=None, **kw):
    """Every row against the oracle, with and without the distributions."""
    tok, pr, st = run(dfl, x, u, T, k, p, m, **kw)
    alone, _, _ = run(dfl, x, u, T, k, p, m, probs=False, **kw)
    _, only, _ = run(dfl, x, u, T, k, p, m, tokens=False, **kw)
    assert tok == alone and np.array_equal(pr, only)
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    xs = x.double().cpu().numpy()
    big = float(torch.finfo(x.dtype).max)
    bad = False
    for n in range(x.shape[0]):
        want = tt.shape(np.where(xs[n] == np.inf, big, xs[n]), 1.0 if T is None else f32(T[n]), 0 if k is None else k[n],
                        1.0 if p is None else f32(p[n]), 0.0 if m is None else f32(m[n]))
        if want is None:
            assert tok[n] == 0 and not pr[n].any()
            bad = True
            continue
        assert ((pr[n] > 0) <= (want > 0)).all() and ((pr[n] == 0) <= (want < 2.0 ** -42)).all(), (n, (pr[n] > 0).sum(), (want > 0).sum())
        assert (np.abs(pr[n] - want) <= 2.0 ** -22 * 1.01 * want + 2.0 ** -43).all(), (n, np.abs(pr[n] - want).max())
        y = tt.draw(want, f32(u[n]))
        border = np.cumsum(want)[min(tok[n], y)]
        assert tok[n] == y or (want[tok[n]] > 0 and not want[min(tok[n], y) + 1:max(tok[n], y)].any()
                               and abs(border - f32(u[n])) <= 2.0 ** -27), (n, tok[n], y, border)
    assert st == (dfl.ERR_INVALID_ARG if bad else 0)
    return tok, pr


def logits(N, V, dtype, seed, kind="zipf"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "zipf":
        x = torch.empty((N, V), device="cuda").exponential_(generator=g) * (1.0 + torch.rand((N, 1), generator=g, device="cuda")) - 5
    else:
        x = torch.randn((N, V), generator=g, device="cuda") * 2.5
    return x.to(dtype)


def settings(N, seed):
    r = np.random.default_rng(seed)
    return dict(T=r.choice([0.0, 0.3, 0.7, 1.0, 1.3], N).tolist(), k=[int(v) for v in r.choice([0, 0, 1, 2, 20, 50, 700], N)],
                p=r.choice([1.0, 0.5, 0.9, 0.95, 0.999, 0.0], N).tolist(), m=r.choice([0.0, 0.0, 0.05, 0.3, 1.0], N).tolist())


def uniforms(N, seed):
    return np.random.default_rng(seed).random(N, dtype=np.float32).tolist()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1003, 4103, 32000, 151936, 200003])
def test_matches_the_oracle(dfl, V, dtype):
    N = 24 if V < 100000 else 10
    for kind in ("zipf", "normal"):
        check(dfl, logits(N, V, dtype, V + len(kind), kind), uniforms(N, V), **settings(N, V))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 3, 37, 150, 320])
def test_rows_by_the_number(dfl, N, dtype):
    """Every way that a row is divided over CTAs."""
    check(dfl, logits(N, 20011, dtype, N), uniforms(N, N), **settings(N, N))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("one", ["T", "k", "p", "m", "none"])
def test_each_setting_alone(dfl, one, dtype):
    N, V = 12, 50257
    s = settings(N, 5)
    s["k"] = [5000, 40000, 60000, 50257, 50256, 513, 4097, 3, -1, 0, 1, 100]
    check(dfl, logits(N, V, dtype, 3), uniforms(N, 3), **{k: v for k, v in s.items() if k == one})


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [500, 30011])
def test_ties(dfl, V, dtype):
    """Values on a coarse grid, also around zero and of either sign of it: borders fall among equal entries."""
    N = 40
    x = (logits(N, V, F32, 7, "normal") / 1.5).round() * 0.5
    x[::2] = torch.where(x[::2] == 0, -0.0, x[::2])
    x[::4, ::3] = torch.where(x[::4, ::3] == 0, 0.0, x[::4, ::3])
    x[5] = 1.25                                 # all equal
    x[6] = -3.0
    x[7] = 0.0
    check(dfl, x.to(dtype), uniforms(N, 8), **settings(N, 9))
    s = settings(N, 10)
    check(dfl, x.to(dtype), uniforms(N, 11), T=[1.0] * N, k=[int(v) for v in np.random.default_rng(1).integers(1, V, N)], p=s["p"])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_masked_infinite_and_extreme_entries(dfl, dtype):
    N, V = 20, 9001
    low, big = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = logits(N, V, dtype, 13)
    x[0, ::2] = -float("inf")
    x[1, 1:] = -float("inf")                    # one entry left
    x[2, :] = -float("inf")                     # none
    x[3, ::3] = low
    x[4, :] = low                               # all of the lowest value: even weights
    x[5, 77] = float("inf")
    x[6, 77:80] = float("inf")                  # even weights
    x[7, ::5] = float("nan")
    x[8, :] = float("nan")
    x[9, :] = big
    x[10, ::2] = low
    x[10, 5] = big
    x[11] = x[11] * 1e-30
    x[12] = x[12] * 1e30
    x[13, :] = -1e-38
    x[14, :8990] = -float("inf")                # the last entries alone
    x[15, 11:] = -float("inf")                  # fewer entries than k
    x[16, 40:] = low
    for s in (settings(N, 17), dict(T=[1.0] * N), dict(T=[1.0] * N, k=[50] * N), dict(T=[0.8] * N, p=[0.9] * N),
              dict(T=[1.0] * N, k=[3000] * N, p=[0.9] * N, m=[0.01] * N), dict(T=[0.0] * N)):
        check(dfl, x, uniforms(N, 19), **s)


def test_temperatures_and_uniforms_at_their_ends(dfl):
    V = 5003
    T = [1e-30, 1e-6, 1e-2, 30.0, 1e6, 1e30, float("inf"), 0.7, 0.7, 0.7, 0.7, 0.7]
    N = len(T)
    x = logits(N, V, F32, 23)
    u = [0.5] * 7 + [0.0, 1e-40, 1e-30, float(np.float32(1 - 2.0 ** -24)), 0.9999]
    check(dfl, x, u, T=[min(t, 3e38) for t in T])
    check(dfl, x, u, T=[min(t, 3e38) for t in T], p=[0.9, 0.9, 0.9, 0.9, 0.9, 0.5, 0.5, 1e-40, 1e-10, 0.0, float(np.float32(1 - 2.0 ** -24)), 0.99])
    tok, pr, st = run(dfl, x, u, T=T)          # an infinite temperature: even weights
    assert st == 0 and np.allclose(pr[6], 1 / V, rtol=1e-6)
    for bad in (-1.0, float("nan")):
        tok, pr, st = run(dfl, x, u, T=T[:3] + [bad] + T[4:])
        assert st == dfl.ERR_INVALID_ARG and tok[3] == 0 and not pr[3].any() and pr[2].any()


@pytest.mark.parametrize("V", [28, 1000, 5000])
@pytest.mark.parametrize("T", [0.69, 0.71, 1.38, 1.42, 2.84, 5.0, 5.52, 5.68, 11.04, 11.36])
def test_equal_entries_far_from_zero(dfl, T, V):
    """Equal entries have equal weights whatever an exponent rounds to, so that exactly p V of them are p of the weight; at
    these temperatures log2(e) / T lies far from the float next to it, at these values that counts most."""
    vals = [s * f * T / 1.4427 for f in (30, 100, 250, 500, 900, 1000) for s in (1, -1)]
    p = [0.25, 0.5, 0.75]
    x = torch.tensor(vals, device="cuda").repeat_interleave(3)[:, None].expand(-1, V).contiguous()
    N = x.shape[0]
    tok, pr, st = run(dfl, x, [0.999] * N, T=[T] * N, p=p * len(vals))
    assert st == 0
    for n in range(N):
        k = int(V * p[n % 3])
        assert (pr[n, :k] > 0).all() and not pr[n, k:].any(), (n, vals[n // 3], p[n % 3], (pr[n] > 0).sum(), k)
        assert tok[n] == int(k * float(np.float32(0.999)))


def test_settings_that_are_off(dfl):
    V, N = 2000, 6
    x, u = logits(N, V, F32, 29), uniforms(N, 29)
    want = run(dfl, x, u)
    nan = float("nan")
    got = run(dfl, x, u, T=[1.0] * N, k=[0, -1, -2 ** 31, V, V + 1, 2 ** 31 - 1], p=[1.0, 2.0, nan, 1.0, 1.0, 7.0],
              m=[0.0, -1.0, nan, 0.0, 0.0, -0.0])
    assert got[0] == want[0] and np.array_equal(got[1], want[1])
    got = run(dfl, x, u, m=[5.0] * N)          # above 1 counts as 1
    assert got[0] == x.argmax(-1).tolist()
    clamped = run(dfl, x, [-3.0, nan, 1.0, 7.0, 0.0, 0.5])
    assert clamped[0][0] == clamped[0][1] == clamped[0][4] == 0


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V,ld,off", [(1001, 1001, 0), (1001, 1009, 3), (4096, 4104, 1), (777, 2000, 5), (30000, 30001, 7)])
def test_rows_at_any_element_and_stride(dfl, V, ld, off, dtype):
    """Entries beside a row belong to others: larger than all of its own."""
    N = 5
    buf = torch.full((N * ld + off + 16,), 30.0, dtype=dtype, device="cuda")
    x = torch.as_strided(buf, (N, V), (ld, 1), off)
    x.copy_(logits(N, V, dtype, 31))
    check(dfl, x, uniforms(N, 31), **settings(N, 37))


def test_a_large_vocabulary(dfl):
    for V, dtype in ((1 << 19, F32), ((1 << 19) - 3, BF), (300007, F32)):
        check(dfl, logits(3, V, dtype, 41), uniforms(3, 41), T=[1.0, 0.8, 1.5], k=[0, 100, 0], p=[1.0, 0.9, 0.8])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_equal_and_flat_rows_of_one_block_each(dfl, dtype):
    """Large batches: a block a row, whose lists and bins overflow: 151936 equal entries, few values, even weights."""
    N, V = 310, 151936
    x = torch.zeros((N, V), dtype=dtype, device="cuda")
    x[1::3] = logits(1, V, F32, 71, "normal")[0].round().to(dtype)
    x[2::3] = logits(1, V, dtype, 72, "normal")[0] * 0.01
    x[5, 70000:] = -float("inf")
    r = np.random.default_rng(71)
    s = dict(T=[1.0] * N, k=r.choice([0, 0, 1300, 90000, 151935], N).tolist(), p=r.choice([0.3, 0.77, 0.9999, 1.0], N).tolist())
    u = uniforms(N, 73)
    tok, pr, st = run(dfl, x, u, **s)
    alone, _, _ = run(dfl, x, u, **s, probs=False)
    assert st == 0 and tok == alone
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    for n in list(range(0, 24)) + [304, 305, 309]:
        want = tt.shape(x[n].double().cpu().numpy(), 1.0, s["k"][n], f32(s["p"][n]))
        assert ((pr[n] > 0) == (want > 0)).all(), n
        assert (np.abs(pr[n] - want) <= 2.0 ** -22 * 1.01 * want + 2.0 ** -43).all()
        y = tt.draw(want, f32(u[n]))
        assert tok[n] == y or abs(np.cumsum(want)[min(tok[n], y)] - f32(u[n])) <= 2.0 ** -27, (n, tok[n], y)


def test_many_rows(dfl):
    N, V = 3000, 1500
    x = logits(N, V, BF, 43)
    check(dfl, x, uniforms(N, 43), **settings(N, 43))


def test_draws_are_distributed_as_the_distribution(dfl):
    N, V = 20000, 37
    x = logits(1, V, F32, 47, "normal").expand(N, V)          # a stride of zero is refused
    with pytest.raises(dfl.DFlashError):
        run(dfl, x, uniforms(N, 47), probs=False)
    tok, _, _ = run(dfl, x.contiguous(), uniforms(N, 47), T=[1.2] * N, k=[20] * N, probs=False)
    want = tt.shape(x[0].double().cpu().numpy(), float(np.float32(1.2)), 20)
    got = np.bincount(tok, minlength=V)
    assert (got[want == 0] == 0).all()
    on = want > 0
    chi = ((got[on] - N * want[on]) ** 2 / (N * want[on])).sum()
    assert chi < 19 + 6 * np.sqrt(2 * 19)                     # 19 degrees of freedom


def test_from_a_graph_on_another_stream_and_beside_another_call(dfl):
    N, V = 17, 151936
    a, b = logits(N, V, F32, 53), logits(40, V, BF, 59)
    sa, sb = settings(N, 53), settings(40, 59)
    ua, ub = uniforms(N, 53), uniforms(40, 59)
    ta, _ = check(dfl, a, ua, **sa)
    tb, _ = check(dfl, b, ub, **sb)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (N, 40)]
    arg = [[dev(u), dict(temperature=dev(s["T"]), top_k=dev(s["k"], torch.int32), top_p=dev(s["p"]), min_p=dev(s["m"]))]
           for u, s in ((ua, sa), (ub, sb))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        dfl.dflash_sample(a, arg[0][0], out[0], st, **arg[0][1])
        dfl.dflash_sample(b, arg[1][0], out[1], st, **arg[1][1], stream=side)
    torch.cuda.synchronize()
    assert out[0].tolist() == ta and out[1].tolist() == tb
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dfl.dflash_sample(a, arg[0][0], out[0], st, **arg[0][1])
    out[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert out[0].tolist() == ta
    a.copy_(logits(N, V, F32, 54))
    graph.replay()
    torch.cuda.synchronize()
    assert out[0].tolist() == run(dfl, a, ua, **sa, probs=False)[0] and int(st) == 0


def test_empty_and_traced(dfl):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, device="cuda")
    dfl.dflash_sample(torch.zeros((0, 50), device="cuda"), none, none.int(), st)
    rec = dfl.TraceRecorder(2)
    run(dfl, logits(3, 500, BF, 61), uniforms(3, 61), trace=rec.struct)
    assert [(k, b) for k, b, _, _ in rec.records()] == [(dfl.K_VERIFY, 3.0 * 500 * 6)]


def spread(at, side, T, V, wide, seed):
    """Rows [len(at), V] whose maxima m have |m| log2(e) / T = at, on one side of zero; the others lie below them by
    T `wide` times an exponential value."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.tensor(at, dtype=torch.float64, device="cuda")[:, None] * (side * float(np.float32(T)) / 1.4426950408889634)
    below = torch.empty((len(at), V), dtype=torch.float64, device="cuda").exponential_(generator=g) * (wide * T)
    below.scatter_(1, torch.randint(V, (len(at), 1), generator=g, device="cuda"), 0.0)
    return (m - below).float()


@pytest.mark.parametrize("wide", [1.6, 0.6], ids=["peaked", "flat"])
@pytest.mark.parametrize("T", [1e-3, 0.7, 1.0, 1e4])
def test_maxima_in_every_range_of_the_weights(dfl, T, wide):
    """Weights reduce x log2(e) / T, or (x - m) log2(e) / T from 32768 on; up to 1024 their sum may be fp32. fp32 rows on
    each side of these and of 65536 (where a multiple of 2^-8 stops being a float), at maxima of either sign."""
    at = [900, 1020, 1030, 5000, 16384, 30000, 32700, 32760, 32767, 32769, 32800, 40000, 65400, 65480, 65500, 65520, 65530, 65540, 65560,
          65600, 1e5, 1e6]
    N = len(at)
    for side in (1, -1):
        x = spread(at, side, T, 3001, wide, 83)
        u = uniforms(N, 84)
        for s in (dict(), dict(p=[0.9] * N), dict(p=[0.6] * N, m=[1e-3] * N), dict(k=[40] * N, p=[0.95] * N), dict(k=[2000] * N, p=[0.7] * N)):
            check(dfl, x, u, T=[T] * N, **s)
    x = spread(at[8:18], -1, T, 60013, wide, 85)
    check(dfl, x, uniforms(10, 86), T=[T] * 10, p=[0.9] * 10)


@pytest.mark.parametrize("V", [28, 1000, 5000])
@pytest.mark.parametrize("T", [0.72108847, 1.4421769, 2.8843539, 5.7687078, 11.537416, 2.79, 5.71])
def test_equal_entries_at_temperatures_whose_factor_lies_farthest_off(dfl, T, V):
    """As above where log2(e) / T lies up to 1.22 half steps above the float that the fp32 sum multiplies by: its own
    rounding, and that of log2(e)."""
    vals = [s * f * T / 1.442696 for f in (300, 700, 980, 1010, 1020, 1023) for s in (1, -1)]
    p = [0.25, 0.5, 0.75]
    x = torch.tensor(vals, device="cuda").repeat_interleave(3)[:, None].expand(-1, V).contiguous()
    N = x.shape[0]
    tok, pr, st = run(dfl, x, [0.999] * N, T=[T] * N, p=p * len(vals))
    assert st == 0
    for n in range(N):
        k = int(V * p[n % 3])
        assert (pr[n, :k] > 0).all() and not pr[n, k:].any(), (n, vals[n // 3], p[n % 3], (pr[n] > 0).sum(), k)
        assert tok[n] == int(k * float(np.float32(0.999)))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1e30, 1e38, 2e38, 3e38, float("inf")])
def test_min_p_at_very_high_temperatures(dfl, T, dtype):
    """Nearly even weights, which no min-p below 1 parts: T ln(min_p) passes fp32's range."""
    V, ms = 3001, [1e-45, 1e-6, 0.05, 0.999]
    x = logits(2 * len(ms), V, dtype, 97, "normal")
    x[1, ::3] = -float("inf")
    N = x.shape[0]
    u = [float(np.float32(v)) for v in np.linspace(0.013, 0.987, N)]
    check(dfl, x, u, T=[T] * N, m=ms * 2)
    check(dfl, x, u, T=[T] * N, m=ms * 2, k=[7, 40, 1700, 2000, 0, 3000, 1, 300])
    # min-p of 1: entries as large as the largest one, and all finite ones where the temperature is infinite
    x[:, 11] = x[:, 2000] = x.amax(1)
    tok, pr, st = run(dfl, x, u, T=[T] * N, m=[1.0] * N)
    f = x.double().cpu().numpy()
    on = f > -np.inf if T == float("inf") else f == f.max(1, keepdims=True)
    assert st == 0 and ((pr > 0) == on).all()
    assert (np.abs(pr - on / on.sum(1, keepdims=True)) <= 2.0 ** -22 * 1.01 * on).all()   # even weights
    for n in range(N):
        assert on[n, tok[n]] and on[n, :tok[n] + 1].sum() == np.floor(on[n].sum() * u[n]) + 1


def test_an_infinite_temperature_is_even_whatever_the_entries(dfl):
    V, big = 2003, torch.finfo(F32).max
    x = logits(6, V, F32, 101, "normal") * 1e37
    x[0, ::2] = -big
    x[0, 1::2] = big
    x[1, :] = -big
    x[2, 5] = float("inf")
    x[3, ::7] = float("nan")
    x[4, 9:] = -float("inf")
    for s in (dict(), dict(k=[30] * 6), dict(k=[1500] * 6, p=[0.71] * 6), dict(p=[0.3] * 6, m=[0.5] * 6)):
        check(dfl, x, [0.0, 0.1, 0.37, 0.613, 0.9, 0.999], T=[float("inf")] * 6, **s)


def test_temperatures_beyond_the_range_count_as_its_ends(dfl):
    V = 1009
    for T, end in ((1e38, 2.0 ** 100), (3e38, 2.0 ** 100), (1e-38, 2.0 ** -100), (1e-45, 2.0 ** -100)):
        x = logits(4, V, F32, 103, "normal") * (1e30 if T > 1 else 1e-30)
        u = uniforms(4, 104)
        for s in (dict(), dict(m=[1e-20, 0.05, 0.9, 1.0]), dict(p=[0.8] * 4)):
            got, want = run(dfl, x, u, T=[T] * 4, **s), run(dfl, x, u, T=[end] * 4, **s)
            assert got[0] == want[0] and np.array_equal(got[1], want[1]) and got[2] == want[2] == 0
            assert (want[1] > 0).sum() > 4 or "m" in s
    # a border below the lowest number: what lies one step under the largest entry has a weight of exp(-16)
    x = torch.full((1, V), torch.finfo(F32).min, device="cuda")
    x[0, 5] = float(np.nextafter(np.float32(torch.finfo(F32).min), np.float32(0)))
    check(dfl, x, [0.99999], T=[2.0 ** 100], m=[1e-12])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(310, 151936), (10, 200003), (3, 1 << 19), (10, 1 << 19)])
def test_nan_and_infinite_entries_of_rows_that_are_read_again(dfl, N, V, dtype):
    """Rows too long for shared memory: every pass reads the entries as they came, NaN and infinities among them."""
    r = np.random.default_rng(N + V)
    x = logits(N, V, dtype, 107)
    for n in range(N):
        row, kind = x[n], n % 8
        if kind in (2, 5):
            row *= 0.01                                  # flat
        if kind in (4, 7):
            row.zero_()                                  # equal
        if kind in (0, 4, 5):
            row[int(r.integers(0, 7))::7] = float("nan")
        if kind in (1, 7):
            row[int(r.integers(0, V // 2)):int(r.integers(V // 2, V))] = float("nan")
        if kind in (1, 2, 5):
            row[3::5] = -float("inf")
        if kind == 3:
            row[int(r.integers(0, V))] = float("inf")
        if kind == 6:
            row[torch.tensor(r.integers(0, V, 50), device="cuda")] = float("inf")
        if kind == 0 and n % 16 == 8:
            row.fill_(float("nan"))
    s = dict(T=r.choice([0.0, 0.7, 1.0, 1.0, 1.3], N).tolist(), k=[int(v) for v in r.choice([0, 0, 0, 20, 1300, 90000], N)],
             p=r.choice([0.3, 0.77, 0.9999, 1.0], N).tolist(), m=r.choice([0.0, 0.0, 0.05], N).tolist())
    u = uniforms(N, 109)
    tok, pr, st = run(dfl, x, u, **s)
    alone, _, _ = run(dfl, x, u, **s, probs=False)
    assert tok == alone
    f32, big = lambda v: float(np.float32(v)), float(torch.finfo(dtype).max)  # noqa: E731
    for n in sorted(set(list(range(min(N, 26))) + [N - 1, N - 2, N - 3])):
        f = x[n].double().cpu().numpy()
        want = tt.shape(np.where(f == np.inf, big, f), f32(s["T"][n]), s["k"][n], f32(s["p"][n]), f32(s["m"][n]))
        if want is None:
            assert tok[n] == 0 and not pr[n].any()
            continue
        assert ((pr[n] > 0) <= (want > 0)).all() and ((pr[n] == 0) <= (want < 2.0 ** -42)).all(), n
        assert (np.abs(pr[n] - want) <= 2.0 ** -22 * 1.01 * want + 2.0 ** -43).all(), n
        y = tt.draw(want, f32(u[n]))
        assert tok[n] == y or abs(np.cumsum(want)[min(tok[n], y)] - f32(u[n])) <= 2.0 ** -27, (n, tok[n], y)
    assert st == (dfl.ERR_INVALID_ARG if N > 8 else 0)
