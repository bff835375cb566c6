"""GPU: per-head norms with rotary positions, dense (dflash_qk_norm_rope) and
on the way into a paged cache (dflash_kv_append_paged), against the float64
oracle.

Bound of one output y = a c - b s (a, b normed values, |c|, |s| <= 1): the
fp32 steps before the rotation (sum of Dh squares in a tree and in registers,
mean, square root, reciprocal, two products: at most 24 roundings of 2^-24
that act on a and b, the sum's own share halved by the root) and the three of
the rotation and the table's one give 32 * 2^-24 * (|a| + |b|); storage in
bf16 adds 2^-8 |y| (half a step), in fp32 2^-24 |y|, inside the former."""
import numpy as np
import pytest
import torch

from oracle import target_ref as tr
from oracle.dflash_ref import f64

pytestmark = pytest.mark.gpu

THETA, EPS = 1e6, 1e-6


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def tables(dfl, dh, n):
    cfg = dfl.make_config(1, 256, 1, 256, 4, 4, dh, 512, 1000, 4, 999, 1, 128, rope_theta=THETA)
    c, s = dfl.dflash_rope_tables(cfg, n)
    return c.cuda(), s.cuda()


def randn(g, shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).cuda()


def assert_rows(got, x, gain, pos, what, theta=THETA):
    want = tr.qk_norm_rope(x, gain, pos, EPS, theta)
    flat = np.abs(tr.qk_norm_rope(x, gain, pos, EPS, 0.0))
    h = flat.shape[-1] // 2
    pair = np.concatenate([flat[..., :h] + flat[..., h:]] * 2, -1)
    store = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    err = np.abs(f64(got) - want)
    assert (err <= 32 * 2.0 ** -24 * pair + store * np.abs(want)).all(), (what, err.max())


TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "f32_to_bf16": (torch.float32, torch.bfloat16),
         "f32": (torch.float32, torch.float32)}


def out_code(dfl, dt):
    return dfl.BF16 if dt == torch.bfloat16 else dfl.F32


@pytest.mark.parametrize("types", TYPES, ids=list(TYPES))
@pytest.mark.parametrize("hq,hkv,dh", [(32, 8, 128), (4, 4, 64), (7, 1, 128), (10, 2, 64), (64, 1, 64), (1, 1, 128)])
@pytest.mark.parametrize("T", [1, 2, 17, 133])
def test_norm_rope_matches_the_oracle(dfl, types, hq, hkv, dh, T):
    ti, to = TYPES[types]
    g = torch.Generator().manual_seed(T * 1000 + hq)
    heads = dfl.make_heads(1, hq, hkv, dh, rms_eps=EPS, dtype=out_code(dfl, to))
    qkv = randn(g, (T, (hq + 2 * hkv) * dh), ti, 2.0)          # parts of one projection's rows
    q, k = qkv[:, :hq * dh].view(T, hq, dh), qkv[:, hq * dh:(hq + hkv) * dh].view(T, hkv, dh)
    gq, gk = randn(g, (dh,), to, 0.1, 1.0), randn(g, (dh,), to, 0.1, 1.0)
    pos = torch.randint(0, 33000, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    cos, sin = tables(dfl, dh, 33000)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full((T, hq, dh), 7.0, dtype=to, device="cuda")
    ko = torch.full((T + 3, hkv + 2, dh), 7.0, dtype=to, device="cuda")       # wider rows, rows behind the last
    dfl.dflash_qk_norm_rope(heads, q, k, pos.cuda(), cos, sin, qo, ko[:T, 1:1 + hkv], st, g_q=gq, g_k=gk)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert_rows(qo, q, gq, pos.numpy(), "q")
    assert_rows(ko[:T, 1:1 + hkv], k, gk, pos.numpy(), "k")
    assert (ko[T:] == 7).all() and (ko[:, 0] == 7).all() and (ko[:, 1 + hkv:] == 7).all()


def test_parts_norms_and_rotation_can_be_left_out(dfl):
    g = torch.Generator().manual_seed(5)
    heads = dfl.make_heads(1, 8, 2, 128, rms_eps=EPS)
    T, bf = 9, torch.bfloat16
    q, k = randn(g, (T, 8, 128), bf), randn(g, (T, 2, 128), bf)
    gq = randn(g, (128,), bf, 0.1, 1.0)
    pos = torch.arange(100, 100 + T, dtype=torch.int32)
    cos, sin = tables(dfl, 128, 200)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dfl.dflash_qk_norm_rope(heads, q, k, pos.cuda(), cos, sin, qo, ko, st, g_q=gq)        # keys rotated only
    assert_rows(qo, q, gq, pos.numpy(), "q normed")
    assert_rows(ko, k, None, pos.numpy(), "k without a norm")
    dfl.dflash_qk_norm_rope(heads, q, None, None, None, None, qo, None, st, g_q=gq)       # norm only
    assert_rows(qo, q, gq, pos.numpy(), "norm only", theta=0.0)
    ko.fill_(3.0)
    dfl.dflash_qk_norm_rope(heads, None, k, pos.cuda(), cos, sin, None, ko, st)
    assert_rows(ko, k, None, pos.numpy(), "keys alone")
    want = qo.clone()
    dfl.dflash_qk_norm_rope(heads, q, k, None, None, None, q, ko, st, g_q=gq)             # in place
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(ko, k) and int(st) == 0


def test_zero_rows_and_far_values(dfl):
    """A head of zeros stays zero (eps keeps the root from zero); values near the top of bf16 and tiny ones norm to unit RMS."""
    heads = dfl.make_heads(1, 3, 1, 64, rms_eps=EPS, dtype=dfl.F32)
    x = torch.zeros((2, 3, 64), device="cuda")
    x[0, 1] = 1e17
    x[0, 2] = 3.0
    g = torch.ones(64, device="cuda")
    out, st = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    dfl.dflash_qk_norm_rope(heads, x, None, None, None, None, out, None, st, g_q=g)
    want = tr.qk_norm_rope(x, g, np.zeros(2), EPS, 0.0)
    np.testing.assert_allclose(f64(out), want, rtol=32 * 2.0 ** -24)
    assert not out[0, 0].any()


def test_a_position_outside_the_tables_is_reported_and_its_row_left(dfl):
    g = torch.Generator().manual_seed(6)
    heads = dfl.make_heads(1, 4, 2, 64, rms_eps=EPS, dtype=dfl.F32)
    q, k = randn(g, (4, 4, 64)), randn(g, (4, 2, 64))
    cos, sin = tables(dfl, 64, 50)
    for bad in (-1, 50):
        pos = torch.tensor([3, bad, 49, 0], dtype=torch.int32)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        qo, ko = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
        dfl.dflash_qk_norm_rope(heads, q, k, pos.cuda(), cos, sin, qo, ko, st)
        assert int(st) == dfl.ERR_INVALID_ARG
        assert (qo[1] == 5).all() and (ko[1] == 5).all()
        keep = [0, 2, 3]
        assert_rows(qo[keep], q[keep], None, pos.numpy()[keep], "others")


# ------------------------------------------------------------------ append
def scene(dfl, types, hq, hkv, dh, ns, ctxs, n_layers=2, extra=4, seed=1, per=None):
    ti, to = TYPES[types]
    g = torch.Generator().manual_seed(seed)
    s = dict(heads=dfl.make_heads(n_layers, hq, hkv, dh, rms_eps=EPS, dtype=out_code(dfl, to)))
    T, B = sum(ns), len(ns)
    rows = randn(g, (T + extra, (hq + 2 * hkv) * dh), ti, 2.0)
    s["rows"] = rows
    s["q"] = rows[:, :hq * dh].view(T + extra, hq, dh)
    s["k"] = rows[:, hq * dh:(hq + hkv) * dh].view(T + extra, hkv, dh)
    s["v"] = rows[:, (hq + hkv) * dh:].view(T + extra, hkv, dh)
    s["gq"], s["gk"] = randn(g, (dh,), to, 0.1, 1.0), randn(g, (dh,), to, 0.1, 1.0)
    need = [(c + n + 127) // 128 for c, n in zip(ctxs, ns)]
    per = per or max(need) + 1
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((B, per), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(need[b]):
            table[b, i] = order.pop()
    s["table"] = table
    shape = (n_layers, n_pages, hkv, 128, dh)
    s["kp"], s["vp"] = torch.full(shape, 9.0, dtype=to, device="cuda"), torch.full(shape, 9.0, dtype=to, device="cuda")
    s["pages"] = dfl.KvPages(s["kp"], s["vp"], table.cuda())
    s["cu"] = torch.tensor([sum(ns[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["ctx"] = torch.tensor(ctxs, dtype=torch.int32, device="cuda")
    s["qo"] = torch.full((T + extra, hq, dh), 9.0, dtype=to, device="cuda")
    s["st"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["cos"], s["sin"] = tables(dfl, dh, max(c + n for c, n in zip(ctxs, ns)) + 1)
    return s


def run_append(dfl, s, layer=1, q=True, **kw):
    dfl.dflash_kv_append_paged(s["heads"], s["q"] if q else None, s["k"], s["v"], s["cu"], s["ctx"], layer, s["pages"],
                               s["cos"], s["sin"], s["qo"] if q else None, s["st"], g_q=s["gq"], g_k=s["gk"], **kw)


def check_append(s, ns, ctxs, layer=1, theta=THETA):
    first, touched = 0, torch.zeros(s["kp"].shape[:2] + (128,), dtype=torch.bool)
    for b, (n, c) in enumerate(zip(ns, ctxs)):
        if n == 0:
            continue
        pos = np.arange(c, c + n)
        page = s["table"][b].numpy()[pos // 128]
        rows = slice(first, first + n)
        got_k = s["kp"][layer].permute(0, 2, 1, 3)[page, pos % 128]
        got_v = s["vp"][layer].permute(0, 2, 1, 3)[page, pos % 128]
        assert_rows(got_k, s["k"][rows], s["gk"], pos, f"K of {b}", theta)
        assert torch.equal(got_v, s["v"][rows].to(got_v.dtype)), f"V of {b}"
        assert_rows(s["qo"][rows], s["q"][rows], s["gq"], pos, f"q of {b}", theta)
        touched[layer, page, pos % 128] = True
        first += n
    for pool in (s["kp"], s["vp"]):    # everything else is as it was
        assert (pool.permute(0, 1, 3, 2, 4)[~touched.cuda()] == 9).all()
    assert (s["qo"][first:] == 9).all()


@pytest.mark.parametrize("types", TYPES, ids=list(TYPES))
@pytest.mark.parametrize("hq,hkv,dh", [(32, 8, 128), (4, 4, 64), (7, 1, 128), (10, 2, 64)])
@pytest.mark.parametrize("ns,ctxs", [([1], [0]), ([17], [2048]), ([1, 1, 1], [127, 128, 0]), ([5, 0, 130, 17], [0, 40, 300, 119]),
                                     ([0, 0, 3, 0], [9, 9, 126, 9]), ([1] * 70, [3 * i for i in range(70)])])
def test_append_matches_the_oracle(dfl, types, hq, hkv, dh, ns, ctxs):
    s = scene(dfl, types, hq, hkv, dh, ns, ctxs)
    run_append(dfl, s)
    torch.cuda.synchronize()
    assert int(s["st"]) == 0
    check_append(s, ns, ctxs)


def test_keys_and_values_alone(dfl):
    s = scene(dfl, "bf16", 8, 2, 128, [3, 4], [5, 600])
    run_append(dfl, s, q=False)
    assert (s["qo"] == 9).all()
    run_append(dfl, s)
    torch.cuda.synchronize()
    check_append(s, [3, 4], [5, 600])


def test_many_sequences_find_their_rows(dfl):
    """More sequences than one probe round of the row search; empty ones among them."""
    ns = [i % 3 for i in range(1500)]
    ctxs = [(7 * i) % 130 for i in range(1500)]
    s = scene(dfl, "bf16", 2, 1, 64, ns, ctxs)
    run_append(dfl, s)
    torch.cuda.synchronize()
    assert int(s["st"]) == 0
    check_append(s, ns, ctxs)


def test_missing_pages_and_full_tables_are_capacity_errors(dfl):
    s = scene(dfl, "bf16", 8, 2, 128, [6, 4], [124, 0])
    s["table"][0, 1] = -1                                    # positions 128.. of sequence 0
    s["pages"] = dfl.KvPages(s["kp"], s["vp"], s["table"].cuda())
    run_append(dfl, s)
    assert int(s["st"]) == dfl.ERR_CAPACITY
    assert (s["qo"][4:6] == 9).all() and (s["qo"][:4] != 9).any() and (s["qo"][6:10] != 9).any()
    t = scene(dfl, "bf16", 8, 2, 128, [6], [124], per=2)
    t["table"][0, 1] = 10 ** 6                               # beyond the pool
    t["pages"] = dfl.KvPages(t["kp"], t["vp"], t["table"].cuda())
    run_append(dfl, t)
    assert int(t["st"]) == dfl.ERR_CAPACITY
    u = scene(dfl, "bf16", 8, 2, 128, [6], [124], per=2)
    u["ctx"][0] = 254                                        # 254, 255, then past the table
    u["cos"], u["sin"] = tables(dfl, 128, 400)
    u["table"][0, 1] = u["table"][0, 0]
    u["pages"] = dfl.KvPages(u["kp"], u["vp"], u["table"].cuda())
    run_append(dfl, u)
    assert int(u["st"]) == dfl.ERR_CAPACITY and (u["qo"][2:] == 9).all() and (u["qo"][:2] != 9).any()
    w = scene(dfl, "bf16", 8, 2, 128, [6], [20])
    w["ctx"][0] = -2                                         # negative positions
    run_append(dfl, w)
    assert int(w["st"]) == dfl.ERR_CAPACITY and (w["qo"][:2] == 9).all() and (w["qo"][2:6] != 9).any()


def test_row_offsets_that_disagree_with_the_rows_stay_inside_them(dfl):
    s = scene(dfl, "bf16", 8, 2, 128, [6, 4], [10, 20])
    s["cu"] = torch.tensor([0, 6, 1 << 30], dtype=torch.int32, device="cuda")   # claims more rows than there are
    s["cos"], s["sin"] = tables(dfl, 128, 400)
    run_append(dfl, s)
    torch.cuda.synchronize()                                  # rows 10..13 take positions 24..27: valid places
    assert int(s["st"]) == 0


def test_replayed_graph_and_another_stream(dfl):
    ns, ctxs = [17, 1, 5], [100, 250, 0]
    s = scene(dfl, "f32_to_bf16", 32, 8, 128, ns, ctxs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_append(dfl, s)
    side.synchronize()
    check_append(s, ns, ctxs)
    s["cos"], s["sin"] = tables(dfl, 128, 400)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_append(dfl, s)
    s["rows"].copy_(torch.randn(s["rows"].shape, generator=torch.Generator().manual_seed(9)).cuda())
    s["ctx"].add_(3)
    for pool in (s["kp"], s["vp"], s["qo"]):
        pool.fill_(9.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert int(s["st"]) == 0
    check_append(s, ns, [c + 3 for c in ctxs])


@pytest.mark.parametrize("types", TYPES, ids=list(TYPES))
@pytest.mark.parametrize("cu,ns", [([0, 6, 1 << 30], [6, 4]),       # claims more rows than there are: cut at the last
                                   ([0, 30, 10], [10, 0]),          # not ascending: sequence 0 takes all rows
                                   ([12, 14, 16], [0, 0])])         # behind the last row: nothing to do
def test_rows_of_offsets_that_disagree_are_written_to_their_places_alone(dfl, types, cu, ns):
    """The operands end with their last row; pages and the output's rows behind it keep what they hold."""
    s = scene(dfl, types, 8, 2, 128, [6, 4], [10, 20], extra=40)
    for part in ("q", "k", "v"):
        s[part] = s[part][:10]
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    run_append(dfl, s)
    torch.cuda.synchronize()
    assert int(s["st"]) == 0
    check_append(s, ns, [10, 20])


@pytest.mark.parametrize("types", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 17, 3000])
def test_parts_of_one_projection_in_place(dfl, types, T):
    """q and k inside the projection's own rows, a row's heads in one block or in several; the values beside them stay."""
    ti, to = TYPES[types]
    hq, hkv, dh = 10, 2, 128
    g = torch.Generator().manual_seed(T)
    heads = dfl.make_heads(1, hq, hkv, dh, rms_eps=EPS, dtype=out_code(dfl, to))
    rows = randn(g, (T, (hq + 2 * hkv) * dh), ti, 2.0)
    was = rows.clone()
    part = lambda r, a, n: r[:, a * dh:(a + n) * dh].view(T, n, dh)  # noqa: E731
    q, k = part(rows, 0, hq), part(rows, hq, hkv)
    gq, gk = randn(g, (dh,), to, 0.1, 1.0), randn(g, (dh,), to, 0.1, 1.0)
    pos = torch.randint(0, 4000, (T,), generator=g, dtype=torch.int32)
    cos, sin = tables(dfl, dh, 4000)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dfl.dflash_qk_norm_rope(heads, q, k, pos.cuda(), cos, sin, q, k, st, g_q=gq, g_k=gk)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert_rows(q, part(was, 0, hq), gq, pos.numpy(), "q")
    assert_rows(k, part(was, hq, hkv), gk, pos.numpy(), "k")
    assert torch.equal(part(rows, hq + hkv, hkv), part(was, hq + hkv, hkv))
