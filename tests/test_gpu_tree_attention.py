"""GPU: masks and positions of drafted trees (dflash_tree_masks) and attention
under a mask over the chunk's own keys (dflash_attention_tree_paged) against the
float64 oracle. Tolerances as for chunk attention (tests/test_gpu_attention_chunk.py):
the arithmetic is the same, fewer keys are seen."""
import numpy as np
import pytest
import torch

from oracle import tree_ref as tt
from oracle.dflash_ref import f64
from tests.test_gpu_attention_chunk import BF, F32, LENS, SHAPES, Scene

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def tree(r, n, wide=3.0):
    return [-1] + [max(0, i - 1 - int(r.exponential(wide))) for i in range(1, n)]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("ns", [[1], [64], [5, 0, 33, 1, 200], [17] * 40, [0, 0, 3], [1000, 7]])
@pytest.mark.parametrize("more", [0, 2])
def test_masks_and_positions(dfl, ns, more):
    r = np.random.default_rng(sum(ns))
    trees = [tree(r, n) if n else [] for n in ns]
    if len(ns) > 2:
        trees[2] = [-1] * len(trees[2])                       # a forest
    T, W = sum(ns), (max(ns) + 31) // 32 + more
    cu, ctx = ints(np.cumsum([0] + ns).tolist()), ints([100 * i for i in range(len(ns))])
    mask = torch.full((T + 3, W), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((T + 3,), 77, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    par = ints([p for t in trees for p in t] + [5, 5, 5])     # rows behind the last sequence
    dfl.dflash_tree_masks(par, cu, ctx, mask, pos, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (mask[T:] == 77).all() and (pos[T:] == 77).all()
    at = 0
    for b, t in enumerate(trees):
        if not t:
            continue
        m = tt.sees(t)
        assert np.array_equal(mask[at:at + len(t)].cpu().numpy(), tt.bits(m, W)), b
        assert pos[at:at + len(t)].tolist() == (100 * b + m.sum(1) - 1).tolist()
        at += len(t)
    again = torch.full_like(mask, 77)
    dfl.dflash_tree_masks(par, cu, None, again, None, st)           # without positions
    torch.cuda.synchronize()
    assert torch.equal(again, mask)


def test_what_is_no_tree_is_reported(dfl):
    for parents, words, bad in [([-1, 0, 2], 1, True), ([-1, 5, 0], 1, True), ([0, 0], 1, True), ([-5, 0], 1, False),
                                ([-1] + list(range(39)), 1, True), ([-1] + list(range(31)), 1, False)]:
        n = len(parents)
        mask = torch.full((n, words), 77, dtype=torch.int32, device="cuda")
        pos, st = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        dfl.dflash_tree_masks(ints(parents), ints([0, n]), ints([7]), mask, pos, st)
        torch.cuda.synchronize()
        assert int(st) == (dfl.ERR_INVALID_ARG if bad else 0), parents
        t = [p if p < i else -1 for i, p in enumerate(parents)]
        m = tt.sees([max(p, -1) for p in t])
        assert np.array_equal(mask.cpu().numpy(), tt.bits(m, words))
        assert pos.tolist() == (7 + m.sum(1) - 1).tolist()


@pytest.mark.parametrize("ns", [[(7 * i) % 5 for i in range(700)], [1] * 513, [2500, 3, 5000, 0, 40], [3] * 520 + [2300, 1, 9]],
                         ids=["700", "513", "2500 and 5000 nodes", "a large one behind 520"])
def test_masks_of_many_sequences_and_of_large_ones(dfl, ns):
    """Offsets and parents that a block does not keep in shared memory."""
    r = np.random.default_rng(sum(ns))
    trees = [tree(r, n, 300.0 if n > 1000 else 3.0) if n else [] for n in ns]     # large ones: few generations
    T, W = sum(ns), (max(ns) + 31) // 32
    cu, ctx = ints(np.cumsum([0] + ns).tolist()), ints([3 * i for i in range(len(ns))])
    mask = torch.full((T + 2, W), 77, dtype=torch.int32, device="cuda")
    pos, st = torch.full((T + 2,), 77, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dfl.dflash_tree_masks(ints([p for t in trees for p in t]), cu, ctx, mask[:T], pos[:T], st)
    torch.cuda.synchronize()
    assert int(st) == 0 and (mask[T:] == 77).all() and (pos[T:] == 77).all()
    got, at, places = mask.cpu().numpy(), 0, pos.tolist()
    for b, t in enumerate(trees):
        if not t:
            continue
        m = tt.sees(t)
        assert np.array_equal(got[at:at + len(t)], tt.bits(m, W)), b
        assert places[at:at + len(t)] == (3 * b + m.sum(1) - 1).tolist()
        at += len(t)


# ------------------------------------------------------------------ attention
class TreeScene(Scene):
    def __init__(self, dfl, dtype, hq, hkv, dh, ns, ctxs, kind="tree", words=None, **kw):
        super().__init__(dfl, dtype, hq, hkv, dh, ns, ctxs, **kw)
        r = np.random.default_rng(sum(ns) + len(kind))
        W = words or max((max(ns) + 31) // 32, 1)
        self.sees, rows = [], []
        for n in ns:
            if kind == "tree":
                m = tt.sees(tree(r, n)) if n else np.zeros((0, 0), bool)
            elif kind == "random":                            # any bits, some rows without any
                m = r.random((n, n)) < r.choice([0.0, 0.1, 0.5, 1.0], (n, 1))
            else:
                m = np.tril(np.ones((n, n), bool)) if kind == "causal" else np.zeros((n, n), bool)
            w = tt.bits(m, W)
            m = m.copy()
            m[:, W * 32:] = False                             # keys that the mask does not reach
            if kind != "tree" and n % 32 and n < W * 32:      # bits behind the sequence's rows are not looked at
                w[:, n // 32] |= np.array(-1 << (n % 32)).astype(np.int32)
                w[:, n // 32 + 1:] = -1
            self.sees.append(m)
            rows.append(w)
        pad = self.q.shape[0] - self.T
        self.mask = torch.from_numpy(np.concatenate(rows + [np.full((pad, W), -1, np.int32)])).cuda()

    def run(self, scale=0.0, max_rows=None, hint=None, ws=None, **kw):
        self.dfl.dflash_attention_tree_paged(
            self.heads, self.q, self.cu, self.ctx, max(self.ns) if max_rows is None else max_rows,
            max(max(self.ctxs), 0) if hint is None else hint, self.layer, self.pages, self.mask, self.out, self.st, ws or self.ws,
            scale=scale, **kw)

    def check(self, scale=0.0, rows=None):
        torch.cuda.synchronize()
        assert int(self.st) == 0
        dh, first = self.q.shape[2], 0
        for b, (n, c) in enumerate(zip(self.ns, self.ctxs)):
            pick = np.arange(n) if rows is None or n <= rows else np.unique(np.linspace(0, n - 1, rows).astype(int))
            k, v = f64(self.k[b]), f64(self.v[b])
            for i in pick:
                want, mass, big = tt.attention(f64(self.q[first + i:first + i + 1]), k, v, c, self.sees[b][i:i + 1], scale)
                got = f64(self.out[first + i:first + i + 1])
                d = (dh + 8) * 2.0 ** -24 * big[..., None] + 2.0 ** -21
                tol = 2 * (d + min(max(c + n, 0), 4096) * 2.0 ** -24) * mass
                if self.dtype == BF:
                    tol = tol + 2.0 ** -8 * (mass + np.abs(want))
                err = np.abs(got - want)
                assert (err <= tol).all(), (b, int(i), n, c, float(err.max()), float((err / np.maximum(tol, 1e-30)).max()))
            first += n
        assert (self.obuf[self.T:] == 9).all() and (self.obuf[:, -1] == 9).all()


@pytest.mark.parametrize("kind", ["tree", "random"])
@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
@pytest.mark.parametrize("shape", SHAPES, ids=list(SHAPES))
def test_matches_the_oracle(dfl, shape, lens, kind):
    ns, ctxs = LENS[lens]
    s = TreeScene(dfl, *SHAPES[shape], ns, ctxs, kind, seed=len(lens))
    s.run()
    s.check(rows=24)


@pytest.mark.parametrize("shape", ["qwen", "mha64", "f32_128"])
@pytest.mark.parametrize("ctx", [0, 1, 31, 63, 64, 96, 127, 128, 129, 255, 256])
def test_trees_at_every_place_of_a_page(dfl, shape, ctx):
    """Windows of the mask begin at any bit, trees end in the next page or the one after."""
    s = TreeScene(dfl, *SHAPES[shape], [64, 130, 17], [ctx, ctx + 3, ctx + 14], "random", seed=ctx)
    s.run()
    s.check(rows=16)


@pytest.mark.parametrize("shape", ["qwen", "g7", "f32_64"])
@pytest.mark.parametrize("ns,ctxs", [([64], [9000]), ([33, 1], [5000, 14]), ([40] * 9, [700 * i for i in range(9)]), ([256], [3000])])
def test_long_contexts_split_over_the_gpu(dfl, shape, ns, ctxs):
    s = TreeScene(dfl, *SHAPES[shape], ns, ctxs, seed=11)
    s.run()
    s.check(rows=8)


@pytest.mark.parametrize("shape", ["qwen", "g5_64", "f32_64"])
def test_a_chain_is_causal_attention_and_rows_may_see_nothing(dfl, shape):
    s = TreeScene(dfl, *SHAPES[shape], [17, 140, 3], [300, 0, 127], "causal", seed=13)
    s.run()
    s.check(rows=10)
    s = TreeScene(dfl, *SHAPES[shape], [6, 200, 2], [0, 0, 5], "nothing", seed=14)
    s.run()
    s.check(rows=10)
    assert not s.out[:206].any() and s.out[206:208].any()


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_masks_of_fewer_words_than_nodes_and_of_more(dfl, shape):
    for words in (1, 2, 9):
        s = TreeScene(dfl, *SHAPES[shape], [70, 33, 8], [200, 0, 90], "random", words=words, seed=17)
        s.run()
        s.check(rows=12)


@pytest.mark.parametrize("shape", ["qwen", "f32_128"])
def test_hints_scales_and_negative_contexts(dfl, shape):
    s = TreeScene(dfl, *SHAPES[shape], [17, 64, 1], [2000, 10, 333], seed=19)
    for max_rows, hint in [(0, 0), (1, 1 << 30), (1 << 30, 5)]:
        s.out[:s.T].fill_(0.0)
        s.run(max_rows=max_rows, hint=hint)
        s.check(rows=8)
    s.run(scale=0.3)
    s.check(scale=float(np.float32(0.3)), rows=8)
    s = TreeScene(dfl, *SHAPES[shape], [9, 40], [-3, -35], "random", seed=20)
    s.run()
    s.check()


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_the_same_bits_every_time_and_from_a_graph(dfl, shape):
    s = TreeScene(dfl, *SHAPES[shape], [64, 30, 1, 0], [3000, 100, 5000, 0], seed=29)
    s.run()
    s.check(rows=6)
    want = s.obuf.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for fill in (255, 0):
        s.out[:s.T].zero_()
        s.ws.buf.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.obuf, want)
    # another tree at the next replay
    t = TreeScene(dfl, *SHAPES[shape], s.ns, s.ctxs, "random", seed=29)
    s.mask.copy_(t.mask)
    s.sees = t.sees
    graph.replay()
    s.check(rows=6)


def test_two_calls_at_once_on_their_own_workspaces(dfl):
    a = TreeScene(dfl, *SHAPES["qwen"], [64], [8000], seed=31)
    b = TreeScene(dfl, *SHAPES["qwen"], [200, 1], [500, 7000], seed=32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run()
        with torch.cuda.stream(side):
            b.run()
    torch.cuda.synchronize()
    a.check(rows=4)
    b.check(rows=4)


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_bad_pages_and_padded_batches(dfl, shape):
    s = TreeScene(dfl, *SHAPES[shape], [17, 4], [300, 50], seed=33, garbage=0.5)
    s.table[0, 1] = -1
    s.pages = dfl.KvPages(s.kp, s.vp, s.table.cuda())
    s.run()
    torch.cuda.synchronize()
    assert int(s.st) == dfl.ERR_CAPACITY
    s = TreeScene(dfl, *SHAPES[shape], [17, 3], [300, 40], seed=57, extra=130)
    s.qbuf[s.T::2] = float("nan")
    s.qbuf[s.T + 1::2] = float("inf")
    s.run()
    s.check(rows=6)


def test_a_step_without_nodes(dfl):
    heads, none = dfl.make_heads(1, 8, 2, 128), torch.zeros((0, 8, 128), dtype=BF, device="cuda")
    pool, st = torch.zeros((1, 3, 2, 128, 128), dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mask = torch.zeros((0, 0), dtype=torch.int32, device="cuda")
    dfl.dflash_tree_masks(ints([]), ints([0, 0]), ints([5]), mask, ints([]), st)
    dfl.dflash_attention_tree_paged(heads, none, ints([0, 0]), ints([5]), 0, 5, 0, dfl.KvPages(pool, pool.clone(), ints([[0, 1]])), mask,
                                    none.clone(), st, dfl.ChunkWorkspace(heads))
    torch.cuda.synchronize()
    assert int(st) == 0
