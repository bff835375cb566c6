"""GPU: the confirmed branch of drafted trees and the move of its rows in a paged
cache (dflash_verify_tree). Whole numbers and moved rows are compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import tree_ref as tt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
PAGE = 128


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Trees:
    def __init__(self, ns, seed=0, wide=2.0, hit=0.8, twins=False):
        r = np.random.default_rng(seed)
        self.ns = ns
        self.parents = [[-1] + [max(0, i - 1 - int(r.exponential(wide))) for i in range(1, n)] if n else [] for n in ns]
        self.tokens, self.drawn = [], []
        for p in self.parents:
            t = r.integers(0, 3 if twins else 100000, len(p)).tolist()      # twins: siblings with the same token
            kids = [[c for c in range(len(p)) if p[c] == i] for i in range(len(p))]
            self.drawn.append([t[int(r.choice(k))] if k and r.random() < hit else 200000 + i for i, k in enumerate(kids)])
            self.tokens.append(t)

    def dev(self, extra=2):
        flat = lambda v: ints([x for y in v for x in y] + [0] * extra)  # noqa: E731
        return flat(self.tokens), flat(self.parents), flat(self.drawn), ints(np.cumsum([0] + self.ns).tolist())


def outs(B, P):
    one = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    return one(B + 1), one(B + 1, P), one(B + 1, P), one(B + 1)


def same(t, got, P):
    tau, com, path, nxt = (x.cpu().numpy() for x in got)
    for b in range(len(t.ns)):
        want = tt.verify_tree(t.tokens[b], t.parents[b], t.drawn[b], P)
        assert (tau[b], com[b].tolist(), path[b].tolist(), nxt[b]) == want, b
    assert all((x[-1] == -9).all() for x in (tau, com, path, nxt))
    return [tt.verify_tree(t.tokens[b], t.parents[b], t.drawn[b], P)[2] for b in range(len(t.ns))]


@pytest.mark.parametrize("P", [1, 3, 24, 1500])
@pytest.mark.parametrize("ns", [[1], [64], [0], [17, 0, 200, 1, 64], [5] * 300, [1024, 3]])
def test_branches(dfl, ns, P):
    for seed, twins in ((1, False), (2, True)):
        t = Trees(ns, seed, hit=0.95, twins=twins)
        got, st = outs(len(ns), P), torch.zeros(1, dtype=torch.int32, device="cuda")
        dfl.dflash_verify_tree(*t.dev(), *got, st)
        torch.cuda.synchronize()
        assert int(st) == 0
        same(t, got, P)


class Cache:
    def __init__(self, dfl, dtype, L, hkv, dh, ctxs, ns, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads = dfl.make_heads(L, hkv, hkv, dh, dtype=dfl.BF16 if dtype == BF else dfl.F32)
        have = [(max(c + n, 0) + PAGE - 1) // PAGE for c, n in zip(ctxs, ns)]
        n_pages = sum(have) + 2
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = [[order.pop() for _ in range(h)] + [-1] * (max(have) + 1 - h) for h in have]
        self.k = torch.randn((L, n_pages, hkv, PAGE, dh), generator=g, device="cuda").to(dtype)
        self.v = torch.randn((L, n_pages, hkv, PAGE, dh), generator=g, device="cuda").to(dtype)
        self.view = dfl.KvPages(self.k, self.v, ints(self.table))
        self.ctxs, self.ctx = ctxs, ints(ctxs)

    def moved(self, paths):
        """What the pools have to hold afterwards."""
        k, v = self.k.clone(), self.v.clone()
        for b, path in enumerate(paths):
            for j, i in enumerate(path):
                if i >= 0 and i != j:
                    f, t = self.ctxs[b] + i, self.ctxs[b] + j
                    for mine, was in ((k, self.k), (v, self.v)):
                        mine[:, self.table[b][t // PAGE], :, t % PAGE] = was[:, self.table[b][f // PAGE], :, f % PAGE]
        return k, v


@pytest.mark.parametrize("dtype,L,hkv,dh", [(BF, 3, 8, 128), (BF, 2, 1, 64), (F32, 2, 2, 128), (F32, 5, 4, 64), (BF, 40, 8, 128)])
@pytest.mark.parametrize("ns,ctxs", [([64], [300]), ([1], [5]), ([17, 64, 2, 0, 200], [0, 100, 127, 5, 250]), ([40] * 30, [7 * i for i in range(30)])])
def test_rows_move_behind_the_context(dfl, dtype, L, hkv, dh, ns, ctxs):
    for wide in (0.3, 6.0):                       # long branches, whose rows overlap, and short ones
        t = Trees(ns, 3, wide=wide, hit=0.97)
        c = Cache(dfl, dtype, L, hkv, dh, ctxs, ns, 5)
        P = 200
        got, st = outs(len(ns), P), torch.zeros(1, dtype=torch.int32, device="cuda")
        paths = [tt.verify_tree(t.tokens[b], t.parents[b], t.drawn[b], P)[2] for b in range(len(ns))]
        k, v = c.moved(paths)
        dfl.dflash_verify_tree(*t.dev(), *got, st, heads=c.heads, ctx_len=c.ctx, pages=c.view)
        torch.cuda.synchronize()
        assert int(st) == 0
        same(t, got, P)
        assert torch.equal(c.k, k) and torch.equal(c.v, v)
    assert any(sum(i >= 0 for i in p) > 1 for p in paths) or max(ns) == 1


def test_a_long_branch_moves_by_one(dfl):
    """Every row's source is the target of the next one."""
    n = 1000
    t = Trees([n], 1)
    t.parents[0] = [-1, 0, 0] + list(range(2, n - 1))
    t.tokens[0] = list(range(n))
    t.drawn[0] = [2] + [0] + list(range(3, n)) + [7]
    c = Cache(dfl, BF, 2, 2, 64, [77], [n], 9)
    got, st = outs(1, n), torch.zeros(1, dtype=torch.int32, device="cuda")
    path = tt.verify_tree(t.tokens[0], t.parents[0], t.drawn[0], n)[2]
    assert path[:4] == [0, 2, 3, 4] and path[n - 2] == n - 1
    k, v = c.moved([path])
    dfl.dflash_verify_tree(*t.dev(0), *got, st, heads=c.heads, ctx_len=c.ctx, pages=c.view)
    torch.cuda.synchronize()
    same(t, got, n)
    assert int(st) == 0 and torch.equal(c.k, k) and torch.equal(c.v, v)


def test_what_does_not_fit_is_reported(dfl):
    B, P = 2, 8
    for what in ("parent", "root", "many", "page", "table"):
        ns = [1100 if what == "many" else 20, 12]
        t = Trees(ns, 11, wide=0.2, hit=1.0)
        c = Cache(dfl, BF, 2, 2, 64, [100, 120], ns, 13)
        if what == "parent":
            t.parents[0][5] = 9                      # its own branch is cut there
        if what == "root":
            t.parents[0][0] = 3
        if what == "page":
            t.parents[0], t.drawn[0] = [-1, 0, 0] + list(range(2, 19)), t.tokens[0][2:3] + [0] + t.tokens[0][3:] + [1]
            c.ctxs[0] = 122
            c.ctx[0] = 122
            c.table[0][1] = -1
            c.view = dfl.KvPages(c.k, c.v, ints(c.table))
        if what == "table":
            t.parents[0], t.drawn[0] = [-1, 0, 0] + list(range(2, 19)), t.tokens[0][2:3] + [0] + t.tokens[0][3:] + [1]
            c.ctx[0] = 10 ** 6
        got, st = outs(B, P), torch.zeros(1, dtype=torch.int32, device="cuda")
        want = tt.verify_tree(t.tokens[1], t.parents[1], t.drawn[1], P)
        dfl.dflash_verify_tree(*t.dev(), *got, st, heads=c.heads, ctx_len=c.ctx, pages=c.view)
        torch.cuda.synchronize()
        assert int(st) == (dfl.ERR_CAPACITY if what in ("page", "table") else dfl.ERR_INVALID_ARG), what
        assert (int(got[0][1]), got[1][1].tolist(), got[2][1].tolist(), int(got[3][1])) == want       # the other is right
        if what in ("root", "many"):
            assert int(got[0][0]) == 0 and (got[1][0] == -1).all() and (got[2][0] == -1).all() and int(got[3][0]) == -1
        if what == "parent":
            t.parents[0][5] = 10 ** 6
            assert got[2][0].tolist() == tt.verify_tree(t.tokens[0], t.parents[0], t.drawn[0], P)[2]


def test_offsets_that_disagree_stay_inside_the_rows(dfl):
    t = Trees([20, 12], 15)
    tok, par, drawn, cu = t.dev(0)
    for bad in ([0, 20, 1 << 30], [-5, 20, 32], [0, 40, 10], [40, 50, 60]):
        got, st = outs(2, 8), torch.zeros(1, dtype=torch.int32, device="cuda")
        dfl.dflash_verify_tree(tok, par, drawn, ints(bad), *got, st)
        torch.cuda.synchronize()
        assert (got[0][:2] >= 0).all() and (got[0][:2] <= 8).all()


def test_from_a_graph_and_another_stream(dfl):
    ns, P = [64, 20], 24
    t = Trees(ns, 17, hit=0.95)
    args, got, st = t.dev(), outs(2, P), torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    dfl.dflash_verify_tree(*args, *got, st)
    with torch.cuda.graph(graph):
        dfl.dflash_verify_tree(*args, *got, st)
    u = Trees(ns, 19, hit=0.95)
    for a, b in zip(args, u.dev()):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    same(u, got, P)
    side = torch.cuda.Stream()
    got = outs(2, P)
    torch.cuda.synchronize()
    dfl.dflash_verify_tree(*args, *got, st, stream=side)
    torch.cuda.synchronize()
    same(u, got, P)
    rec = dfl.TraceRecorder(2)
    dfl.dflash_verify_tree(*args, *got, st, trace=rec.struct)
    assert [k for k, _, _, _ in rec.records()] == [dfl.K_VERIFY]
