"""GPU: the pages' bookkeeping (dflash_pages_release / _fork / _reserve) against
a step-by-step simulation; tables, counts, lengths and copied rows are compared
bit for bit."""
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


class Book:
    def __init__(self, dfl, lens, n_pages, per, dtype=BF, L=2, hkv=2, dh=64, seed=0):
        self.dfl, self.lens = dfl, list(lens)
        order = np.random.default_rng(seed).permutation(n_pages).tolist()
        self.table = [[order.pop() if j * PAGE < n else -1 for j in range(per)] for n in lens]
        refs = np.zeros(n_pages, int)
        for row in self.table:
            for e in row:
                if e >= 0:
                    refs[e] += 1
        self.sim = tt.Pages(self.table, refs, self.lens)
        self.heads = dfl.make_heads(L, hkv, hkv, dh, dtype=dfl.BF16 if dtype == BF else dfl.F32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.randn((L, n_pages, hkv, PAGE, dh), generator=g, device="cuda").to(dtype) for _ in range(2))
        self.dtable, self.refs, self.ctx = ints(self.table), ints(refs.tolist()), ints(self.lens)
        self.view = dfl.KvPages(self.k, self.v, self.dtable)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def release(self, keep, **kw):
        self.dfl.dflash_pages_release(self.view, self.refs, ints(keep), self.st, **kw)
        self.sim.release(keep)

    def reserve(self, want, **kw):
        self.dfl.dflash_pages_reserve(self.view, self.refs, ints(want), self.st, **kw)
        self.sim.reserve(want)

    def fork(self, src, dst, **kw):
        self.sim.copies = []
        k, v = self.k.clone(), self.v.clone()
        self.dfl.dflash_pages_fork(self.heads, self.view, self.refs, self.ctx, ints(src), ints(dst), self.st, **kw)
        left_out = self.sim.fork(src, dst)
        for f, t, n in self.sim.copies:
            k[:, t, :, :n] = k[:, f, :, :n]
            v[:, t, :, :n] = v[:, f, :, :n]
        torch.cuda.synchronize()
        assert torch.equal(self.k, k) and torch.equal(self.v, v)
        return left_out

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.st) == status
        self.st.zero_()
        assert self.dtable.tolist() == self.sim.table
        assert self.refs.tolist() == self.sim.refs
        assert self.ctx.tolist() == self.sim.length
        # a count for every entry
        n = np.zeros(len(self.sim.refs), int)
        for row in self.sim.table:
            for e in row:
                n[e] += e >= 0
        assert n.tolist() == self.sim.refs


@pytest.mark.parametrize("B,per,n_pages", [(1, 1, 1), (3, 4, 20), (40, 9, 500), (700, 3, 9000), (4096, 2, 20000)])
def test_release_and_reserve(dfl, B, per, n_pages):
    r = np.random.default_rng(B)
    top = min(per, n_pages // B) * PAGE
    b = Book(dfl, r.integers(0, top + 1, B).tolist(), n_pages, per)
    for step in range(4):
        b.release([int(x * r.random()) for x in b.lens])
        b.check()
        b.lens = r.integers(0, top + 1, B).tolist()
        b.reserve(b.lens)
        b.check()
    b.release([-5] * B)
    b.check()
    assert not b.refs.any() and (b.dtable == -1).all()


def test_many_pages_for_one_sequence_in_several_rounds(dfl):
    b = Book(dfl, [0, 300, 0], 30000, 20000)
    b.reserve([19000 * PAGE, 500, 9000 * PAGE + 1])
    b.check()
    b.release([10000 * PAGE, 0, 0])
    b.check()
    b.reserve([10001 * PAGE, 4 * PAGE, 5])
    b.check()


def test_holes_are_filled_and_other_entries_stay(dfl):
    b = Book(dfl, [640, 640], 30, 8)
    for row, j in ((0, 1), (0, 3), (1, 0)):
        e = b.sim.table[row][j]
        b.sim.table[row][j] = -1
        b.sim.refs[e] -= 1
    b.sim.table[1][6] = -1
    b.dtable.copy_(ints(b.sim.table))
    b.refs.copy_(ints(b.sim.refs))
    b.reserve([600, 1000])
    b.check()


def test_pages_that_run_out(dfl):
    b = Book(dfl, [200, 100, 0], 8, 6)
    b.reserve([500, 300, 700])                      # 3 are held; 2 + 2 + 6 more are wanted, 5 are there
    assert b.sim.full
    b.check(dfl.ERR_CAPACITY)
    b.release([0, 300, 0])
    b.check()
    b.reserve([6 * PAGE + 1, 0, 0])                 # beyond the table
    b.check(dfl.ERR_CAPACITY)


def test_a_page_without_a_count_is_reported(dfl):
    b = Book(dfl, [200, 100], 8, 3)
    e = b.sim.table[0][0]
    b.refs[e] = 0
    b.dfl.dflash_pages_release(b.view, b.refs, ints([0, 100]), b.st)
    torch.cuda.synchronize()
    assert int(b.st) == dfl.ERR_INVALID_ARG and int(b.refs[e]) == 0 and (b.refs >= 0).all()


@pytest.mark.parametrize("dtype,L,hkv,dh", [(BF, 3, 8, 128), (BF, 2, 1, 64), (F32, 2, 2, 128), (F32, 5, 3, 64)])
def test_forks(dfl, dtype, L, hkv, dh):
    b = Book(dfl, [300, 128, 127, 1, 0, 513, 200, 640, 256, 5], 60, 6, dtype, L, hkv, dh)
    assert not b.fork([0, 0, 5], [9, 3, 6])
    b.check()
    assert not b.fork([0, 0, 5], [9, 3, 6])         # again: the targets' pages are given back first
    b.check()
    assert not b.fork([1, 4, 7, 2], [0, 5, 8, 9])   # whole pages, nothing, whole pages, less than one
    b.check()
    b.reserve([n + 70 for n in b.sim.length])
    b.check()
    assert not b.fork([0], [1])
    b.check()
    b.release([0] * 10)
    b.check()
    assert not b.refs.any()


def test_many_forks_of_one_sequence(dfl):
    B = 1024
    b = Book(dfl, [700] + [3] * (B - 1), 2 * B + 10, 7, L=1, hkv=1)
    assert not b.fork([0] * (B - 1), list(range(1, B)))
    b.check()
    assert max(b.sim.refs) == B


def test_pairs_that_cannot_be_are_left_out(dfl):
    for src, dst in [([0, 1], [2, 2]), ([0, 2], [2, 3]), ([1], [1]), ([0, 9], [3, 1]), ([-1, 0], [2, 3]), ([0], [4]), ([0, 1], [2, -7])]:
        b = Book(dfl, [300, 128, 127, 1], 20, 4)
        assert b.fork(src, dst)
        b.check(dfl.ERR_INVALID_ARG)
    b = Book(dfl, [300, 128, 127, 1], 20, 4)
    b.ctx[0], b.sim.length[0] = 4 * PAGE + 1, 4 * PAGE + 1
    assert b.fork([0, 1], [2, 3])
    b.check(dfl.ERR_INVALID_ARG)


def test_forks_without_a_page_leave_the_target_empty(dfl):
    b = Book(dfl, [300, 200, 127, 128], 7, 4)       # none is free but what the targets give back: one page each
    assert not b.fork([0, 1], [2, 3])
    b.check()
    b = Book(dfl, [300, 200, 0, 0], 6, 4)           # one is free
    assert not b.fork([0, 1], [2, 3])
    assert b.sim.length[3] == 0
    b.check(dfl.ERR_CAPACITY)
    b = Book(dfl, [300, 200, 5, 0], 16, 4)          # a source that lacks a page
    e = b.sim.table[0][1]
    b.sim.table[0][1], b.sim.refs[e] = -1, 0
    b.dtable.copy_(ints(b.sim.table))
    b.refs.copy_(ints(b.sim.refs))
    assert not b.fork([0, 1], [2, 3])
    assert b.sim.length[2] == 0
    b.check(dfl.ERR_CAPACITY)


def test_from_a_graph_and_traced(dfl):
    b = Book(dfl, [300, 128, 127, 1], 20, 4)
    keep, want, src, dst = ints([300, 128, 0, 1]), ints([400, 200, 300, 1]), ints([0]), ints([3])

    def cycle(**kw):
        dfl.dflash_pages_release(b.view, b.refs, keep, b.st, **kw)
        dfl.dflash_pages_fork(b.heads, b.view, b.refs, b.ctx, src, dst, b.st, **kw)
        dfl.dflash_pages_reserve(b.view, b.refs, want, b.st, **kw)

    def simulate():
        b.sim.release(keep.tolist())
        b.sim.fork(src.tolist(), dst.tolist())
        b.sim.reserve(want.tolist())

    cycle()
    simulate()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cycle()
    for _ in range(3):
        graph.replay()
        simulate()
        b.check()
    src[0], dst[0] = 1, 2
    graph.replay()
    simulate()
    b.check()
    rec = dfl.TraceRecorder(8)
    cycle(trace=rec.struct)
    assert [k for k, _, _, _ in rec.records()] == [dfl.K_PAGES] * 4
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    cycle(stream=side)
    simulate()
    simulate()
    b.check()
