"""GPU: attention of ragged chunks of new tokens over a paged cache
(dflash_attention_chunk_paged) against the float64 oracle.

Bound of one output. With s the scaled scores, p the softmax weights and
A = sum p |v|: a score is off by at most (Dh + 8) 2^-24 sum |q_d k_d| scale
(Dh products of exact inputs and sums in fp32, the scaling, the shift by the
maximum), its exponential by 2^-21 more (approximate exp2, and the fp32 shift's
own rounding of values up to 2^3 of rescaling); weights below 2^-8 of the
sum's rounding cannot matter. Call this d. Numerator and denominator are each
off by d and by the sums' n 2^-24 (n keys at most, taken as min(n, 4096) as the
tiles are summed apart): the quotient by 2 (d + n 2^-24) A. bf16 weights add
2^-8 A (half a step each), a bf16 output 2^-8 |out|."""
import numpy as np
import pytest
import torch

from oracle import target_ref as tr
from oracle.dflash_ref import f64

pytestmark = pytest.mark.gpu

PAGE = 128
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


class Scene:
    def __init__(self, dfl, dtype, hq, hkv, dh, ns, ctxs, seed=0, n_layers=2, layer=1, extra=2, spread=1.5, garbage=float("nan"),
                 spare_pages=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dfl, self.ns, self.ctxs, self.layer, self.dtype = dfl, ns, ctxs, layer, dtype
        self.heads = dfl.make_heads(n_layers, hq, hkv, dh, dtype=dfl.BF16 if dtype == BF else dfl.F32)
        T, B = sum(ns), len(ns)
        self.T = T
        # rows of a wider buffer: strided, and rows behind the last sequence
        self.qbuf = (torch.randn((T + extra, hq + 2, dh), generator=g, device="cuda") * spread).to(dtype)
        self.q = self.qbuf[:, 1:1 + hq]
        need = [max(c + n, 0) for c, n in zip(ctxs, ns)]
        per = max(max(need) // PAGE + 1, 1)
        n_pages = sum((x + PAGE - 1) // PAGE for x in need) + spare_pages
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((B, per), -1, dtype=torch.int32)
        self.kp = torch.full((n_layers, n_pages, hkv, PAGE, dh), garbage, dtype=dtype, device="cuda")
        self.vp = torch.full((n_layers, n_pages, hkv, PAGE, dh), garbage, dtype=dtype, device="cuda")
        self.k, self.v = [], []
        for b in range(B):
            k = torch.randn((hkv, need[b], dh), generator=g, device="cuda").to(dtype)
            v = torch.randn((hkv, need[b], dh), generator=g, device="cuda").to(dtype)
            for i in range((need[b] + PAGE - 1) // PAGE):
                pg = order.pop()
                self.table[b, i] = pg
                n = min(PAGE, need[b] - i * PAGE)
                self.kp[layer, pg, :, :n] = k[:, i * PAGE:i * PAGE + n]
                self.vp[layer, pg, :, :n] = v[:, i * PAGE:i * PAGE + n]
            self.k.append(k)
            self.v.append(v)
        self.pages = dfl.KvPages(self.kp, self.vp, self.table.cuda())
        self.cu = torch.tensor([sum(ns[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        self.ctx = torch.tensor(ctxs, dtype=torch.int32, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = dfl.ChunkWorkspace(self.heads)
        self.ws.buf.fill_(255)                    # NaN everywhere: scratch is not read before it is written
        self.obuf = torch.full((T + extra, hq + 1, dh), 9.0, dtype=dtype, device="cuda")
        self.out = self.obuf[:, :hq]

    def run(self, causal=True, scale=0.0, max_rows=None, hint=None, ws=None, out=None, **kw):
        self.dfl.dflash_attention_chunk_paged(
            self.heads, self.q, self.cu, self.ctx, max(self.ns) if max_rows is None else max_rows,
            max(max(self.ctxs), 0) if hint is None else hint, self.layer, self.pages, self.out if out is None else out, self.st,
            ws or self.ws, causal=causal, scale=scale, **kw)

    def check(self, causal=True, scale=0.0, rows=None, out=None):
        """Every row against the oracle (rows: at most that many of each sequence, the first and last among them)."""
        torch.cuda.synchronize()
        assert int(self.st) == 0
        got_all = self.out if out is None else out
        dh, first = self.q.shape[2], 0
        for b, (n, c) in enumerate(zip(self.ns, self.ctxs)):
            pick = np.arange(n) if rows is None or n <= rows else np.unique(np.linspace(0, n - 1, rows).astype(int))
            k, v = f64(self.k[b]), f64(self.v[b])
            for i in pick:
                q = f64(self.q[first + i:first + i + 1])
                end = c + int(i) + 1 if causal else c + n
                want, mass, big = tr.chunk_attention(q, k[:, :max(end, 0)], v[:, :max(end, 0)], max(end, 0) - 1, True, scale) \
                    if end > 0 else (np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2]))
                got = f64(got_all[first + i:first + i + 1])
                d = (dh + 8) * 2.0 ** -24 * big[..., None] + 2.0 ** -21
                tol = 2 * (d + min(max(end, 0), 4096) * 2.0 ** -24) * mass
                if self.dtype == BF:
                    tol = tol + 2.0 ** -8 * (mass + np.abs(want))
                err = np.abs(got - want)
                assert (err <= tol).all(), (b, int(i), n, c, float(err.max()), float((err / np.maximum(tol, 1e-30)).max()))
            first += n
        assert (self.obuf[self.T:] == 9).all() and (self.obuf[:, -1] == 9).all()


SHAPES = {"qwen": (BF, 32, 8, 128), "mha64": (BF, 4, 4, 64), "g7": (BF, 7, 1, 128), "g5_64": (BF, 10, 2, 64), "g16_64": (BF, 16, 1, 64),
          "g64": (BF, 64, 1, 128), "f32_64": (F32, 4, 4, 64), "f32_128": (F32, 8, 2, 128), "f32_g7": (F32, 7, 1, 64)}
LENS = {"one": ([1], [0]), "decode": ([1] * 5, [0, 126, 127, 128, 700]), "block": ([17, 17, 17], [300, 0, 111]),
        "ragged": ([1, 0, 33, 130, 17, 2], [500, 77, 0, 129, 255, 126]), "chunk": ([300], [0]), "chunk_ctx": ([257, 3], [250, 1000]),
        "page_end": ([128, 1, 127], [0, 255, 1])}


@pytest.mark.parametrize("lens", LENS, ids=list(LENS))
@pytest.mark.parametrize("shape", SHAPES, ids=list(SHAPES))
def test_matches_the_oracle(dfl, shape, lens):
    ns, ctxs = LENS[lens]
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=len(lens))
    s.run()
    s.check(rows=24)


@pytest.mark.parametrize("shape", ["qwen", "g5_64", "f32_64"])
@pytest.mark.parametrize("ns,ctxs", [([17, 5], [300, 0]), ([1, 200], [129, 60])])
def test_every_row_sees_the_whole_block_when_not_causal(dfl, shape, ns, ctxs):
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=7)
    s.run(causal=False)
    s.check(causal=False, rows=20)


@pytest.mark.parametrize("shape", ["qwen", "mha64", "f32_128"])
@pytest.mark.parametrize("ns,ctxs", [([17], [9000]), ([1], [20000]), ([3, 1], [5000, 14]), ([300], [6000])])
def test_long_contexts_split_over_the_gpu(dfl, shape, ns, ctxs):
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=11)
    s.run()
    s.check(rows=8)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv", [(28, 4), (8, 2), (64, 1), (3, 3)])
@pytest.mark.parametrize("ns,ctxs", [([64, 17, 64], [700, 0, 333]), ([1, 200, 0, 131], [64, 1000, 5, 127])])
def test_fp32_chunks_of_many_rows(dfl, causal, hq, hkv, ns, ctxs):
    """Units of 64 and of 128 rows, in one part and in several, whichever the sizes call for."""
    s = Scene(dfl, F32, hq, hkv, 128, ns, ctxs, seed=29)
    s.run(causal=causal)
    s.check(causal=causal, rows=12)


@pytest.mark.parametrize("B,hq,hkv", [(47, 8, 2), (300, 4, 4)])
def test_fp32_units_of_many_sequences_in_parts(dfl, B, hq, hkv):
    """More split units than CTAs, and more units than can be split."""
    ns = [9 + (5 * i) % 9 for i in range(B)]
    ctxs = [640 + (37 * i) % 90 if B < 100 else (91 * i) % 300 for i in range(B)]
    s = Scene(dfl, F32, hq, hkv, 64, ns, ctxs, seed=31)
    s.run()
    s.check(rows=3)


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_hints_do_not_change_what_is_computed(dfl, shape):
    """Any hint is allowed: too small ones, too large ones."""
    s = Scene(dfl, *SHAPES[shape], [17, 140, 1], [2000, 10, 333], seed=13)
    for max_rows, hint in [(0, 0), (1, 1), (1, 1 << 30), (1 << 30, 5), (140, 2000)]:
        s.out[:s.T].fill_(0.0)
        s.run(max_rows=max_rows, hint=hint)
        s.check(rows=8)


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_many_sequences(dfl, shape):
    ns = [(3 * i) % 5 for i in range(200)]
    ctxs = [(37 * i) % 400 for i in range(200)]
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=17)
    s.run()
    s.check(rows=2)


@pytest.mark.parametrize("shape", ["qwen", "g16_64"])
def test_a_prompt_chunk_next_to_single_tokens(dfl, shape):
    ns = [700] + [1] * 12 + [64, 65]
    ctxs = [100] + [150 * i for i in range(12)] + [0, 500]
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=19)
    s.run()
    s.check(rows=12)


@pytest.mark.parametrize("shape", ["qwen", "f32_128"])
def test_peaked_flat_and_shifted_scores(dfl, shape):
    dt, hq, hkv, dh = SHAPES[shape]
    s = Scene(dfl, dt, hq, hkv, dh, [17, 1], [600, 400], seed=23, spread=12.0)          # near one-hot rows
    s.run()
    s.check()
    s = Scene(dfl, dt, hq, hkv, dh, [17], [600], seed=24, spread=0.0)                   # a plain mean
    s.run()
    s.check()
    s = Scene(dfl, dt, hq, hkv, dh, [17], [600], seed=25)
    s.run(scale=0.3)
    s.check(scale=float(np.float32(0.3)))
    # a maximum that rises tile after tile: every tile rescales what was summed before
    s = Scene(dfl, dt, hq, hkv, dh, [9], [900], seed=26)
    ramp = torch.linspace(-4.0, 4.0, 909, device="cuda")
    s.k[0] = (s.k[0] * 0.1 + ramp[None, :, None]).to(dt)
    for i in range(8):
        n = min(PAGE, 909 - i * PAGE)
        s.kp[1, int(s.table[0, i]), :, :n] = s.k[0][:, i * PAGE:i * PAGE + n]
    s.qbuf.abs_()
    s.run()
    s.check()


def test_a_row_without_keys_gives_zeros(dfl):
    for shape in ("qwen", "f32_64"):
        s = Scene(dfl, *SHAPES[shape], [6, 2], [-3, 5], seed=27)
        s.run(hint=5)
        s.check()
        assert not s.out[:3].any()


def test_the_same_bits_every_time_and_from_a_graph(dfl):
    s = Scene(dfl, *SHAPES["qwen"], [17, 300, 1, 1], [3000, 100, 9000, 0], seed=29)
    s.run()
    torch.cuda.synchronize()
    want = s.obuf.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(4):
        s.out[:s.T].zero_()
        s.ws.buf.fill_(255 if i % 2 else 0)
        if i < 2:
            s.run()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.obuf, want)
    # a replay takes the lengths that the device holds then
    s.ns, s.ctxs = [10, 200, 5, 104], [20, 300, 8990, 0]
    s.cu.copy_(torch.tensor([0, 10, 210, 215, 319], dtype=torch.int32))
    s.ctx.copy_(torch.tensor(s.ctxs, dtype=torch.int32))
    s2 = Scene(dfl, *SHAPES["qwen"], s.ns, s.ctxs, seed=30)
    for mine, other in ((s.qbuf, s2.qbuf),):
        mine.copy_(other)
    # its own pages: the second scene's table and pools are copied over the first's where they fit
    n = min(s.kp.shape[1], s2.kp.shape[1])
    assert int(s2.table.max()) < s.kp.shape[1] and s2.table.shape[1] <= s.table.shape[1]
    s.kp[:, :n].copy_(s2.kp[:, :n])
    s.vp[:, :n].copy_(s2.vp[:, :n])
    full = torch.full_like(s.table, -1)
    full[:, :s2.table.shape[1]] = s2.table
    s.pages._keep[2].copy_(full.cuda())
    s.k, s.v = s2.k, s2.v
    graph.replay()
    s.check(rows=6)


@pytest.mark.parametrize("shape,ns,ctxs", [("qwen", [17, 64, 1, 0], [200, 60, 0, 9]), ("qwen", [300], [90]),
                                           ("f32_128", [64, 17, 3], [900, 0, 333]), ("f32_64", [1, 1], [1900, 7])])
def test_whole_units_and_fp32_give_the_same_bits_from_a_graph(dfl, shape, ns, ctxs):
    """Whatever the workspace holds, in one launch or two."""
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=37)
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


def test_two_calls_at_once_on_their_own_workspaces(dfl):
    a = Scene(dfl, *SHAPES["qwen"], [17], [8000], seed=31)
    b = Scene(dfl, *SHAPES["qwen"], [200, 1], [500, 7000], seed=32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run()
        with torch.cuda.stream(side):
            b.run()
    torch.cuda.synchronize()
    a.check(rows=4)
    b.check(rows=4)


def test_bad_pages_are_capacity_errors(dfl):
    for shape in ("qwen", "f32_64"):
        for bad in (-1, 10 ** 6):
            s = Scene(dfl, *SHAPES[shape], [17, 4], [300, 50], seed=33, garbage=0.5)
            s.table[0, 1] = bad
            s.pages = dfl.KvPages(s.kp, s.vp, s.table.cuda())
            s.run()
            torch.cuda.synchronize()
            assert int(s.st) == dfl.ERR_CAPACITY
            for i in range(4):                     # the other sequence is right
                o, mass, _ = tr.chunk_attention(f64(s.q[17 + i:18 + i]), f64(s.k[1])[:, :51 + i], f64(s.v[1])[:, :51 + i], 50 + i)
                # 2 d A with sum |q k| scale below 64, as above, and bf16's two roundings
                assert (np.abs(f64(s.out[17 + i:18 + i]) - o) <= 2.0 ** -8 * (mass + np.abs(o)) + 2.0 ** -9 * mass).all()
        t = Scene(dfl, *SHAPES[shape], [17], [100], seed=34, garbage=0.5)
        t.ctx[0] = 300                             # 317 keys in a table of one page
        t.run()
        torch.cuda.synchronize()
        assert int(t.st) == dfl.ERR_CAPACITY


def test_row_offsets_that_disagree_with_the_rows_stay_inside_them(dfl):
    s = Scene(dfl, *SHAPES["qwen"], [17, 4], [100, 50], seed=35, garbage=0.5)
    s.cu.copy_(torch.tensor([0, 17, 1 << 30], dtype=torch.int32))
    s.run()
    torch.cuda.synchronize()
    s.cu.copy_(torch.tensor([0, 30, 10], dtype=torch.int32))      # not ascending
    s.run()
    torch.cuda.synchronize()
    assert int(s.st) in (0, dfl.ERR_CAPACITY)


def test_pools_past_32_bits_of_elements(dfl):
    """The layer's pages start beyond 2^32 bytes and 2^31 elements of the pool."""
    hkv, dh = 8, 128
    n_pages = 9000
    n_layers = 3                                                   # 3 * 9000 * 8 * 128 * 128 = 3.5e9 elements
    s = Scene(dfl, BF, 32, hkv, dh, [17, 1], [500, 200], seed=36, n_layers=1, layer=0)
    kp = torch.empty((n_layers, n_pages, hkv, PAGE, dh), dtype=BF, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.full_like(s.table, -1)
    at = n_pages - 1
    for b in range(2):
        for i in range(s.table.shape[1]):
            if int(s.table[b, i]) >= 0:
                kp[2, at].copy_(s.kp[0, int(s.table[b, i])])
                vp[2, at].copy_(s.vp[0, int(s.table[b, i])])
                table[b, i] = at
                at -= 1
    s.heads = dfl.make_heads(n_layers, 32, hkv, dh)
    s.layer, s.pages = 2, dfl.KvPages(kp, vp, table.cuda())
    s.run()
    s.check(rows=6)


def test_empty_batches(dfl):
    s = Scene(dfl, *SHAPES["qwen"], [0, 0], [10, 0], seed=37)
    s.run()
    torch.cuda.synchronize()
    assert (s.obuf == 9).all() and int(s.st) == 0


def test_more_sequences_than_threads(dfl):
    ns = [(3 * i) % 4 for i in range(900)]
    ctxs = [(53 * i) % 300 for i in range(900)]
    s = Scene(dfl, *SHAPES["mha64"], ns, ctxs, seed=41)
    s.run()
    s.check(rows=1)


@pytest.mark.parametrize("shape", ["g64", "g16_64"])
def test_many_units_of_one_sequence(dfl, shape):
    """Units of few tokens: hundreds of them in one sequence, found by threads that share it."""
    s = Scene(dfl, *SHAPES[shape], [1500, 1], [70, 3], seed=43)
    s.run()
    s.check(rows=12)


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_sequences_that_share_a_prefix(dfl, shape):
    """Two sequences' tables name the same pages for their common context."""
    s = Scene(dfl, *SHAPES[shape], [5, 9], [256, 256], seed=45)
    s.table[1, :2] = s.table[0, :2]
    s.pages = dfl.KvPages(s.kp, s.vp, s.table.cuda())
    s.k[1], s.v[1] = s.k[1].clone(), s.v[1].clone()
    s.k[1][:, :256], s.v[1][:, :256] = s.k[0][:, :256], s.v[0][:, :256]
    s.run()
    s.check()


def test_tracing_records_the_kernel_and_its_merge(dfl):
    s = Scene(dfl, *SHAPES["qwen"], [17], [900], seed=47)
    rec = dfl.TraceRecorder(8)
    s.run(trace=rec.struct)
    s.check(rows=4)
    got = rec.records()
    assert [k for k, _, _, _ in got] == [dfl.K_ATTN, dfl.K_ATTN]
    T = s.q.shape[0]      # the rows that the call got: two lie behind the sequence
    assert got[0][1] == 2.0 * (900 + T) * 8 * 128 * 2 + 2.0 * T * 32 * 128 * 2 and got[1][1] == 0.0
    assert all(ms >= 0 for _, _, _, ms in got)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv", [(16, 2), (64, 1), (3, 3)])
@pytest.mark.parametrize("ns,ctxs", [([200], [900]), ([70, 1, 129], [0, 500, 60])])
def test_fp32_chunks_of_many_rows_of_64(dfl, causal, hq, hkv, ns, ctxs):
    """Heads of 64 keep units of 64 rows, in one part and in several."""
    s = Scene(dfl, F32, hq, hkv, 64, ns, ctxs, seed=53)
    s.run(causal=causal)
    s.check(causal=causal, rows=12)


@pytest.mark.parametrize("shape", ["qwen", "g5_64", "f32_64", "f32_128"])
@pytest.mark.parametrize("cu,right", [([0, 17, 1 << 30], [17, 4]),      # claims more rows than there are: cut at the last
                                      ([-5, 17, 21], [17, 4]),          # begins before the first row
                                      ([0, 30, 10], [17, 0]),           # not ascending: sequence 0 takes all rows
                                      ([40, 50, 60], [0, 0])])          # behind the last row: nothing to do
def test_rows_of_offsets_that_disagree_are_right_and_none_is_written_behind_them(dfl, shape, cu, right):
    """q ends with its last row and rows of other use lie behind the output's."""
    s = Scene(dfl, *SHAPES[shape], [17, 4], [100, 50], seed=55, garbage=0.5, extra=40)
    s.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    s.q, s.out = s.q[:s.T], s.out[:s.T]
    s.run()
    torch.cuda.synchronize()
    got = s.out.clone()
    if right == [17, 4]:
        s.check()
    elif right == [17, 0]:       # rows 0..16 see the keys that they would; the four behind them see finite rows of the page
        for i in range(17):
            o, mass, _ = tr.chunk_attention(f64(s.q[i:i + 1]), f64(s.k[0])[:, :101 + i], f64(s.v[0])[:, :101 + i], 100 + i)
            # as for the sequence beside a bad page
            assert (np.abs(f64(got[i:i + 1]) - o) <= 2.0 ** -8 * (mass + np.abs(o)) + 2.0 ** -9 * mass).all(), i
        assert torch.isfinite(got).all()
    else:
        assert (got == 9).all()
    assert (s.obuf[s.T:] == 9).all() and (s.obuf[:, -1] == 9).all()
    assert int(s.st) == 0


@pytest.mark.parametrize("shape", ["qwen", "g7", "mha64", "f32_64", "f32_128"])
@pytest.mark.parametrize("ns,ctxs", [([17, 3], [300, 40]), ([1], [0]), ([140], [5]), ([5], [9000])])
def test_rows_behind_the_last_sequence_may_hold_anything(dfl, shape, ns, ctxs):
    """A padded batch: infinities and NaN in the rows that share a tile with the last sequence's."""
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=57, extra=130)
    s.qbuf[s.T::2] = float("nan")
    s.qbuf[s.T + 1::2] = float("inf")
    s.run()
    s.check(rows=6)


@pytest.mark.parametrize("shape", ["qwen", "g7", "mha64", "f32_128"])
@pytest.mark.parametrize("ns,ctxs", [([17], [9000]), ([300, 1], [5000, 2000]), ([6, 200], [-3, -150]), ([1, 4], [-1, -9])])
def test_whole_blocks_over_long_contexts_and_before_the_first_position(dfl, shape, ns, ctxs):
    """Not causal: units split over the GPU, and chunks that begin at negative positions."""
    s = Scene(dfl, *SHAPES[shape], ns, ctxs, seed=59)
    s.run(causal=False)
    s.check(causal=False, rows=6)


@pytest.mark.parametrize("shape", ["qwen", "f32_64"])
def test_a_table_without_a_place_left(dfl, shape):
    """The last key is the last row of the last page that the table names."""
    s = Scene(dfl, *SHAPES[shape], [17, 3], [495, 509], seed=61)
    s.pages = dfl.KvPages(s.kp, s.vp, s.table[:, :4].contiguous().cuda())
    s.run()
    s.check()
