"""GPU: the operators around a drafted tree together, as a speculative loop runs
them: pages are reserved, the nodes of a tree a sequence pass through a small
target model over the paged cache (positions by depth, rows by number, tree
attention), a token is drawn behind every node, the confirmed branch's rows move
behind the context, pages of the others are released, sequences are forked. Every
node's logits are checked against a float64 model that knows neither cache nor
trees: it computes each branch from its tokens alone."""
import numpy as np
import pytest
import torch

from oracle import dflash_ref as ref
from oracle import tree_ref as tt
from tests.test_gpu_target_pass import D, DH, EPS, HKV, HQ, L, THETA, V, GAMMA, Target, oracle_logits, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class TreeTarget(Target):
    """The target with a table that the library fills."""

    def __init__(self, dfl, W, dt, B, pages_per_seq=4, spare=3):
        super().__init__(dfl, W, dt, B, pages_per_seq)
        n = 2 * B + spare
        nan = float("nan")
        pool = lambda: torch.full((L, n, HKV, 128, DH), nan, dtype=dt, device="cuda")  # noqa: E731
        self.table = torch.full((B, pages_per_seq), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.pages = dfl.KvPages(pool(), pool(), self.table)

    def tree_logits(self, tokens, parents):
        """Logits of all nodes of a tree a sequence."""
        n = [len(t) for t in tokens]
        T = sum(n)
        cu, par = ints(np.cumsum([0] + n).tolist()), ints([p for t in parents for p in t])
        mask = torch.empty((T, (max(n) + 31) // 32), dtype=torch.int32, device="cuda")
        pos = torch.empty(T, dtype=torch.int32, device="cuda")
        self.dfl.dflash_tree_masks(par, cu, self.ctx, mask, pos, self.status)
        h = self.W["embed"][torch.tensor([x for t in tokens for x in t], device="cuda")].float()
        for l, w in enumerate(self.W["layers"]):
            y = self.linear(self.norm(h), w["qkv"])
            q, k = y[:, :HQ * DH].view(T, HQ, DH), y[:, HQ * DH:(HQ + HKV) * DH].view(T, HKV, DH)
            v = y[:, (HQ + HKV) * DH:].reshape(T, HKV, DH).to(self.dt)
            qo, ko = (torch.empty((T, x, DH), dtype=self.dt, device="cuda") for x in (HQ, HKV))
            o = torch.empty_like(qo)
            # turned by depth, stored by number
            self.dfl.dflash_qk_norm_rope(self.heads, q, k, pos, self.cos, self.sin, qo, ko, self.status, g_q=w["gq"], g_k=w["gk"])
            self.dfl.dflash_kv_append_paged(self.heads, None, ko, v, cu, self.ctx, l, self.pages, None, None, None, self.status)
            self.dfl.dflash_attention_tree_paged(self.heads, qo, cu, self.ctx, max(n), int(self.ctx.max()), l, self.pages, mask, o,
                                                 self.status, self.ws)
            h = h + self.linear(o.view(T, -1), w["o"])
        return self.linear(self.norm(h), self.W["head"]), cu, par


def draft(rng, W, seq, n):
    """A tree of n nodes: the anchor, then candidates, half of them the model's own choice."""
    tokens, parents, ways = [seq[-1]], [-1], [list(seq)]
    while len(tokens) < n:
        at = max(0, len(tokens) - 1 - int(rng.exponential(1.5)))
        best = int(oracle_logits(W, ways[at])[-1].argmax())
        new = best if rng.random() < 0.6 else int(rng.integers(0, V))
        if any(p == at and t == new for p, t in zip(parents, tokens)):
            new = int(rng.integers(0, V))
        parents.append(at)
        tokens.append(new)
        ways.append(ways[at] + [new])
    return tokens, parents, ways


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_loop_of_trees_matches_the_model_without_a_cache(dfl, dt):
    W, B = weights(5, dt), 3
    t = TreeTarget(dfl, W, dt, B)
    rng = np.random.default_rng(7)
    seqs = [list(rng.integers(0, V, n)) for n in (150, 1, 40)]
    sim = tt.Pages(t.table.tolist(), t.refs.tolist(), [0] * B)
    # the prompts, all but the anchor, as chains
    t.dfl.dflash_pages_reserve(t.pages, t.refs, ints([len(s) + 15 for s in seqs]), t.status)
    sim.reserve([len(s) + 15 for s in seqs])
    done = [0] * B
    while any(done[b] < len(seqs[b]) - 1 for b in range(B)):
        part = [seqs[b][done[b]:min(done[b] + 64, len(seqs[b]) - 1)] for b in range(B)]
        t.forward(part)
        t.ctx += ints([len(x) for x in part])
        done = [d + len(x) for d, x in zip(done, part)]
    tol = 0.01 if dt == torch.float32 else 0.05     # as for the loop of chains
    taus, forks = [], [(0, 1), (2, 0)]
    for cycle in range(6):
        trees = [draft(rng, W, seqs[b], n) for b, n in enumerate((14, 5, 9))]
        logits, cu, par = t.tree_logits([x[0] for x in trees], [x[1] for x in trees])
        at = 0
        for b, (tokens, parents, ways) in enumerate(trees):
            for i in range(len(tokens)):
                want = oracle_logits(W, ways[i])[-1]
                err = np.sqrt(np.mean((ref.f64(logits[at + i]) - want) ** 2)) / np.sqrt(np.mean(want ** 2))
                assert err < tol, (cycle, b, i, err)
            at += len(tokens)
        # a token behind every node: at most of the temperatures the model's choice is likely
        u = rng.random(at, dtype=np.float32)
        T, k, p = ([float(x) for x in rng.choice(c, at)] for c in ((0.0, 0.1, 0.3), (0, 5, 40), (1.0, 0.9)))
        drawn = torch.empty(at, dtype=torch.int32, device="cuda")
        f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
        dfl.dflash_sample(logits, f(u), drawn, t.status, temperature=f(T), top_k=ints([int(x) for x in k]), top_p=f(p))
        x = logits.double().cpu().numpy()
        y = [tt.draw(tt.shape(x[i], float(np.float32(T[i])), int(k[i]), float(np.float32(p[i]))), float(u[i])) for i in range(at)]
        assert drawn.tolist() == y
        tau, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
        com, path = (torch.empty((B, 8), dtype=torch.int32, device="cuda") for _ in range(2))
        dfl.dflash_verify_tree(ints([z for tr in trees for z in tr[0]]), par, drawn, cu, tau, com, path, nxt, t.status, heads=t.heads,
                               ctx_len=t.ctx, pages=t.pages)
        torch.cuda.synchronize()
        assert int(t.status) == 0
        first = 0
        for b, (tokens, parents, _) in enumerate(trees):
            want = tt.verify_tree(tokens, parents, y[first:first + len(tokens)], 8)
            assert (int(tau[b]), com[b].tolist(), path[b].tolist(), int(nxt[b])) == want
            seqs[b] += want[1][:want[0]]
            taus.append(want[0])
            first += len(tokens)
        t.ctx += tau
        # rows that were not kept give their pages back; sequences branch; room for the next trees
        dfl.dflash_pages_release(t.pages, t.refs, t.ctx, t.status)
        sim.release(t.ctx.tolist())
        sim.length = t.ctx.tolist()
        if cycle in (1, 3):
            s, d = forks[cycle // 2]
            dfl.dflash_pages_fork(t.heads, t.pages, t.refs, t.ctx, ints([s]), ints([d]), t.status)
            sim.fork([s], [d])
            seqs[d] = list(seqs[s])
        dfl.dflash_pages_reserve(t.pages, t.refs, t.ctx + 15, t.status)
        sim.reserve([n + 15 for n in sim.length])
        torch.cuda.synchronize()
        assert t.table.tolist() == sim.table and t.refs.tolist() == sim.refs and t.ctx.tolist() == sim.length
        assert int(t.status) == 0 and not sim.full
        assert [len(s) - 1 for s in seqs] == t.ctx.tolist()
    assert max(taus) > 2 and min(taus) >= 1


def test_shaped_distributions_feed_the_verification_of_a_block(dfl):
    """dflash_sample's probs are dflash_verify_probs' targets: temperature and top-p of the caller's own."""
    B, m = 3, GAMMA
    cfg = dfl.make_config(1, D, 1, D, HQ, HKV, DH, 512, V, m, V - 1, B, 512, rope_theta=THETA, rms_eps=EPS)
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((B * (m + 1), V), generator=g, device="cuda") * 3
    one = lambda v: torch.full((B * (m + 1),), v, device="cuda")  # noqa: E731
    probs, st = torch.empty_like(logits), torch.zeros(1, dtype=torch.int32, device="cuda")
    dfl.dflash_sample(logits, None, None, st, temperature=one(0.7), top_p=one(0.9), probs=probs)
    p = probs.view(B, m + 1, V)
    draft_ids = p[:, :m].argmax(-1).to(torch.int32)
    ua, ud = torch.rand((B, m), generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    tau, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    com = torch.empty((B, m + 1), dtype=torch.int32, device="cuda")
    dfl.dflash_verify_probs(cfg, p, None, draft_ids, ua, ud, tau, com, nxt, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    from oracle import target_ref as tr
    for b in range(B):
        a, c, y = tr.verify_probs(p[b].cpu(), None, draft_ids[b].tolist(), ua[b].cpu().numpy(), float(ud[b]))
        assert (int(tau[b]), com[b].tolist(), int(nxt[b])) == (a, c.tolist(), y)
        assert p[b, a - 1, y] > 0


# ------------------------------------------------------------------ refusals
def test_operands_on_the_host_are_refused(dfl):
    from tests.test_gpu_target_refusals import refused_for_each
    bf, dev = torch.bfloat16, "cuda"
    heads = dfl.make_heads(1, 4, 2, 64)
    T = 5
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    st, cu, ctx = zeros(1), ints([0, T]), ints([100])
    par, tok, drawn = ints([-1, 0, 1, 1, 0]), ints([1, 2, 3, 4, 5]), ints([2, 3, 9, 9, 9])
    pool = lambda: torch.zeros((1, 3, 2, 128, 64), dtype=bf, device=dev)  # noqa: E731
    kp, vp, table = pool(), pool(), ints([[2, 0]])
    q = torch.randn((T, 4, 64), device=dev).to(bf)
    ws = dfl.ChunkWorkspace(heads)
    refused_for_each(dfl, lambda dev_status, **kw: dfl.dflash_tree_masks(**kw, dev_status=dev_status),
                     dict(parents=par, cu_rows=cu, ctx_len=ctx, mask=zeros(T, 1), positions=zeros(T), dev_status=st))

    def attend(q, cu, ctx, kp, vp, table, mask, out, dev_status):
        dfl.dflash_attention_tree_paged(heads, q, cu, ctx, T, 100, 0, dfl.KvPages(kp, vp, table), mask, out, dev_status, ws)

    refused_for_each(dfl, attend, dict(q=q, cu=cu, ctx=ctx, kp=kp, vp=vp, table=table, mask=zeros(T, 1), out=torch.empty_like(q), dev_status=st))
    f = lambda: torch.full((3,), 0.5, device=dev)  # noqa: E731
    refused_for_each(dfl, lambda **kw: dfl.dflash_sample(**kw),
                     dict(logits=torch.randn((3, 50), device=dev), u=f(), tokens=zeros(3), dev_status=st, temperature=f(), top_k=zeros(3),
                          top_p=f(), min_p=f(), probs=torch.empty((3, 50), device=dev)))

    def verify(kp, vp, table, **kw):
        dfl.dflash_verify_tree(**kw, heads=heads, pages=dfl.KvPages(kp, vp, table))

    refused_for_each(dfl, verify, dict(tokens=tok, parents=par, drawn=drawn, cu_rows=cu, tau=zeros(1), committed=zeros(1, 4), path=zeros(1, 4),
                                       next_anchor=zeros(1), dev_status=st, ctx_len=ctx, kp=kp, vp=vp, table=table))
    refs = ints([1, 0, 1])
    for call in (dfl.dflash_pages_release, dfl.dflash_pages_reserve):
        refused_for_each(dfl, lambda kp, vp, table, refs, n, dev_status: call(dfl.KvPages(kp, vp, table), refs, n, dev_status),
                         dict(kp=kp, vp=vp, table=table, refs=refs, n=ints([200]), dev_status=st))
    two = ints([[2, 0], [-1, -1]])
    refused_for_each(dfl, lambda kp, vp, table, refs, ctx, src, dst, dev_status: dfl.dflash_pages_fork(
        heads, dfl.KvPages(kp, vp, table), refs, ctx, src, dst, dev_status),
        dict(kp=kp, vp=vp, table=two, refs=refs, ctx=ints([100, 0]), src=ints([0]), dst=ints([1]), dev_status=st))
