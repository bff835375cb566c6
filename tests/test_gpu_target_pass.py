"""GPU: the target-side operators together, as a speculative decoding loop runs
them: a small target model reads its prompts in chunks (projections, per-head
norms and rotation on the way into the paged cache, chunk attention), then
cycles of drafted blocks are verified against its probabilities, the rejected
tokens' cache rows being overwritten by the next block. Every cycle is checked
against a float64 model that knows no cache: it computes each sequence from its
tokens alone."""
import numpy as np
import pytest
import torch

from oracle import dflash_ref as ref
from oracle import target_ref as tr

pytestmark = pytest.mark.gpu

D, HQ, HKV, DH, L, V, GAMMA, THETA, EPS = 256, 8, 2, 64, 2, 311, 5, 1e4, 1e-6


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def weights(seed, dt):
    g = torch.Generator().manual_seed(seed)
    lin = lambda o, i: (torch.randn((o, i), generator=g) * i ** -0.5).to(dt)  # noqa: E731
    gain = lambda n: (1 + 0.1 * torch.randn(n, generator=g)).to(dt)  # noqa: E731
    return {"embed": (torch.randn((V, D), generator=g)).to(dt), "head": lin(V, D) * 3,
            "layers": [{"qkv": lin((HQ + 2 * HKV) * DH, D), "o": lin(D, HQ * DH), "gq": gain(DH), "gk": gain(DH)} for _ in range(L)]}


def oracle_logits(W, tokens):
    """Logits of the last rows, from the tokens alone: no cache, no chunks."""
    h = ref.f64(W["embed"])[np.asarray(tokens)]
    pos = np.arange(len(tokens))
    for w in W["layers"]:
        x = h / np.sqrt((h * h).mean(-1, keepdims=True) + EPS)
        y = x @ ref.f64(w["qkv"]).T
        q, k, v = np.split(y, [HQ * DH, (HQ + HKV) * DH], -1)
        q = tr.qk_norm_rope(q.reshape(-1, HQ, DH), w["gq"], pos, EPS, THETA)
        k = tr.qk_norm_rope(k.reshape(-1, HKV, DH), w["gk"], pos, EPS, THETA).transpose(1, 0, 2)
        v = v.reshape(-1, HKV, DH).transpose(1, 0, 2)
        o, _, _ = tr.chunk_attention(q, k, v, 0)
        h = h + o.reshape(len(tokens), -1) @ ref.f64(w["o"]).T
    x = h / np.sqrt((h * h).mean(-1, keepdims=True) + EPS)
    return x @ ref.f64(W["head"]).T


class Target:
    """The same model over the library's calls."""

    def __init__(self, dfl, W, dt, B, pages_per_seq=4):
        self.dfl, self.dt = dfl, dt
        code = dfl.BF16 if dt == torch.bfloat16 else dfl.F32
        self.heads = dfl.make_heads(L, HQ, HKV, DH, rms_eps=EPS, dtype=code)
        self.W = {"embed": W["embed"].cuda(), "head": W["head"].cuda(), "layers": [{k: v.cuda() for k, v in w.items()} for w in W["layers"]]}
        n = B * pages_per_seq
        shape = (L, n, HKV, 128, DH)
        order = torch.randperm(n, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(B, pages_per_seq)
        nan = float("nan")
        self.pages = dfl.KvPages(torch.full(shape, nan, dtype=dt, device="cuda"), torch.full(shape, nan, dtype=dt, device="cuda"),
                                 order.cuda())
        self.ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ws = dfl.ChunkWorkspace(self.heads)
        cfg = dfl.make_config(1, D, 1, D, HQ, HKV, DH, 512, V, GAMMA, V - 1, B, pages_per_seq * 128, rope_theta=THETA)
        self.cfg = cfg
        self.lin_ws = dfl.Workspace(cfg, 16)
        self.cos, self.sin = (t.cuda() for t in dfl.dflash_rope_tables(cfg, pages_per_seq * 128))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def linear(self, x, w):
        y = torch.empty((x.shape[0], w.shape[0]), dtype=torch.float32, device="cuda")
        self.dfl.dflash_linear(x, w, y, self.lin_ws)
        return y

    def norm(self, h):
        return (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)).to(self.dt)

    def forward(self, tokens):
        """tokens: new token ids per sequence (ragged); returns the logits [T, V] of all new rows."""
        T = sum(len(t) for t in tokens)
        n = [len(t) for t in tokens]
        cu = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device="cuda")
        ids = torch.tensor([x for t in tokens for x in t], device="cuda")
        h = self.W["embed"][ids].float()
        hint = int(self.ctx.max())
        for l, w in enumerate(self.W["layers"]):
            y = self.linear(self.norm(h), w["qkv"])          # fp32 rows: Q, K, V heads side by side
            q = y[:, :HQ * DH].view(T, HQ, DH)
            k = y[:, HQ * DH:(HQ + HKV) * DH].view(T, HKV, DH)
            v = y[:, (HQ + HKV) * DH:].view(T, HKV, DH)
            qo = torch.empty((T, HQ, DH), dtype=self.dt, device="cuda")
            o = torch.empty_like(qo)
            self.dfl.dflash_kv_append_paged(self.heads, q, k, v, cu, self.ctx, l, self.pages, self.cos, self.sin, qo, self.status,
                                            g_q=w["gq"], g_k=w["gk"])
            self.dfl.dflash_attention_chunk_paged(self.heads, qo, cu, self.ctx, max(n), hint, l, self.pages, o, self.status, self.ws)
            h = h + self.linear(o.view(T, -1), w["o"])
        return self.linear(self.norm(h), self.W["head"])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_a_speculative_loop_matches_the_model_without_a_cache(dfl, dt):
    W = weights(5, dt)
    B = 3
    t = Target(dfl, W, dt, B)
    rng = np.random.default_rng(1)
    # the drafts that a greedy drafter would make: half of them the model's own choice
    seqs = [list(rng.integers(0, V, n)) for n in (150, 1, 40)]
    # prompts in chunks of up to 64 tokens, all but the last token (the anchor)
    done = [0] * B
    while any(done[b] < len(seqs[b]) - 1 for b in range(B)):
        part = [seqs[b][done[b]:min(done[b] + 64, len(seqs[b]) - 1)] for b in range(B)]
        t.forward(part)
        n = torch.tensor([len(x) for x in part], dtype=torch.int32, device="cuda")
        t.ctx += n
        done = [d + len(x) for d, x in zip(done, part)]
    # logits of fp32 pass through two layers of fp32 (tf32 projections: 2^-11 an operand): 1 % of their RMS; bf16: 5 %
    tol = 0.01 if dt == torch.float32 else 0.05
    taus = []
    for cycle in range(6):
        drafts = []
        for b in range(B):
            d = []
            for j in range(GAMMA):
                best = int(oracle_logits(W, seqs[b] + d)[-1].argmax())
                d.append(best if rng.random() < 0.7 else int(rng.integers(0, V)))
            drafts.append(d)
        logits = t.forward([[seqs[b][-1]] + drafts[b] for b in range(B)]).view(B, GAMMA + 1, V)
        for b in range(B):
            want = oracle_logits(W, seqs[b] + drafts[b])[-(GAMMA + 1):]
            err = np.sqrt(np.mean((ref.f64(logits[b]) - want) ** 2)) / np.sqrt(np.mean(want ** 2))
            assert err < tol, (cycle, b, err)
        p = torch.softmax(logits, -1)
        ua, ud = torch.rand((B, GAMMA), device="cuda"), torch.rand(B, device="cuda")
        draft = torch.tensor(drafts, dtype=torch.int32, device="cuda")
        tau, nxt = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        com = torch.empty((B, GAMMA + 1), dtype=torch.int32, device="cuda")
        dfl.dflash_verify_probs(t.cfg, p, None, draft, ua, ud, tau, com, nxt, t.status)
        torch.cuda.synchronize()
        assert int(t.status) == 0
        for b in range(B):
            a, c, y = tr.verify_probs(p[b].cpu(), None, drafts[b], ua[b].cpu().numpy(), float(ud[b]))
            assert (int(tau[b]), int(nxt[b]), com[b].tolist()) == (a, y, c.tolist())
            seqs[b] += c[:a].tolist()
            taus.append(a)
        t.ctx += tau        # the anchor and the kept drafts stay; the rest is overwritten next cycle
    assert min(taus) < GAMMA + 1 and max(taus) > 1
    assert [len(s) - 1 for s in seqs] == t.ctx.tolist()


def test_dense_and_paged_forms_of_the_norm_agree(dfl):
    """dflash_qk_norm_rope on the rows and positions of a ragged batch gives the queries of dflash_kv_append_paged bit for bit."""
    W = weights(6, torch.bfloat16)
    t = Target(dfl, W, torch.bfloat16, 2)
    g = torch.Generator().manual_seed(2)
    rows = torch.randn((9, (HQ + 2 * HKV) * DH), generator=g).cuda()
    q, k = rows[:, :HQ * DH].view(9, HQ, DH), rows[:, HQ * DH:(HQ + HKV) * DH].view(9, HKV, DH)
    v = rows[:, (HQ + HKV) * DH:].view(9, HKV, DH)
    cu = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    t.ctx.copy_(torch.tensor([126, 3], dtype=torch.int32))
    w = t.W["layers"][0]
    qa, qb = (torch.empty((9, HQ, DH), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb = torch.empty((9, HKV, DH), dtype=torch.bfloat16, device="cuda")
    dfl.dflash_kv_append_paged(t.heads, q, k, v, cu, t.ctx, 0, t.pages, t.cos, t.sin, qa, t.status, g_q=w["gq"], g_k=w["gk"])
    pos = torch.tensor([126, 127, 128, 129, 3, 4, 5, 6, 7], dtype=torch.int32, device="cuda")
    dfl.dflash_qk_norm_rope(t.heads, q, k, pos, t.cos, t.sin, qb, kb, t.status, g_q=w["gq"], g_k=w["gk"])
    torch.cuda.synchronize()
    assert int(t.status) == 0 and torch.equal(qa, qb)
    table, pool = t.pages._keep[2].cpu().numpy(), t.pages._keep[0]
    for i, (b, p) in enumerate([(0, 126), (0, 127), (0, 128), (0, 129)] + [(1, x) for x in range(3, 8)]):
        assert torch.equal(pool[0, int(table[b, p // 128]), :, p % 128], kb[i])
