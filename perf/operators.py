"""Cases of the target-side operators of a speculative decoding step.

A drafting cycle hands gamma drafted tokens to the target model, which runs
them (and, before the first cycle, the prompt) as a chunk of new tokens over
its own paged KV cache and decides which drafts stand. Four operators:

  norm_rope   per-head RMSNorm of queries and keys, then the position rotation
  append      the same on the way into a paged cache: rotated keys and plain
              values into their pages, rotated queries out
  attention   causal attention of a ragged batch of chunks over the paged cache
  verify      acceptance of drafted tokens against the target's probabilities
              from given random numbers, with the replacement or bonus token

`run` computes a case in its plain form (elementary torch operations in 32
bits, in 64 where sums are long or values sit next to a border) or, where
`own` is true, by the framework's calls. Lengths are a function of the case,
values of the seed.
"""
import math
import random

import torch

own = False

PAGE = 128
EPS = 1e-6
THETA = 1e6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    qwen = dict(hq=32, hkv=8, dh=128)          # Qwen3-8B heads
    tiny = dict(hq=4, hkv=4, dh=64)            # the tiny fp32 drafter's heads
    att = dict(op="attention", dtype="bf16", **qwen)
    return [
        # one sequence's drafted block (anchor + 16 drafts) over a short context: latency
        dict(att, name="attn_verify_B1_ctx2048", batch=1, rows=17, rows_min=17, ctx=2048, ctx_min=2048),
        # the same over a long context: the cache's bytes
        dict(att, name="attn_verify_B1_ctx32768", batch=1, rows=17, rows_min=17, ctx=32768, ctx_min=32768),
        # a serving step without drafts: one token each of a ragged batch
        dict(att, name="attn_decode_B64_ragged", batch=64, rows=1, rows_min=1, ctx=8192, ctx_min=512),
        # a chunk of a long prompt, behind what earlier chunks left in the cache
        dict(att, name="attn_prefill_2048_ctx6000", batch=1, rows=2048, rows_min=2048, ctx=6000, ctx_min=6000),
        # the tiny fp32 shapes, ragged blocks, one of them over an empty context
        dict(op="attention", dtype="f32", **tiny, name="attn_f32_tiny_B3", batch=3, rows=17, rows_min=1, ctx=900,
             ctx_min=0),
        # one block of a batch-1 cycle: latency
        dict(op="norm_rope", dtype="bf16", in_dtype="bf16", **qwen, name="norm_rope_17", batch=1, rows=17, rows_min=17,
             ctx=2048, ctx_min=2048),
        # a long prompt in one pass
        dict(op="norm_rope", dtype="bf16", in_dtype="bf16", **qwen, name="norm_rope_32768", batch=1, rows=32768,
             rows_min=32768, ctx=0, ctx_min=0),
        # a ragged batch's blocks, from the fp32 outputs of the projection
        dict(op="append", dtype="bf16", in_dtype="f32", **qwen, name="append_B16_blocks_f32in", batch=16, rows=17,
             rows_min=1, ctx=8192, ctx_min=512),
        # prompts of a ragged batch, appended behind shared prefixes
        dict(op="append", dtype="bf16", in_dtype="bf16", **qwen, name="append_B5_prompts", batch=5, rows=4000, rows_min=300,
             ctx=1000, ctx_min=0),
        # sampling verification of one sequence: latency
        dict(op="verify", dtype="f32", name="verify_B1", batch=1, gamma=16, vocab=151936, greedy=False),
        # a batch whose drafts came from a greedy drafter (q is one token)
        dict(op="verify", dtype="f32", name="verify_B16_greedy_drafts", batch=16, gamma=16, vocab=151936, greedy=True),
        # a large serving batch
        dict(op="verify", dtype="f32", name="verify_B64", batch=64, gamma=16, vocab=151936, greedy=False),
    ]


def _logint(rng, lo, hi):
    """An integer between lo and hi, even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "norm_rope", "verify"])
    if op == "verify":
        vocab = _logint(rng, 1003, 200003)
        return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), batch=_logint(rng, 1, max(1, min(64, 9700000 // vocab))),
                    gamma=rng.randint(1, 16), vocab=vocab, greedy=rng.random() < 0.3)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hq, hkv, dh = rng.choice([(32, 8, 128), (32, 8, 128), (8, 2, 64), (4, 4, 64), (28, 4, 128), (10, 2, 128), (16, 1, 64)])
    c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, dh=dh)
    if op != "attention":
        c["in_dtype"] = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        batch = _logint(rng, 1, 64)
        rows = _logint(rng, 1, max(1, 16000 // batch))
        ctx = _logint(rng, 1, 8192)
        return dict(c, batch=batch, rows=rows, rows_min=rng.randint(1, rows), ctx=ctx, ctx_min=rng.randint(0, ctx))
    batch = _logint(rng, 1, 64)
    ctx = _logint(rng, 1, max(64, min(32768, (250000 if dtype == "bf16" else 120000) * 1024 // (hkv * dh) // batch)))
    # the padded plain form's scores, batch * hq * rows * (ctx + rows), are bounded
    most = int((math.sqrt(ctx * ctx + 4 * 5e8 / (batch * hq)) - ctx) / 2)
    if dtype == "f32":
        most = min(most, 64)
    rows = _logint(rng, 1, max(1, min(2048, most)))
    return dict(c, batch=batch, rows=rows, rows_min=rng.randint(1, rows), ctx=ctx, ctx_min=rng.randint(0, ctx))


# ------------------------------------------------------------------ inputs
def _lens(case):
    """(new rows, context) of each sequence: the longest of both first, the others spread over their ranges."""
    r = random.Random("%(batch)d %(rows)d %(rows_min)d %(ctx)d %(ctx_min)d" % case)
    n = [case["rows"]] + [r.randint(case["rows_min"], case["rows"]) for _ in range(case["batch"] - 1)]
    c = [case["ctx"]] + [r.randint(case["ctx_min"], case["ctx"]) for _ in range(case["batch"] - 1)]
    if case["batch"] > 1 and case["ctx_min"] == 0:
        c[-1] = 0
    return n, c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & ((1 << 62) - 1))


def _normal(g, shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).add_(shift).to(dtype)


def _rope(n, dh):
    """fp32 tables [n, dh/2] of cos and sin of p * THETA^(-2j/dh), from 64-bit angles."""
    j = torch.arange(dh // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * THETA ** (-2.0 * j / dh)
    return a.cos().float(), a.sin().float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "verify":
        B, m, V = case["batch"], case["gamma"], case["vocab"]
        # a peaked drafter and a target near it, as in a trained pair
        lg = _normal(g, (B, m + 1, V), scale=2.5)
        q = torch.softmax(lg[:, :m], -1)
        p = torch.softmax(lg.add_(_normal(g, (B, m + 1, V), scale=0.6)), -1)
        del lg
        if case["greedy"]:
            draft = q.argmax(-1)
            s["draft_probs"] = None
            # the target agrees with a greedy drafter most of the time
            p[:, :m].mul_(0.25).scatter_add_(2, draft[..., None], torch.full((B, m, 1), 0.75, device="cuda"))
        else:
            draft = torch.multinomial(q.view(B * m, V), 1, generator=g).view(B, m)
            s["draft_probs"] = q
        s["target_probs"] = p.to(DTYPES[case["dtype"]])
        s["draft"] = draft.to(torch.int32)
        s["u_accept"] = torch.rand((B, m), generator=g, device="cuda")
        s["u_draw"] = torch.rand((B,), generator=g, device="cuda")
        s["tau"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["committed"] = torch.zeros((B, m + 1), dtype=torch.int32, device="cuda")
        s["next_anchor"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    n, ctx = _lens(case)
    B, T, hq, hkv, dh = case["batch"], sum(n), case["hq"], case["hkv"], case["dh"]
    dt = DTYPES[case["dtype"]]
    s["max_rows"], s["max_ctx"] = max(n), max(ctx)
    s["cu_rows"] = _ints([sum(n[:b]) for b in range(B + 1)])
    s["ctx_len"] = _ints(ctx)
    need = max(c + m for c, m in zip(ctx, n))
    if case["op"] != "norm_rope":
        # pages of all sequences, scattered over the pool; pages of other sequences' tokens between them
        per = (need + PAGE - 1) // PAGE
        have = [(c + m + PAGE - 1) // PAGE for c, m in zip(ctx, n)]
        n_pages = sum(have) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            table[b, : have[b]] = order[at:at + have[b]]
            at += have[b]
        s["page_table"] = table
        s["k_pool"] = _normal(g, (1, n_pages, hkv, PAGE, dh), dt)
        s["v_pool"] = _normal(g, (1, n_pages, hkv, PAGE, dh), dt)
    if case["op"] == "attention":
        s["q"] = _normal(g, (T, hq, dh), dt, scale=1.5)      # rotated queries, a little peaked
        s["out"] = torch.zeros((T, hq, dh), dtype=dt, device="cuda")
        return s
    # the projection's rows: Q heads, K heads, V heads side by side
    qkv = _normal(g, (T, (hq + 2 * hkv) * dh), DTYPES[case["in_dtype"]])
    s["q"] = qkv[:, : hq * dh].view(T, hq, dh)
    s["k"] = qkv[:, hq * dh:(hq + hkv) * dh].view(T, hkv, dh)
    s["v"] = qkv[:, (hq + hkv) * dh:].view(T, hkv, dh)
    s["g_q"] = _normal(g, (dh,), dt, scale=0.1, shift=1.0)
    s["g_k"] = _normal(g, (dh,), dt, scale=0.1, shift=1.0)
    s["cos"], s["sin"] = _rope(max(need, PAGE), dh)
    s["q_out"] = torch.zeros((T, hq, dh), dtype=dt, device="cuda")
    if case["op"] == "norm_rope":
        s["k_out"] = torch.zeros((T, hkv, dh), dtype=dt, device="cuda")
        s["positions"] = torch.cat([torch.arange(c, c + m, dtype=torch.int32, device="cuda") for c, m in zip(ctx, n)])
    return s


# ------------------------------------------------------------------ plain forms
def _norm_rope(x, gain, cos, sin):
    """x [T, H, Dh] -> gain * x / rms(x), its halves rotated by cos / sin [T, Dh/2]; 32 bits."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    h = x.shape[-1] // 2
    a, b, c, s = x[..., :h], x[..., h:], cos[:, None], sin[:, None]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _token_place(s, T):
    """Sequence and position of each packed row."""
    cu, t = s["cu_rows"].long(), torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, s["ctx_len"].long()[seq] + t - cu[seq]


def _plain_norm_rope(s):
    p = s["positions"].long()
    cos, sin = s["cos"][p], s["sin"][p]
    s["q_out"].copy_(_norm_rope(s["q"], s["g_q"], cos, sin))
    s["k_out"].copy_(_norm_rope(s["k"], s["g_k"], cos, sin))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_append(s):
    seq, p = _token_place(s, s["q"].shape[0])
    cos, sin = s["cos"][p], s["sin"][p]
    s["q_out"].copy_(_norm_rope(s["q"], s["g_q"], cos, sin))
    page = s["page_table"].long()[seq, p // PAGE]
    k, v = s["k_pool"][0], s["v_pool"][0]
    k[page, :, p % PAGE] = _norm_rope(s["k"], s["g_k"], cos, sin).to(k.dtype)
    v[page, :, p % PAGE] = s["v"].to(v.dtype)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_attention(s):
    hq, hkv, dh, B, T = s["hq"], s["hkv"], s["dh"], s["batch"], s["q"].shape[0]
    G, R = hq // hkv, s["max_rows"]
    seq, pos = _token_place(s, T)
    row = torch.arange(T, device="cuda") - s["cu_rows"].long()[seq]
    table = s["page_table"].long().clamp(min=0)
    n_keys = table.shape[1] * PAGE

    def rows_of(pool):          # [B, hkv, keys, dh] in 32 bits
        return pool[0][table].transpose(1, 2).reshape(B, hkv, n_keys, dh).float()

    keys = torch.arange(n_keys, device="cuda")
    length = s["ctx_len"].long() + s["cu_rows"].long().diff()
    q = torch.zeros((B, R, hq, dh), device="cuda")
    q[seq, row] = s["q"].float()
    last = torch.full((B, R), -1, dtype=torch.long, device="cuda")      # the last key that a row sees
    last[seq, row] = pos
    q = q.view(B, R, hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * R, dh)
    x = torch.matmul(q, rows_of(s["k_pool"]).transpose(2, 3)) * (dh ** -0.5)
    hidden = (keys > last[:, :, None])[:, None, None].expand(B, 1, G, R, n_keys).reshape(B, 1, G * R, n_keys)
    x = x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    v = rows_of(s["v_pool"]).masked_fill_((keys >= length[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, hkv, G, R, dh).permute(0, 3, 1, 2, 4).reshape(B, R, hq, dh)
    s["out"].copy_(o[seq, row])
    return s["out"]


def _plain_verify(s):
    p, x, m = s["target_probs"], s["draft"].long(), s["gamma"]
    px = p[:, :m].gather(2, x[..., None])[..., 0].double()
    if s["draft_probs"] is None:
        qx = torch.ones_like(px)
    else:
        qx = s["draft_probs"].gather(2, x[..., None])[..., 0].double()
    kept = (s["u_accept"].double() * qx < px).long().cumprod(-1)        # 64 bits: the products are exact
    a = kept.sum(-1)
    b = torch.arange(a.shape[0], device="cuda")
    at = a.clamp(max=m - 1)
    w = p[b, a].double()
    if s["draft_probs"] is None:
        left = w.scatter(1, x[b, at][:, None], 0.0)
    else:
        left = (w - s["draft_probs"][b, at].double()).clamp_(min=0.0)
    left = torch.where((a < m)[:, None], left, w)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, w)
    c = left.cumsum(-1)
    y = (c <= s["u_draw"].double()[:, None] * c[:, -1:]).sum(-1).clamp(max=p.shape[2] - 1)
    s["tau"].copy_(a + 1)
    j = torch.arange(m + 1, device="cuda")
    drafts = torch.cat((x, x[:, :1]), 1)
    com = torch.where(j < a[:, None], drafts, torch.where(j == a[:, None], y[:, None], -1))
    s["committed"].copy_(com)
    s["next_anchor"].copy_(y)
    return {"tau": s["tau"], "committed": s["committed"], "next_anchor": s["next_anchor"]}


# ------------------------------------------------------------------ the framework's calls
def _handles(s):
    """What a program keeps beside its tensors: the layout, the page view, the scratch; made once for a state."""
    import block_diffusion_drafter_gb300 as dfl
    if "lib" not in s:
        s["lib"] = dfl
        dt = dfl.BF16 if s["dtype"] == "bf16" else dfl.F32
        if s["op"] == "verify":
            s["cfg"] = dfl.make_config(1, 256, 1, 256, 4, 4, 64, 512, s["vocab"], s["gamma"], s["vocab"] - 1, s["batch"], 128)
        else:
            s["heads"] = dfl.make_heads(1, s["hq"], s["hkv"], s["dh"], rms_eps=EPS, dtype=dt)
        if "page_table" in s:
            s["pages"] = dfl.KvPages(s["k_pool"], s["v_pool"], s["page_table"])
        if s["op"] == "attention":
            s["ws"] = dfl.ChunkWorkspace(s["heads"])
    return s["lib"]


def run(s):
    op = s["op"]
    if not own:
        return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attention": _plain_attention,
                "verify": _plain_verify}[op](s)
    dfl = _handles(s)
    if op == "norm_rope":
        dfl.dflash_qk_norm_rope(s["heads"], s["q"], s["k"], s["positions"], s["cos"], s["sin"], s["q_out"], s["k_out"],
                                s["status"], g_q=s["g_q"], g_k=s["g_k"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        dfl.dflash_kv_append_paged(s["heads"], s["q"], s["k"], s["v"], s["cu_rows"], s["ctx_len"], 0, s["pages"], s["cos"],
                                   s["sin"], s["q_out"], s["status"], g_q=s["g_q"], g_k=s["g_k"])
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "attention":
        dfl.dflash_attention_chunk_paged(s["heads"], s["q"], s["cu_rows"], s["ctx_len"], s["max_rows"], s["max_ctx"], 0,
                                         s["pages"], s["out"], s["status"], s["ws"])
        return s["out"]
    dfl.dflash_verify_probs(s["cfg"], s["target_probs"], s["draft_probs"], s["draft"], s["u_accept"], s["u_draw"], s["tau"],
                            s["committed"], s["next_anchor"], s["status"])
    return {"tau": s["tau"], "committed": s["committed"], "next_anchor": s["next_anchor"]}


# ------------------------------------------------------------------ work
def _bytes(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] == "verify":
        # the rows that the last token is drawn from, and the drafts' own entries
        B, m, V = case["batch"], case["gamma"], case["vocab"]
        row = _bytes(case["dtype"]) + (0 if case["greedy"] else 4)
        return {"bytes": B * (V * row + m * (row + 8) + (m + 1) * 4 + 8.0), "flops": 3.0 * B * V}
    n, ctx = _lens(case)
    T, hq, hkv, dh = sum(n), case["hq"], case["hkv"], case["dh"]
    es = _bytes(case["dtype"])
    if case["op"] == "attention":
        keys = sum(c + m for c, m in zip(ctx, n))
        seen = sum(m * c + m * (m + 1) / 2 for c, m in zip(ctx, n))
        return {"bytes": 2.0 * keys * hkv * dh * es + 2.0 * T * hq * dh * es, "flops": 4.0 * seen * hq * dh}
    heads = hq + hkv + (hkv if case["op"] == "append" else 0)
    tables = (max(c + m for c, m in zip(ctx, n)) if case["batch"] == 1 and ctx[0] == 0 else T) * dh * 4.0
    return {"bytes": T * heads * dh * float(_bytes(case["in_dtype"]) + es) + tables, "flops": 7.0 * T * (hq + hkv) * dh}


# ------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    n, ctx = _lens(case)
    if case["op"] == "attention":
        return _exact_attention(s, n, ctx)
    pos = [c + i for c, m in zip(ctx, n) for i in range(m)]
    at = torch.tensor(pos, device="cuda")
    # a rotation by the angle of (cos, sin) is a product of complex numbers
    turn = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]

    def turned(x, gain):
        x = x.double()
        x = x / ((x ** 2).sum(-1, keepdim=True) / case["dh"] + EPS).sqrt() * gain.double()
        z = torch.complex(*x.split(case["dh"] // 2, -1)) * turn
        return torch.cat((z.real, z.imag), -1)

    q, k = turned(s["q"], s["g_q"]), turned(s["k"], s["g_k"])
    if case["op"] == "norm_rope":
        return {"q": q, "k": k}
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    first = 0
    for b in range(case["batch"]):
        pages = s["page_table"][b].tolist()
        for p0 in range(ctx[b] - ctx[b] % PAGE, ctx[b] + n[b], PAGE):
            lo, hi = max(p0, ctx[b]), min(p0 + PAGE, ctx[b] + n[b])
            rows = slice(first + lo - ctx[b], first + hi - ctx[b])
            kp[0, pages[p0 // PAGE], :, lo - p0:hi - p0] = k[rows].transpose(0, 1)
            vp[0, pages[p0 // PAGE], :, lo - p0:hi - p0] = s["v"][rows].double().transpose(0, 1)
        first += n[b]
    return {"q": q, "k_pool": kp, "v_pool": vp}


def _exact_attention(s, n, ctx):
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    if sum(m * c + m * m / 2 for c, m in zip(ctx, n)) * hq * dh * 4 > 4e11:
        return None
    out, first = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b in range(s["batch"]):
        keys = ctx[b] + n[b]
        pages = s["page_table"][b, : (keys + PAGE - 1) // PAGE].long()
        for h in range(hkv):
            k = s["k_pool"][0, pages, h].reshape(-1, dh)[:keys].double()
            v = s["v_pool"][0, pages, h].reshape(-1, dh)[:keys].double()
            for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                x = s["q"][first:first + n[b], i].double() @ k.T / math.sqrt(dh)
                x = x + torch.full_like(x, -math.inf).triu(ctx[b] + 1)
                out[first:first + n[b], i] = torch.softmax(x, -1) @ v
        first += n[b]
    return out


def _exact_verify(s):
    B, m, V = s["batch"], s["gamma"], s["vocab"]
    draft, u, ud = s["draft"].tolist(), s["u_accept"].double().tolist(), s["u_draw"].double().tolist()
    tau, com, last = [], [], []
    for b in range(B):
        p = s["target_probs"][b]
        q = None if s["draft_probs"] is None else s["draft_probs"][b]
        a = 0
        while a < m and u[b][a] * (1.0 if q is None else float(q[a, draft[b][a]])) < float(p[a, draft[b][a]]):
            a += 1
        w = p[a].double()
        if a < m:
            r = w.clone()
            if q is None:
                r[draft[b][a]] = 0.0
            else:
                r = torch.maximum(r - q[a].double(), torch.zeros_like(r))
            w = r if float(r.sum()) > 0 else w
        c = torch.cumsum(w, 0)
        y = min(V - 1, int(torch.searchsorted(c, torch.tensor([ud[b]], dtype=torch.float64, device="cuda") * c[-1], right=True)))
        tau.append(a + 1)
        com.append(draft[b][:a] + [y] + [-1] * (m - a))
        last.append(y)
    return {"tau": _ints(tau), "committed": _ints(com), "next_anchor": _ints(last)}
