"""Cases of the operators around a drafted token tree.

Instead of one chain, a drafter may hand the target model a tree: several
candidates for a position, each with continuations of its own. The target runs
all nodes at once over its paged cache, draws a token behind every node, follows
the branch that the draws confirm and keeps that branch's rows of the cache.
Four operators:

  attention  nodes of a ragged batch of trees over the paged cache: each sees
             the context, its ancestors and itself (with the masks and positions
             that follow from the parents)
  sample     a token for every row of logits from given random numbers, after
             temperature, top-k, top-p and min-p; also the shaped distribution
  commit     the confirmed branch of each tree, its rows of every layer's pages
             moved behind the context
  pages      a cycle of the pages' bookkeeping: pages behind the kept positions
             released, sequences forked (full pages shared, the last one
             copied), pages for the next tree reserved

`run` computes a case in its plain form (elementary torch operations in 32
bits, in 64 where values sit next to a border) or, where `own` is true, by the
framework's calls. Lengths are a function of the case, values of the seed.
"""
import math
import random

import torch

own = False

PAGE = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    qwen = dict(hq=32, hkv=8, dh=128)          # Qwen3-8B heads
    tiny = dict(hq=4, hkv=4, dh=64)            # the tiny fp32 drafter's heads
    att = dict(op="attention", dtype="bf16", **qwen)
    vocab = 151936
    return [
        # one sequence's tree over a short context: latency
        dict(att, name="tree_B1_n64_ctx2048", batch=1, rows=64, rows_min=64, ctx=2048, ctx_min=2048),
        # the same over a long context: the cache's bytes
        dict(att, name="tree_B1_n64_ctx32768", batch=1, rows=64, rows_min=64, ctx=32768, ctx_min=32768),
        # a serving batch, trees and contexts of all sizes
        dict(att, name="tree_B16_ragged", batch=16, rows=64, rows_min=9, ctx=8192, ctx_min=512),
        # the tiny fp32 shapes, one sequence over an empty context
        dict(op="attention", dtype="f32", **tiny, name="tree_f32_tiny_B3", batch=3, rows=33, rows_min=1, ctx=900, ctx_min=0),
        # plain decoding of one sequence at usual settings: latency
        dict(op="sample", dtype="bf16", name="sample_1_top_k_top_p", rows=1, vocab=vocab, mode="top_k_top_p", probs=False),
        # the nodes of one tree, or a batch of requests with settings of their own
        dict(op="sample", dtype="f32", name="sample_64_mixed", rows=64, vocab=vocab, mode="mixed", probs=False),
        # 16 drafted blocks of 17 rows: the shaped distributions that their verification takes
        dict(op="sample", dtype="f32", name="sample_272_top_p_probs", rows=272, vocab=vocab, mode="top_p", probs=True),
        # the nodes of 16 trees
        dict(op="sample", dtype="bf16", name="sample_1024_mixed", rows=1024, vocab=vocab, mode="mixed", probs=False),
        # one tree, all layers of the target: latency
        dict(op="commit", dtype="bf16", name="commit_B1_L36", layers=36, hkv=8, dh=128, batch=1, rows=64, rows_min=64, ctx=300,
             ctx_min=300),
        dict(op="commit", dtype="bf16", name="commit_B32_L36", layers=36, hkv=8, dh=128, batch=32, rows=64, rows_min=9, ctx=400,
             ctx_min=10),
        # one prompt that goes on in four samples
        dict(op="pages", dtype="bf16", name="pages_B4_fork3", layers=36, hkv=8, dh=128, batch=4, forks=3, grow=64, ctx=1000,
             ctx_min=1000),
        # a serving batch, some of whose sequences branch
        dict(op="pages", dtype="bf16", name="pages_B128_fork24", layers=8, hkv=8, dh=128, batch=128, forks=24, grow=64, ctx=4000,
             ctx_min=1),
    ]


def _logint(rng, lo, hi):
    """An integer between lo and hi, even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "sample", "sample", "commit", "pages"])
    if op == "sample":
        vocab = _logint(rng, 1003, 200003)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=_logint(rng, 1, max(1, min(1024, 40000000 // vocab))), vocab=vocab,
                    mode=rng.choice(["mixed", "mixed", "top_p", "top_k_top_p", "plain"]), probs=rng.random() < 0.4)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hq, hkv, dh = rng.choice([(32, 8, 128), (32, 8, 128), (8, 2, 64), (4, 4, 64), (28, 4, 128), (10, 2, 128), (16, 1, 64)])
    c = dict(op=op, dtype=dtype, hkv=hkv, dh=dh)
    es = _bytes(dtype)
    if op == "attention":
        batch = _logint(rng, 1, 64)
        ctx = _logint(rng, 1, max(64, min(32768, (250000 if dtype == "bf16" else 60000) * 1024 // (hkv * dh) // batch)))
        # the padded plain form's scores, batch * hq * rows * (ctx + rows), are bounded
        rows = _logint(rng, 1, max(1, min(256 if dtype == "bf16" else 64, int(4e8 / (batch * hq * (ctx + 256))))))
        return dict(c, hq=hq, batch=batch, rows=rows, rows_min=rng.randint(1, rows), ctx=ctx, ctx_min=rng.randint(0, ctx))
    layers = _logint(rng, 1, 36)
    page = layers * hkv * PAGE * dh * es              # bytes of one page in one pool
    if op == "commit":
        batch, rows = _logint(rng, 1, max(1, min(64, int(1.5e9 / page / 4)))), _logint(rng, 2, 128)
        ctx = _logint(rng, 1, max(2, min(2000, int(1.5e9 / page / batch - 2) * PAGE)))
        return dict(c, layers=layers, batch=batch, rows=rows, rows_min=rng.randint(1, rows), ctx=ctx, ctx_min=rng.randint(0, ctx))
    batch = _logint(rng, 2, max(2, min(256, int(1.5e9 / page / 4))))
    ctx = _logint(rng, 1, max(2, min(8000, int(1.5e9 / page / batch - 2) * PAGE)))
    return dict(c, layers=layers, batch=batch, forks=rng.randint(1, max(1, batch // 4)), grow=rng.randint(1, 256), ctx=ctx,
                ctx_min=rng.randint(0, ctx))


# ------------------------------------------------------------------ inputs
def _lens(case):
    """(nodes, context) of each sequence: the longest of both first, the others spread over their ranges."""
    rows, rows_min = case.get("rows", 1), case.get("rows_min", 1)
    r = random.Random("%d %d %d %d %d" % (case["batch"], rows, rows_min, case["ctx"], case["ctx_min"]))
    n = [rows] + [r.randint(rows_min, rows) for _ in range(case["batch"] - 1)]
    c = [case["ctx"]] + [r.randint(case["ctx_min"], case["ctx"]) for _ in range(case["batch"] - 1)]
    if case["batch"] > 1 and case["ctx_min"] == 0:
        c[-1] = 0
    return n, c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & ((1 << 62) - 1))


def _normal(g, shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).add_(shift).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree(r, n):
    """Parents of a tree of n nodes in the order of their depth's discovery: long branches, a few candidates a node."""
    return [-1] + [max(0, i - 1 - int(r.expovariate(0.35))) for i in range(1, n)]


def _table(g, have, spare):
    """Pages of all sequences, scattered over the pool, and how many pages that takes."""
    n_pages = sum(have) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(have), max(have) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _settings(case, g, r):
    """Temperature, top-k, top-p and min-p of every row."""
    N, mode = case["rows"], case["mode"]
    t, k, p, m = [0.6] * N, [20] * N, [0.95] * N, [0.0] * N
    if mode == "plain":
        t, k, p = [1.0] * N, [0] * N, [1.0] * N
    if mode == "top_p":
        t, k, p = [0.7] * N, [0] * N, [0.95] * N
    if mode == "mixed":   # requests with settings of their own
        t = [r.choice([0.0, 0.3, 0.6, 0.7, 1.0, 1.2]) for _ in range(N)]
        k = [r.choice([0, 0, 1, 20, 50, 500]) for _ in range(N)]
        p = [r.choice([1.0, 0.8, 0.9, 0.95, 0.99]) for _ in range(N)]
        m = [r.choice([0.0, 0.0, 0.05, 0.1, 0.001]) for _ in range(N)]
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    return f(t), _ints(k), f(p), f(m)


def prepare(case, seed):
    g, r = _gen(seed), random.Random(int(seed))
    s = dict(case)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "sample":
        N, V = case["rows"], case["vocab"]
        # the r-th most likely token of a language model has a probability of about r^-a: a row's logits are a times exponential values
        x = torch.empty((N, V), device="cuda").exponential_(generator=g)
        a = torch.rand((N, 1), generator=g, device="cuda") * 0.8 + 1.0
        s["logits"] = x.mul_(a).sub_(6.0).to(DTYPES[case["dtype"]])
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _settings(case, g, r)
        s["u"] = torch.rand((N,), generator=g, device="cuda")
        s["tokens"] = torch.zeros(N, dtype=torch.int32, device="cuda")
        s["probs"] = torch.zeros((N, V), device="cuda") if case["probs"] else None
        return s
    n, ctx = _lens(case)
    B, hkv, dh, dt = case["batch"], case["hkv"], case["dh"], DTYPES[case["dtype"]]
    s["ctx_len"] = _ints(ctx)
    if case["op"] == "pages":
        # every sequence holds its pages and those of a tree that was not kept; the forked ones go where others have ended
        F = case["forks"]
        have = [(c + case["grow"] + PAGE - 1) // PAGE for c in ctx]
        s["table"], s["n_pages"] = _table(g, have, (case["grow"] // PAGE + 2) * F + 8)
        s["refs"] = torch.zeros(s["n_pages"], dtype=torch.int32, device="cuda")
        held = s["table"][s["table"] >= 0].long()
        s["refs"][held] = 1
        ends = r.sample(range(1, B), min(F, B - 1))
        s["dst"] = _ints(ends)
        goes = [b for b in range(B) if b not in set(ends)]
        s["src"] = _ints([goes[0]] + [r.choice(goes) for _ in ends[1:]])
        s["grow_by"] = torch.full((B,), case["grow"], dtype=torch.int32, device="cuda")
        s["k_pool"] = _normal(g, (case["layers"], s["n_pages"], hkv, PAGE, dh), dt)
        s["v_pool"] = _normal(g, (case["layers"], s["n_pages"], hkv, PAGE, dh), dt)
        # room for the longest of them everywhere
        most = (case["ctx"] + case["grow"] + PAGE - 1) // PAGE + 1
        s["table"] = torch.cat((s["table"], torch.full((B, max(0, most - s["table"].shape[1])), -1, dtype=torch.int32, device="cuda")), 1)
        return s
    T = sum(n)
    s["max_rows"], s["max_ctx"] = max(n), max(ctx)
    s["cu_rows"] = _ints([sum(n[:b]) for b in range(B + 1)])
    trees = [_tree(r, m) for m in n]
    s["parents"] = _ints([p for t in trees for p in t])
    s["table"], s["n_pages"] = _table(g, [(c + m + PAGE - 1) // PAGE for c, m in zip(ctx, n)], 3)
    layers = case.get("layers", 1)
    s["k_pool"] = _normal(g, (layers, s["n_pages"], hkv, PAGE, dh), dt)
    s["v_pool"] = _normal(g, (layers, s["n_pages"], hkv, PAGE, dh), dt)
    if case["op"] == "attention":
        s["q"] = _normal(g, (T, case["hq"], dh), dt, scale=1.5)      # rotated queries, a little peaked
        s["out"] = torch.zeros((T, case["hq"], dh), dtype=dt, device="cuda")
        s["mask"] = torch.zeros((T, (max(n) + 31) // 32), dtype=torch.int32, device="cuda")
        s["positions"] = torch.zeros(T, dtype=torch.int32, device="cuda")
        return s
    # the target draws one of a node's candidates three times of four
    tokens, drawn = [], []
    for t in trees:
        mine = [r.randrange(151936) for _ in t]
        kids = [[c for c in range(len(t)) if t[c] == i] for i in range(len(t))]
        drawn += [mine[r.choice(k)] if k and r.random() < 0.75 else r.randrange(151936) for k in kids]
        tokens += mine
    s["tokens"], s["drawn"] = _ints(tokens), _ints(drawn)
    s["max_path"] = 24
    s["tau"], s["next_anchor"] = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    s["committed"], s["path"] = (torch.zeros((B, s["max_path"]), dtype=torch.int32, device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------------ plain forms
def _places(s):
    """Sequence and number of each packed node, and which of the padded places [B, R] hold one."""
    cu, t = s["cu_rows"].long(), torch.arange(s["parents"].numel(), device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, t - cu[seq]


def _ancestors(s, seq, row):
    """[B, R, R]: whether j is i or an ancestor of it."""
    B, R = s["batch"], s["max_rows"]
    up = torch.zeros((B, R, R), device="cuda")
    p = s["parents"].long()
    up[seq, row, p.clamp(min=0)] = (p >= 0).float()
    eye = torch.eye(R, device="cuda").expand(B, R, R)
    # (I - up)^-1 = I + up + up^2 + ...: whole numbers, one for every ancestor
    return torch.linalg.solve_triangular(eye - up, eye, upper=False, unitriangular=True) > 0.5


def _plain_attention(s):
    hq, hkv, dh, B, T = s["hq"], s["hkv"], s["dh"], s["batch"], s["q"].shape[0]
    G, R, W = hq // hkv, s["max_rows"], s["mask"].shape[1]
    seq, row = _places(s)
    sees = _ancestors(s, seq, row)
    s["positions"].copy_(s["ctx_len"][seq] + sees[seq, row].sum(-1) - 1)
    bits = torch.zeros((T, W * 32), dtype=torch.long, device="cuda")
    bits[:, :R] = sees[seq, row].long()
    words = (bits.view(T, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    s["mask"].copy_(torch.where(words >= 1 << 31, words - (1 << 32), words))
    table = s["table"].long().clamp(min=0)
    n_keys = table.shape[1] * PAGE

    def rows_of(pool):          # [B, hkv, keys, dh] in 32 bits
        return pool[0][table].transpose(1, 2).reshape(B, hkv, n_keys, dh).float()

    keys, ctx = torch.arange(n_keys, device="cuda"), s["ctx_len"].long()
    node = (keys - ctx[:, None]).clamp(0, R - 1)[:, None].expand(B, R, n_keys)
    n = s["cu_rows"].long().diff()
    inside = (keys >= ctx[:, None]) & (keys < (ctx + n)[:, None])
    seen = (keys < ctx[:, None])[:, None] | (inside[:, None] & sees.gather(2, node))
    q = torch.zeros((B, R, hq, dh), device="cuda")
    q[seq, row] = s["q"].float()
    q = q.view(B, R, hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * R, dh)
    x = torch.matmul(q, rows_of(s["k_pool"]).transpose(2, 3)) * (dh ** -0.5)
    x = x.view(B, hkv, G, R, n_keys).masked_fill_(~seen[:, None, None], -math.inf).view(B, hkv, G * R, n_keys)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    v = rows_of(s["v_pool"]).masked_fill_((keys >= (ctx + n)[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, hkv, G, R, dh).permute(0, 3, 1, 2, 4).reshape(B, R, hq, dh)
    s["out"].copy_(o[seq, row])
    return {"out": s["out"], "mask": s["mask"], "positions": s["positions"]}


def _plain_sample(s):
    x, V = s["logits"].float(), s["vocab"]
    t, k = s["temperature"].double()[:, None], s["top_k"].long()[:, None]
    best, order = x.sort(dim=-1, descending=True, stable=True)          # equal ones in their order
    # 64 bits: weights are compared with borders
    w = torch.exp((best.double() - best[:, :1].double()) / torch.where(t > 0, t, torch.ones_like(t)))
    rank = torch.arange(V, device="cuda")[None]
    k = torch.where(k > 0, k, torch.full_like(k, V)).clamp(max=V)
    k = torch.where(t > 0, k, torch.ones_like(k))
    w = torch.where(rank < k, w, 0.0)
    before = w.cumsum(-1)
    total = before[:, -1:].clone()
    before -= w
    p = s["top_p"].double()[:, None]
    keep = (rank < k) & ((before < p * total) | (p >= 1)) & (w >= s["min_p"].double()[:, None]) | (rank == 0)
    w = torch.where(keep, w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)
    c = w.cumsum(-1)
    y = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(-1).clamp(max=V - 1)
    s["tokens"].copy_(y)
    if s["probs"] is None:
        return {"tokens": s["tokens"]}
    s["probs"].copy_(w / c[:, -1:])
    return {"tokens": s["tokens"], "probs": s["probs"]}


def _plain_commit(s):
    B, R, P = s["batch"], s["max_rows"], s["max_path"]
    seq, row = _places(s)
    cu, par = s["cu_rows"].long(), s["parents"].long()
    up = cu[seq] + par.clamp(min=0)
    hit = torch.zeros((B, R), dtype=torch.bool, device="cuda")
    hit[seq, row] = (par < 0) & (row == 0) | (par >= 0) & (s["tokens"] == s["drawn"][up])
    # of several candidates with the drawn token the first one counts
    parent = torch.full((B, R), -2, dtype=torch.long, device="cuda")
    parent[seq, row] = par
    j = torch.arange(R, device="cuda")
    earlier = (parent[:, :, None] == parent[:, None, :]) & hit[:, None, :] & (j[None, :] < j[:, None])
    hit &= ~earlier.any(-1)
    on = ~(_ancestors(s, seq, row) & ~hit[:, None, :]).any(-1)          # the node and all its ancestors
    here = torch.zeros((B, R), dtype=torch.bool, device="cuda")
    here[seq, row] = True
    on &= here
    nth = on.long().cumsum(1) - 1
    on &= nth < P
    s["tau"].copy_(on.sum(1))
    path = torch.full((B, P + 1), -1, dtype=torch.long, device="cuda")
    path.scatter_(1, torch.where(on, nth, P), torch.where(on, j, -1))
    path = path[:, :P]
    s["path"].copy_(path)
    tau = s["tau"].long()
    at = cu[:-1, None] + path.clamp(min=0)
    last = cu[:-1] + path.gather(1, (tau - 1)[:, None])[:, 0]
    s["next_anchor"].copy_(s["drawn"][last])
    i = torch.arange(P, device="cuda")
    nxt = s["tokens"][at].roll(-1, 1)
    com = torch.where(i < (tau - 1)[:, None], nxt, torch.where(i == (tau - 1)[:, None], s["next_anchor"][:, None], -1))
    s["committed"].copy_(com)
    # rows of the cache: every row goes to itself where there is nothing to move
    frm = s["ctx_len"].long()[:, None] + torch.where(path >= 0, path, 0)
    to = s["ctx_len"].long()[:, None] + torch.where(path >= 0, i, 0)
    table = s["table"].long()
    fp, tp = table.gather(1, frm // PAGE), table.gather(1, to // PAGE)
    for_k, for_v = s["k_pool"][:, fp, :, frm % PAGE], s["v_pool"][:, fp, :, frm % PAGE]
    s["k_pool"][:, tp, :, to % PAGE] = for_k
    s["v_pool"][:, tp, :, to % PAGE] = for_v
    return {m: s[m] for m in ("tau", "committed", "path", "next_anchor", "k_pool", "v_pool")}


def _count(refs, pages, by):
    """refs[page] += by for every page of a list, -1 for none."""
    held = (pages >= 0).to(torch.int32) * by
    return refs.index_add_(0, pages.clamp(min=0).long().reshape(-1), held.reshape(-1))


def _plain_pages(s):
    table, refs, L = s["table"], s["refs"], s["ctx_len"]
    col = torch.arange(table.shape[1], device="cuda")[None]
    # what lies behind the kept positions
    behind = col >= ((L + PAGE - 1) // PAGE)[:, None]
    _count(refs, torch.where(behind, table, -1), -1)
    table.masked_fill_(behind, -1)
    # forks: the full pages are shared, the last one is a page of its own
    src, dst = s["src"].long(), s["dst"].long()
    _count(refs, table[dst], -1)
    n = L[src]
    full = (n // PAGE)[:, None]
    rows = torch.where(col < full, table[src], -1)
    _count(refs, rows, 1)
    part = n % PAGE > 0
    free = torch.argsort((refs > 0).to(torch.int32), stable=True).to(torch.int32)          # the free ones, lowest first
    mine = free[(part.long().cumsum(0) - 1).clamp(min=0)]
    rows = torch.where((col == full) & part[:, None], mine[:, None], rows)
    frm = table[src].gather(1, full.long().clamp(max=table.shape[1] - 1))[:, 0].long()
    table[dst] = rows
    _count(refs, torch.where(part, mine, -1), 1)
    L[dst] = n
    line = torch.arange(PAGE, device="cuda")
    for_copy = (line[None] < (n % PAGE)[:, None])[None, :, None, :, None]
    # nothing to copy: a page that nobody writes (the first sequence's) goes to itself, as it is
    idle = table[0, 0].long()
    frm, to = torch.where(part, frm, idle), torch.where(part, mine.long(), idle)
    s["k_pool"][:, to] = torch.where(for_copy, s["k_pool"][:, frm], s["k_pool"][:, to])
    s["v_pool"][:, to] = torch.where(for_copy, s["v_pool"][:, frm], s["v_pool"][:, to])
    # pages for the next nodes
    miss = (table < 0) & (col < ((L + s["grow_by"] + PAGE - 1) // PAGE)[:, None])
    nth = miss.reshape(-1).long().cumsum(0) - 1
    free = torch.argsort((refs > 0).to(torch.int32), stable=True).to(torch.int32)
    new = free[nth.clamp(0, free.numel() - 1)].view(table.shape)
    new = torch.where(miss, new, -1)
    table.copy_(torch.where(miss, new, table))
    _count(refs, new, 1)
    return {m: s[m] for m in ("table", "refs", "ctx_len", "k_pool", "v_pool")}


# ------------------------------------------------------------------ the framework's calls
def _handles(s):
    """What a program keeps beside its tensors: the layout, the page view, the scratch; made once for a state."""
    import block_diffusion_drafter_gb300 as dfl
    if "lib" not in s:
        s["lib"] = dfl
        if s["op"] != "sample":
            s["heads"] = dfl.make_heads(s.get("layers", 1), s.get("hq", s["hkv"]), s["hkv"], s["dh"],
                                        dtype=dfl.BF16 if s["dtype"] == "bf16" else dfl.F32)
            s["view"] = dfl.KvPages(s["k_pool"], s["v_pool"], s["table"])
        if s["op"] == "attention":
            s["ws"] = dfl.ChunkWorkspace(s["heads"])
    return s["lib"]


def run(s):
    op = s["op"]
    if not own:
        return {"attention": _plain_attention, "sample": _plain_sample, "commit": _plain_commit, "pages": _plain_pages}[op](s)
    dfl = _handles(s)
    if op == "attention":
        dfl.dflash_tree_masks(s["parents"], s["cu_rows"], s["ctx_len"], s["mask"], s["positions"], s["status"])
        dfl.dflash_attention_tree_paged(s["heads"], s["q"], s["cu_rows"], s["ctx_len"], s["max_rows"], s["max_ctx"], 0, s["view"],
                                        s["mask"], s["out"], s["status"], s["ws"])
        return {"out": s["out"], "mask": s["mask"], "positions": s["positions"]}
    if op == "sample":
        dfl.dflash_sample(s["logits"], s["u"], s["tokens"], s["status"], temperature=s["temperature"], top_k=s["top_k"],
                          top_p=s["top_p"], min_p=s["min_p"], probs=s["probs"])
        return {"tokens": s["tokens"]} if s["probs"] is None else {"tokens": s["tokens"], "probs": s["probs"]}
    if op == "commit":
        dfl.dflash_verify_tree(s["tokens"], s["parents"], s["drawn"], s["cu_rows"], s["tau"], s["committed"], s["path"],
                               s["next_anchor"], s["status"], heads=s["heads"], ctx_len=s["ctx_len"], pages=s["view"])
        return {m: s[m] for m in ("tau", "committed", "path", "next_anchor", "k_pool", "v_pool")}
    dfl.dflash_pages_release(s["view"], s["refs"], s["ctx_len"], s["status"])
    dfl.dflash_pages_fork(s["heads"], s["view"], s["refs"], s["ctx_len"], s["src"], s["dst"], s["status"])
    dfl.dflash_pages_reserve(s["view"], s["refs"], s["ctx_len"] + s["grow_by"], s["status"])
    return {m: s[m] for m in ("table", "refs", "ctx_len", "k_pool", "v_pool")}


# ------------------------------------------------------------------ work
def _bytes(name):
    return 2 if name == "bf16" else 4


def work(case):
    es = _bytes(case["dtype"])
    if case["op"] == "sample":
        N, V = case["rows"], case["vocab"]
        return {"bytes": N * (V * (es + (4.0 if case["probs"] else 0.0)) + 24.0), "flops": 2.0 * N * V}
    n, ctx = _lens(case)
    B, hkv, dh = case["batch"], case["hkv"], case["dh"]
    if case["op"] == "attention":
        T, hq = sum(n), case["hq"]
        keys = sum(c + m for c, m in zip(ctx, n))
        # a node sees the context and a branch, of the length that such trees have
        seen = sum(m * (c + 1 + m / 4.0) for c, m in zip(ctx, n))
        return {"bytes": 2.0 * keys * hkv * dh * es + 2.0 * T * hq * dh * es + T * (12 + (max(n) + 31) // 32 * 4),
                "flops": 4.0 * seen * hq * dh}
    row = 2.0 * 2.0 * case["layers"] * hkv * dh * es            # one position, read and written
    if case["op"] == "commit":
        # the anchor stays where it is; three drafts of four are confirmed, as far as a branch goes
        return {"bytes": sum(2.0 * min(1.0, m / 8.0) for m in n) * row + sum(n) * 12.0 + B * 100 * 4.0, "flops": 0.0}
    return {"bytes": case["forks"] * (PAGE / 2) * row + sum((c + case["grow"]) // PAGE + 1 for c in ctx) * 12.0, "flops": 0.0}


# ------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "sample": _exact_sample, "commit": _exact_commit, "pages": _exact_pages}[case["op"]](s, case)


def _branch(parents, i):
    """Node i and its ancestors."""
    got = []
    while i >= 0:
        got.append(i)
        i = parents[i]
    return got


def _exact_attention(s, case):
    n, ctx = _lens(case)
    hq, hkv, dh = s["hq"], s["hkv"], s["dh"]
    if sum(m * (c + m) for c, m in zip(ctx, n)) * hq * dh * 4 > 2e11:
        return None
    out, first = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    mask, positions, W = [], [], s["mask"].shape[1]
    for b in range(s["batch"]):
        keys, par = ctx[b] + n[b], s["parents"][first:first + n[b]].tolist()
        hidden = torch.full((n[b], keys), -math.inf, dtype=torch.float64)
        hidden[:, :ctx[b]] = 0.0
        for i in range(n[b]):
            up = _branch(par, i)
            hidden[i, [ctx[b] + j for j in up]] = 0.0
            positions.append(ctx[b] + len(up) - 1)
            words = [sum(1 << (j % 32) for j in up if j // 32 == w) for w in range(W)]
            mask.append([w - (1 << 32) if w >> 31 else w for w in words])
        hidden = hidden.cuda()
        pages = s["table"][b, : (keys + PAGE - 1) // PAGE].long()
        for h in range(hkv):
            k = s["k_pool"][0, pages, h].reshape(-1, dh)[:keys].double()
            v = s["v_pool"][0, pages, h].reshape(-1, dh)[:keys].double()
            for i in range(h * hq // hkv, (h + 1) * hq // hkv):
                x = s["q"][first:first + n[b], i].double() @ k.T / math.sqrt(dh)
                out[first:first + n[b], i] = torch.softmax(x + hidden, -1) @ v
        first += n[b]
    return {"out": out, "mask": _ints(mask), "positions": _ints(positions)}


def _exact_sample(s, case):
    N, V = case["rows"], case["vocab"]
    tokens, probs = [], torch.zeros((N, V), dtype=torch.float64, device="cuda") if case["probs"] else None
    for i in range(N):
        x = s["logits"][i].double()
        T, k, p, m, u = (float(s[key][i]) for key in ("temperature", "top_k", "top_p", "min_p", "u"))
        if T <= 0:
            x, T, k = torch.where(torch.arange(V, device="cuda") == x.argmax(), x, -math.inf), 1.0, 1
        z = torch.softmax(x / T, -1)
        # the tokens from the most likely one on, of equal ones the first one first
        at = torch.argsort(-x, stable=True)[: int(k) if 0 < k < V else V]
        q = z[at] / z[at].sum()
        if p < 1.0:
            at = at[: 1 + int((q.cumsum(0)[:-1] < p).sum())]
        at = at[z[at] >= m * z[at[0]]]
        kept = torch.zeros(V, dtype=torch.float64, device="cuda")
        kept[at] = z[at] / z[at].sum()
        c = kept.cumsum(0)
        tokens.append(min(V - 1, int(torch.searchsorted(c, (u * c[-1]).reshape(1), right=True))))
        if probs is not None:
            probs[i] = kept
    out = {"tokens": _ints(tokens)}
    return out if probs is None else {**out, "probs": probs}


def _exact_commit(s, case):
    n, ctx = _lens(case)
    P, first = s["max_path"], 0
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    tau, com, paths, last = [], [], [], []
    for b in range(case["batch"]):
        par, tok, drawn = (s[key][first:first + n[b]].tolist() for key in ("parents", "tokens", "drawn"))
        at = [0]
        while len(at) < P:
            nxt = [c for c in range(n[b]) if par[c] == at[-1] and tok[c] == drawn[at[-1]]]
            if not nxt:
                break
            at.append(nxt[0])
        tau.append(len(at))
        com.append([tok[i] for i in at[1:]] + [drawn[at[-1]]] + [-1] * (P - len(at)))
        paths.append(at + [-1] * (P - len(at)))
        last.append(drawn[at[-1]])
        page = s["table"][b].tolist()
        for j, i in enumerate(at):      # a row moves down, behind rows that have moved
            f, t = ctx[b] + i, ctx[b] + j
            for pool in (kp, vp):
                pool[:, page[t // PAGE], :, t % PAGE] = pool[:, page[f // PAGE], :, f % PAGE].clone()
        first += n[b]
    return {"tau": _ints(tau), "committed": _ints(com), "path": _ints(paths), "next_anchor": _ints(last), "k_pool": kp, "v_pool": vp}


def _exact_pages(s, case):
    table, refs, length = s["table"].tolist(), s["refs"].tolist(), s["ctx_len"].tolist()
    kp, vp = s["k_pool"].double(), s["v_pool"].double()

    def drop(b, keep):
        for j in range((keep + PAGE - 1) // PAGE, len(table[b])):
            if table[b][j] >= 0:
                refs[table[b][j]] -= 1
            table[b][j] = -1

    for b in range(case["batch"]):
        drop(b, length[b])
    pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
    for _, d in pairs:
        drop(d, 0)
    for f, d in pairs:
        for j in range(length[f] // PAGE):
            table[d][j] = table[f][j]
            refs[table[d][j]] += 1
    for f, d in pairs:
        length[d], j, left = length[f], length[f] // PAGE, length[f] % PAGE
        if left:
            table[d][j] = refs.index(0)
            refs[table[d][j]] = 1
            for pool in (kp, vp):
                pool[:, table[d][j], :, :left] = pool[:, table[f][j], :, :left]
    for b in range(case["batch"]):
        for j in range((length[b] + case["grow"] + PAGE - 1) // PAGE):
            if table[b][j] < 0:
                table[b][j] = refs.index(0)
                refs[table[b][j]] = 1
    return {"table": _ints(table), "refs": _ints(refs), "ctx_len": _ints(length), "k_pool": kp, "v_pool": vp}
