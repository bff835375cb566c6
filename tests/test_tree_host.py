"""Refusals of the calls around a drafted tree, all decided on the host before
any launch, and the oracle's own definitions against plain counting (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import tree_ref as tt

FAKE = 1 << 20     # a 16-byte aligned address; nothing is dereferenced


@pytest.fixture(scope="module")
def heads(lib):
    return lib.make_heads(2, 8, 2, 128)


def pages_of(lib, **kw):
    p = lib.KvPages.__new__(lib.KvPages)
    ctypes.Structure.__init__(p, **{**dict(k_pool=FAKE, v_pool=FAKE + (1 << 19), page_table=FAKE, n_pages=4, pages_per_seq=3), **kw})
    return p


def ref(x):
    return ctypes.byref(x) if x is not None else None


def refused(lib, call, cases):
    for kw, want in cases:
        assert call(**kw) == getattr(lib, "ERR_" + want), kw


def test_masks(lib):
    def call(**kw):
        a = {**dict(par=FAKE, cu=FAKE, ctx=FAKE, B=2, T=9, words=1, mask=FAKE, pos=FAKE, st=FAKE), **kw}
        return lib.load().dflash_tree_masks(a["par"], a["cu"], a["ctx"], a["B"], a["T"], a["words"], a["mask"], a["pos"], a["st"],
                                            None, None)

    assert call(T=0) == lib.OK and call(B=0) == lib.OK
    refused(lib, call, [({n: None}, "INVALID_ARG") for n in ("par", "cu", "ctx", "mask", "st")] + [
        (dict(T=-1), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"), (dict(words=0), "INVALID_ARG"), (dict(T=2 ** 31 - 1), "TOO_LARGE")])


def test_attention(lib, heads):
    def call(h=heads, **kw):
        a = {**dict(q=FAKE, ldq=1024, cu=FAKE, ctx=FAKE, B=2, T=5, rows=5, hint=100, layer=1, pages=pages_of(lib), mask=FAKE, words=1,
                    scale=0.0, out=2 * FAKE, ldo=1024, st=FAKE, ws=FAKE, nb=1 << 40), **kw}
        return lib.load().dflash_attention_tree_paged(
            ref(h), a["q"], a["ldq"], a["cu"], a["ctx"], a["B"], a["T"], a["rows"], a["hint"], a["layer"], ref(a["pages"]), a["mask"],
            a["words"], a["scale"], a["out"], a["ldo"], a["st"], a["ws"], a["nb"], None, None)

    assert call(T=0) == lib.OK and call(B=0, mask=None) == lib.OK
    refused(lib, call, [({n: None}, "INVALID_ARG") for n in ("q", "cu", "ctx", "pages", "mask", "out", "st", "h")] + [
        (dict(words=0), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(hint=-1), "INVALID_ARG"), (dict(layer=2), "INVALID_ARG"),
        (dict(scale=float("nan")), "INVALID_ARG"), (dict(out=FAKE), "INVALID_ARG"), (dict(ldq=1028), "ALIGN"), (dict(q=FAKE + 2), "ALIGN"),
        (dict(ws=None), "WORKSPACE"), (dict(nb=1000), "WORKSPACE"), (dict(T=1 << 30), "TOO_LARGE")])


def test_sample(lib):
    def call(**kw):
        a = {**dict(x=FAKE, dt=lib.F32, ld=100, N=3, V=100, t=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, tok=FAKE, probs=2 * FAKE, st=FAKE), **kw}
        return lib.load().dflash_sample(a["x"], a["dt"], a["ld"], a["N"], a["V"], a["t"], a["k"], a["p"], a["m"], a["u"], a["tok"],
                                        a["probs"], a["st"], None, None)

    assert call(N=0) == lib.OK
    refused(lib, call, [
        (dict(dt=2), "DTYPE"), (dict(N=-1), "INVALID_ARG"), (dict(V=0), "INVALID_ARG"), (dict(ld=99), "INVALID_ARG"),
        (dict(x=None), "INVALID_ARG"), (dict(st=None), "INVALID_ARG"), (dict(u=None), "INVALID_ARG"), (dict(tok=None), "INVALID_ARG"),
        (dict(u=None, tok=None, probs=None), "INVALID_ARG"), (dict(probs=FAKE), "INVALID_ARG"), (dict(x=FAKE + 2), "ALIGN"),
        (dict(probs=FAKE + 1), "ALIGN"), (dict(x=FAKE + 1, dt=lib.BF16), "ALIGN"), (dict(N=(1 << 20) + 1), "TOO_LARGE"),
        (dict(V=(1 << 19) + 1, ld=1 << 20), "TOO_LARGE")])


def test_verify(lib, heads):
    def call(h=heads, **kw):
        a = {**dict(tok=FAKE, par=FAKE, drawn=FAKE, cu=FAKE, ctx=FAKE, B=2, T=9, P=4, pages=pages_of(lib), tau=FAKE, com=FAKE, path=FAKE,
                    nxt=FAKE, st=FAKE), **kw}
        return lib.load().dflash_verify_tree(ref(h), a["tok"], a["par"], a["drawn"], a["cu"], a["ctx"], a["B"], a["T"], a["P"],
                                             ref(a["pages"]), a["tau"], a["com"], a["path"], a["nxt"], a["st"], None, None)

    assert call(B=0) == lib.OK and call(B=0, h=None, pages=None, ctx=None) == lib.OK
    refused(lib, call, [({n: None}, "INVALID_ARG") for n in ("tok", "par", "drawn", "cu", "ctx", "tau", "com", "path", "nxt", "st", "h")] + [
        (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(P=0), "INVALID_ARG"), (dict(h=lib.make_heads(1, 3, 2, 64)), "SHAPE"),
        (dict(pages=pages_of(lib, n_pages=0)), "INVALID_ARG"), (dict(pages=pages_of(lib, page_table=None)), "INVALID_ARG"),
        (dict(pages=pages_of(lib, pages_per_seq=1 << 25)), "INVALID_ARG"), (dict(pages=pages_of(lib, v_pool=FAKE)), "INVALID_ARG"),
        (dict(pages=pages_of(lib, k_pool=FAKE + 8)), "ALIGN")])


def test_pages(lib, heads):
    def book(name):
        def call(**kw):
            a = {**dict(pages=pages_of(lib), refs=FAKE, n=FAKE, B=2, st=FAKE), **kw}
            return getattr(lib.load(), name)(ref(a["pages"]), a["refs"], a["n"], a["B"], a["st"], None, None)
        return call

    for name in ("dflash_pages_release", "dflash_pages_reserve"):
        assert book(name)(B=0) == lib.OK
        refused(lib, book(name), [({n: None}, "INVALID_ARG") for n in ("pages", "refs", "n", "st")] + [
            (dict(B=-1), "INVALID_ARG"), (dict(pages=pages_of(lib, n_pages=0)), "INVALID_ARG"),
            (dict(pages=pages_of(lib, n_pages=2 ** 31 - 1)), "INVALID_ARG"), (dict(pages=pages_of(lib, pages_per_seq=0)), "INVALID_ARG"),
            (dict(pages=pages_of(lib, page_table=None)), "INVALID_ARG")])
    assert book("dflash_pages_reserve")(B=4097) == lib.ERR_TOO_LARGE

    def fork(h=heads, **kw):
        a = {**dict(pages=pages_of(lib), refs=FAKE, ctx=FAKE, seqs=4, src=FAKE, dst=FAKE, n=2, st=FAKE), **kw}
        return lib.load().dflash_pages_fork(ref(h), ref(a["pages"]), a["refs"], a["ctx"], a["seqs"], a["src"], a["dst"], a["n"], a["st"],
                                            None, None)

    assert fork(n=0) == lib.OK
    refused(lib, fork, [({n: None}, "INVALID_ARG") for n in ("h", "pages", "refs", "ctx", "src", "dst", "st")] + [
        (dict(n=-1), "INVALID_ARG"), (dict(seqs=-1), "INVALID_ARG"), (dict(n=1025), "TOO_LARGE"),
        (dict(pages=pages_of(lib, v_pool=FAKE)), "INVALID_ARG"), (dict(pages=pages_of(lib, v_pool=FAKE + 4)), "ALIGN")])


def test_the_binding_refuses_what_the_library_cannot_see(lib, heads):
    i32, bf = torch.int32, torch.bfloat16
    one = lambda *s: torch.zeros(s, dtype=i32)  # noqa: E731
    pool = torch.zeros((2, 4, 2, 128, 128), dtype=bf)
    view = lib.KvPages(pool, pool.clone(), one(2, 2))
    st, cu, ctx = one(1), one(3), one(2)

    def fails(f, *status):
        with pytest.raises(lib.DFlashError) as e:
            f()
        assert e.value.status in [getattr(lib, "ERR_" + s) for s in status], e.value

    masks = lambda par=one(4), cu=cu, ctx=ctx, mask=one(4, 1), pos=one(4): lib.dflash_tree_masks(par, cu, ctx, mask, pos, st)  # noqa: E731
    for kw, want in [(dict(par=one(4).long()), "DTYPE"), (dict(mask=one(3, 1)), "SHAPE"), (dict(mask=one(4)), "SHAPE"),
                     (dict(mask=one(4, 2)[:, :1]), "SHAPE"), (dict(mask=torch.zeros(4, 1)), "DTYPE"), (dict(pos=one(3)), "SHAPE"),
                     (dict(ctx=one(1)), "SHAPE"), (dict(ctx=None), "INVALID_ARG")]:
        fails(lambda: masks(**kw), want)

    q = torch.zeros((4, 8, 128), dtype=bf)

    class NoScratch:
        ptr, nbytes = None, 0

    att = lambda q=q, out=q.clone(), mask=one(4, 1), pages=view: lib.dflash_attention_tree_paged(  # noqa: E731
        heads, q, cu, ctx, 4, 0, 0, pages, mask, out, st, NoScratch())
    fails(att, "WORKSPACE")                            # all else is right
    for kw, want in [(dict(mask=one(3, 1)), "SHAPE"), (dict(mask=one(4, 1).long()), "DTYPE"), (dict(out=q[:3]), "SHAPE"),
                     (dict(q=q.float()), "DTYPE"), (dict(q=None), "INVALID_ARG"),
                     (dict(pages=lib.KvPages(pool[:1], pool[:1], one(2, 2))), "SHAPE")]:
        fails(lambda: att(**kw), want)

    x, f = torch.zeros((3, 50)), lambda n=3: torch.zeros(n)  # noqa: E731
    sample = lambda x=x, u=f(), tok=one(3), st=None, **kw: lib.dflash_sample(x, u, tok, st, **kw)  # noqa: E731
    fails(sample, "INVALID_ARG")                       # no status word; all else is right
    for kw, want in [(dict(x=x.double()), "DTYPE"), (dict(x=x[0]), "SHAPE"), (dict(x=x.t()), "SHAPE"), (dict(u=f(2)), "SHAPE"),
                     (dict(u=f().double()), "DTYPE"), (dict(tok=one(2)), "SHAPE"), (dict(tok=one(3).long()), "DTYPE"),
                     (dict(temperature=f(2)), "SHAPE"), (dict(top_k=f()), "DTYPE"), (dict(top_p=one(3)), "DTYPE"),
                     (dict(min_p=f(2)), "SHAPE"), (dict(probs=torch.zeros((3, 49))), "SHAPE"), (dict(probs=torch.zeros((3, 50), dtype=bf)), "DTYPE"),
                     (dict(tok=None), "INVALID_ARG"), (dict(u=None), "INVALID_ARG")]:
        fails(lambda: sample(**kw), want)

    ver = lambda tok=one(4), par=one(4), drawn=one(4), tau=one(2), com=one(2, 5), path=one(2, 5), nxt=one(2), st=st, **kw: (  # noqa: E731
        lib.dflash_verify_tree(tok, par, drawn, cu, tau, com, path, nxt, st, **kw))
    for kw, want in [(dict(par=one(3)), "SHAPE"), (dict(drawn=one(4).long()), "DTYPE"), (dict(tau=one(1)), "SHAPE"),
                     (dict(com=one(2, 4)), "SHAPE"), (dict(com=one(1, 5)), "SHAPE"), (dict(path=one(1, 5)), "SHAPE"),
                     (dict(pages=view), "INVALID_ARG"), (dict(pages=view, heads=heads), "INVALID_ARG"),
                     (dict(pages=view, heads=heads, ctx_len=one(1)), "SHAPE"),
                     (dict(pages=view, heads=lib.make_heads(2, 8, 1, 128), ctx_len=ctx), "SHAPE")]:
        fails(lambda: ver(**kw), want)

    for call in (lib.dflash_pages_release, lib.dflash_pages_reserve):
        for pages, refs, n, want in [(view, one(3), one(2), "SHAPE"), (view, one(4).long(), one(2), "DTYPE"), (view, one(4), one(3), "SHAPE"),
                                     (view, one(4), one(2).long(), "DTYPE"), (lib.KvPages(pool, pool, one(2, 2).long()), one(4), one(2), "SHAPE")]:
            fails(lambda: call(pages, refs, n, st), want)
    fork = lambda refs=one(4), ctx=ctx, src=one(2), dst=one(2): lib.dflash_pages_fork(heads, view, refs, ctx, src, dst, st)  # noqa: E731
    for kw, want in [(dict(refs=one(3)), "SHAPE"), (dict(ctx=one(3)), "SHAPE"), (dict(dst=one(1)), "SHAPE"), (dict(src=one(2).long()), "DTYPE")]:
        fails(lambda: fork(**kw), want)


# ------------------------------------------------------------------ the oracle's definitions
def test_wide_masks_and_overlapping_rows_are_refused(lib, heads):
    """Masks whose bits pass 31 bits, and distributions written over logits that are still read."""
    word = lib.load().dflash_tree_masks(FAKE, FAKE, FAKE, 1, 1, 1 << 26, FAKE, FAKE, FAKE, None, None)
    tree = lib.load().dflash_attention_tree_paged(ref(heads), FAKE, 1024, FAKE, FAKE, 1, 1, 1, 9, 0, ref(pages_of(lib)), FAKE, 1 << 26,
                                                  0.0, 2 * FAKE, 1024, FAKE, FAKE, 1 << 40, None, None)
    assert word == tree == lib.ERR_TOO_LARGE

    def sample(probs, dt=lib.F32, ld=100):
        return lib.load().dflash_sample(FAKE, dt, ld, 3, 100, None, None, None, None, FAKE, FAKE, probs, FAKE, None, None)

    for probs in (FAKE, FAKE + 4, FAKE + 1196, FAKE - 1196):
        assert sample(probs) == lib.ERR_INVALID_ARG, probs - FAKE
    assert sample(FAKE + 596, lib.BF16) == sample(FAKE + 2000, ld=250) == lib.ERR_INVALID_ARG
    # side by side: nothing to refuse (no GPU of the right kind here, or these addresses would be read)
    if not torch.cuda.is_available():
        for call in (sample(FAKE + 1200), sample(FAKE - 1200), sample(FAKE + 600, lib.BF16)):
            assert call not in (lib.ERR_INVALID_ARG, lib.ERR_ALIGN, lib.OK)


def test_an_empty_batch_needs_no_mask(lib, heads):
    """A step without any node: its mask is [0, 0]. Nothing is launched."""
    call, tree = lib.load().dflash_tree_masks, lib.load().dflash_attention_tree_paged
    for B, T in ((0, 0), (2, 0), (0, 3)):
        for words in (0, 1, 1 << 26):
            assert call(None, None, None, B, T, words, None, None, None, None, None) == lib.OK, (B, T, words)
            assert tree(ref(heads), None, 0, None, None, B, T, 0, 0, 0, None, None, words, 0.0, None, 0, None, None, 0, None, None) == lib.OK
        for words in (-1, -2 ** 31):
            assert call(FAKE, FAKE, FAKE, B, T, words, FAKE, None, FAKE, None, None) == lib.ERR_INVALID_ARG
    assert call(FAKE, FAKE, FAKE, -1, 0, 0, FAKE, None, FAKE, None, None) == lib.ERR_INVALID_ARG
    assert tree(ref(heads), None, 0, None, None, 0, 0, 0, 0, 2, None, None, 0, 0.0, None, 0, None, None, 0, None, None) == lib.ERR_INVALID_ARG
    assert tree(None, None, 0, None, None, 0, 0, 0, 0, 0, None, None, 0, 0.0, None, 0, None, None, 0, None, None) == lib.ERR_INVALID_ARG
    if torch.cuda.is_available():
        return          # the binding wants its operands on the device then (tests/test_gpu_tree_attention.py)
    one = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    lib.dflash_tree_masks(one(0), one(3), one(2), one(0, 0), one(0), one(1))
    lib.dflash_tree_masks(one(0), one(1), None, one(0, 0), None, one(1))
    pool, q = torch.zeros((2, 4, 2, 128, 128), dtype=torch.bfloat16), torch.zeros((0, 8, 128), dtype=torch.bfloat16)

    class NoScratch:
        ptr, nbytes = None, 0

    lib.dflash_attention_tree_paged(heads, q, one(3), one(2), 0, 0, 0, lib.KvPages(pool, pool.clone(), one(2, 2)), one(0, 0), q.clone(),
                                    one(1), NoScratch())



def test_reserve_refuses_tables_whose_entries_it_cannot_count(lib):
    """Missing entries are summed over the batch in 32 bits."""
    def reserve(B, per):
        return lib.load().dflash_pages_reserve(ref(pages_of(lib, pages_per_seq=per)), FAKE, FAKE, B, FAKE, None, None)

    assert reserve(4096, 1 << 19) == reserve(2049, 1 << 20) == reserve(4096, (1 << 24) - 1) == lib.ERR_TOO_LARGE
    assert reserve(0, (1 << 24) - 1) == lib.OK
    if not torch.cuda.is_available():   # nothing to refuse but the machine
        for call in (reserve(4096, (1 << 19) - 1), reserve(2047, 1 << 20), reserve(128, (1 << 24) - 1)):
            assert call not in (lib.ERR_INVALID_ARG, lib.ERR_TOO_LARGE, lib.OK)


def test_shaped_distributions_by_plain_counting():
    r = np.random.default_rng(0)
    for _ in range(200):
        V = int(r.integers(1, 12))
        x = r.integers(-3, 4, V) * 0.5
        T, k, p, m = r.choice([0.5, 1.0, 2.0]), int(r.integers(0, V + 2)), r.choice([0.3, 0.8, 1.0]), r.choice([0.0, 0.2])
        got = tt.shape(x, T, k, p, m)
        # one token after another, the most likely first
        left = sorted(range(V), key=lambda v: (-x[v], v))[: k if k > 0 else V]
        w = {v: np.exp((x[v] - max(x)) / T) for v in left}
        total, mass, kept = sum(w.values()), 0.0, []
        for v in left:
            if not kept or ((p >= 1 or mass < p * total * (1 - 1e-12)) and w[v] >= m * (1 - 1e-12)):
                kept.append(v)
            mass += w[v]
        want = np.zeros(V)
        for v in kept:
            want[v] = w[v] / sum(w[i] for i in kept)
        assert np.allclose(got, want, atol=1e-12), (x, T, k, p, m)
    assert tt.shape(np.array([1.0, 3.0, 3.0]), 0.0).tolist() == [0, 1, 0]
    assert tt.shape(np.array([-np.inf, np.nan])) is None
    q = np.array([0.25, 0.0, 0.5, 0.25])
    assert [tt.draw(q, u) for u in (0.0, 0.2499, 0.25, 0.7, 0.75, 0.999)] == [0, 0, 2, 2, 3, 3]


def test_trees_and_branches_by_plain_counting():
    r = np.random.default_rng(1)
    for n in (1, 2, 40, 100):
        par = [-1] + [int(r.integers(0, i)) for i in range(1, n)]
        m = tt.sees(par)
        assert m.diagonal().all() and not np.triu(m, 1).any()
        for i in range(1, n):
            assert (m[i] == (m[par[i]] | (np.arange(n) == i))).all()
        w = tt.bits(m, 4).view(np.uint32)
        assert all(bool(w[i, j // 32] >> (j % 32) & 1) == m[i, j] for i in range(n) for j in range(n))
        tok, drawn = r.integers(0, 4, n).tolist(), r.integers(0, 4, n).tolist()
        tau, com, path, nxt = tt.verify_tree(tok, par, drawn, 200)
        assert path[0] == 0 and len(path) == len(com) == 200 and com[tau - 1] == nxt == drawn[path[tau - 1]]
        for a, b in zip(path[:tau - 1], path[1:tau]):
            assert par[b] == a and tok[b] == drawn[a]
        assert not any(par[c] == path[tau - 1] and tok[c] == nxt for c in range(n))


def test_attention_of_a_chain_is_causal():
    from oracle import target_ref as tr
    r = np.random.default_rng(2)
    q, k, v = r.normal(size=(5, 4, 8)), r.normal(size=(2, 12, 8)), r.normal(size=(2, 12, 8))
    a = tt.attention(q, k, v, 7, tt.sees([-1, 0, 1, 2, 3]))
    b = tr.chunk_attention(q, k, v, 7)
    assert all(np.allclose(x, y) for x, y in zip(a, b))


def test_pages_of_two_forks():
    p = tt.Pages([[3, 1, -1], [0, -1, -1], [-1] * 3], [1, 1, 0, 1, 0], [200, 5, 0])
    assert not p.fork([0], [2])
    assert p.table[2] == [3, 2, -1] and p.refs == [1, 1, 1, 2, 0] and p.copies == [(1, 2, 72)] and p.length == [200, 5, 200]
    p.reserve([200, 200, 200])
    assert p.table[1] == [0, 4, -1] and not p.full
    p.release([0, 128, 200])
    assert p.table[0] == [-1] * 3 and p.refs == [1, 0, 1, 1, 0]
    # the second pair is left out; five positions are part of a page: a page of its own, the lowest that is free
    assert p.fork([1, 1], [2, 2]) and p.table[2] == [1, -1, -1] and p.copies[-1] == (0, 1, 5)
