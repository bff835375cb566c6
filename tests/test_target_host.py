"""Refusals of the target-side calls, all decided on the host before any
launch (no GPU: a call that passed the checks would answer ERR_ARCH or
ERR_CUDA instead, and every case below is refused before that)."""
import ctypes

import pytest
import torch

import synth

FAKE = 1 << 20     # a 16-byte aligned address; nothing is dereferenced


@pytest.fixture(scope="module")
def heads(lib):
    return lib.make_heads(2, 8, 2, 128)


def test_layouts(lib):
    ok = dict(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128)
    assert lib.dflash_check_heads(lib.make_heads(**ok)) == lib.OK
    assert lib.dflash_check_heads(lib.make_heads(1, 64, 1, 64, dtype=lib.F32)) == lib.OK
    for change, want in [(dict(n_layers=0), lib.ERR_INVALID_ARG), (dict(n_kv_heads=0), lib.ERR_INVALID_ARG),
                         (dict(n_kv_heads=3), lib.ERR_SHAPE), (dict(head_dim=96), lib.ERR_SHAPE),
                         (dict(n_q_heads=65, n_kv_heads=1), lib.ERR_SHAPE), (dict(dtype=5), lib.ERR_DTYPE),
                         (dict(rms_eps=-1.0), lib.ERR_INVALID_ARG), (dict(rms_eps=float("nan")), lib.ERR_INVALID_ARG)]:
        assert lib.dflash_check_heads(lib.make_heads(**{**ok, **change})) == want, change
    assert lib.load().dflash_check_heads(None) == lib.ERR_INVALID_ARG
    assert lib.dflash_attention_chunk_bytes(lib.make_heads(**ok)) > 0
    assert lib.dflash_attention_chunk_bytes(lib.make_heads(**{**ok, "head_dim": 32})) == 0


def norm_rope(lib, heads, **kw):
    a = dict(in_dtype=lib.BF16, q=FAKE, ldq=1024, k=FAKE, ldk=256, gq=FAKE, gk=FAKE, pos=FAKE, cos=FAKE, sin=FAKE, n=64,
             T=3, qo=FAKE, ldqo=1024, ko=FAKE, ldko=256, st=FAKE)
    a.update(kw)
    return lib.load().dflash_qk_norm_rope(
        ctypes.byref(heads), a["in_dtype"], a["q"], a["ldq"], a["k"], a["ldk"], a["gq"], a["gk"], a["pos"], a["cos"], a["sin"],
        a["n"], a["T"], a["qo"], a["ldqo"], a["ko"], a["ldko"], a["st"], None, None)


def test_norm_rope_refusals(lib, heads):
    assert norm_rope(lib, heads, T=0) == lib.OK
    for kw, want in [(dict(T=-1), "INVALID_ARG"), (dict(q=None, k=None), "INVALID_ARG"), (dict(st=None), "INVALID_ARG"),
                     (dict(qo=None), "INVALID_ARG"), (dict(ko=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"),
                     (dict(sin=None), "INVALID_ARG"), (dict(n=0), "INVALID_ARG"), (dict(ldq=1016), "INVALID_ARG"),
                     (dict(ldq=1025), "ALIGN"), (dict(k=FAKE + 8), "ALIGN"), (dict(gk=FAKE + 2), "ALIGN"),
                     (dict(cos=FAKE + 4), "ALIGN"), (dict(in_dtype=4), "DTYPE")]:
        assert norm_rope(lib, heads, **kw) == getattr(lib, "ERR_" + want), kw
    # bf16 rows are not stored as fp32
    assert norm_rope(lib, lib.make_heads(2, 8, 2, 128, dtype=lib.F32)) == lib.ERR_DTYPE
    assert norm_rope(lib, lib.make_heads(2, 8, 3, 128)) == lib.ERR_SHAPE


def pages_of(lib, n_pages=9, per_seq=4, k=FAKE, v=FAKE, table=FAKE):
    p = lib.KvPages.__new__(lib.KvPages)
    ctypes.Structure.__init__(p, k, v, table, n_pages, per_seq)
    return p


def append(lib, heads, **kw):
    a = dict(in_dtype=lib.F32, q=FAKE, ldq=1024, k=FAKE, ldk=256, v=FAKE, ldv=256, gq=None, gk=None, cos=None, sin=None, n=0,
             cu=FAKE, ctx=FAKE, B=2, T=5, layer=1, pages=pages_of(lib), qo=FAKE, ldqo=1024, st=FAKE)
    a.update(kw)
    pg = ctypes.byref(a["pages"]) if a["pages"] is not None else None
    return lib.load().dflash_kv_append_paged(
        ctypes.byref(heads), a["in_dtype"], a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["gq"], a["gk"], a["cos"],
        a["sin"], a["n"], a["cu"], a["ctx"], a["B"], a["T"], a["layer"], pg, a["qo"], a["ldqo"], a["st"], None, None)


def test_append_refusals(lib, heads):
    assert append(lib, heads, T=0) == lib.OK and append(lib, heads, B=0) == lib.OK
    for kw, want in [(dict(T=-1), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"), (dict(layer=2), "INVALID_ARG"),
                     (dict(layer=-1), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
                     (dict(cu=None), "INVALID_ARG"), (dict(ctx=None), "INVALID_ARG"), (dict(pages=None), "INVALID_ARG"),
                     (dict(pages=pages_of(lib, n_pages=0)), "INVALID_ARG"),
                     (dict(pages=pages_of(lib, per_seq=0)), "INVALID_ARG"),
                     (dict(pages=pages_of(lib, per_seq=1 << 25)), "INVALID_ARG"),
                     (dict(pages=pages_of(lib, table=None)), "INVALID_ARG"), (dict(qo=None), "INVALID_ARG"),
                     (dict(cos=FAKE), "INVALID_ARG"), (dict(st=None), "INVALID_ARG"), (dict(ldv=255), "INVALID_ARG"),
                     (dict(ldv=258), "ALIGN"), (dict(pages=pages_of(lib, v=FAKE + 2)), "ALIGN"), (dict(in_dtype=-1), "DTYPE")]:
        assert append(lib, heads, **kw) == getattr(lib, "ERR_" + want), kw


def attend(lib, heads, **kw):
    a = dict(q=FAKE, ldq=1024, cu=FAKE, ctx=FAKE, B=2, T=5, rows=5, hint=100, layer=1, pages=pages_of(lib), causal=1, scale=0.0,
             out=FAKE, ldo=1024, st=FAKE, ws=FAKE, nb=1 << 40)
    a.update(kw)
    pg = ctypes.byref(a["pages"]) if a["pages"] is not None else None
    return lib.load().dflash_attention_chunk_paged(
        ctypes.byref(heads), a["q"], a["ldq"], a["cu"], a["ctx"], a["B"], a["T"], a["rows"], a["hint"], a["layer"], pg,
        a["causal"], a["scale"], a["out"], a["ldo"], a["st"], a["ws"], a["nb"], None, None)


def test_chunk_attention_refusals(lib, heads):
    assert attend(lib, heads, T=0) == lib.OK and attend(lib, heads, B=0) == lib.OK
    for kw, want in [(dict(T=-1), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(hint=-1), "INVALID_ARG"),
                     (dict(layer=2), "INVALID_ARG"), (dict(causal=2), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"),
                     (dict(scale=float("inf")), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
                     (dict(cu=None), "INVALID_ARG"), (dict(ctx=None), "INVALID_ARG"), (dict(st=None), "INVALID_ARG"),
                     (dict(pages=None), "INVALID_ARG"), (dict(ldo=512), "INVALID_ARG"), (dict(ldo=1028), "ALIGN"),
                     (dict(q=FAKE + 2), "ALIGN"), (dict(ws=FAKE + 4), "ALIGN"), (dict(ws=None), "WORKSPACE"),
                     (dict(nb=1000), "WORKSPACE"), (dict(T=1 << 30), "TOO_LARGE"),
                     (dict(pages=pages_of(lib, n_pages=1 << 30)), "TOO_LARGE")]:
        assert attend(lib, heads, **kw) == getattr(lib, "ERR_" + want), kw


def verify(lib, cfg, **kw):
    a = dict(p=FAKE, dt=lib.F32, q=FAKE, d=FAKE, g=None, ua=FAKE, ud=FAKE, B=1, tau=FAKE, com=FAKE, nxt=FAKE, st=FAKE)
    a.update(kw)
    return lib.load().dflash_verify_probs(ctypes.byref(cfg), a["p"], a["dt"], a["q"], a["d"], a["g"], a["ua"], a["ud"], a["B"],
                                          a["tau"], a["com"], a["nxt"], a["st"], None, None)


def test_verify_probs_refusals(lib):
    cfg = lib.config_from_workload(synth.WORKLOADS["tiny_f32_L1_N128"])
    for kw, want in [(dict(dt=3), "DTYPE"), (dict(B=0), "INVALID_ARG"), (dict(B=cfg.max_batch + 1), "INVALID_ARG")] + [
            ({name: None}, "INVALID_ARG") for name in ("p", "d", "ua", "ud", "tau", "com", "nxt", "st")]:
        assert verify(lib, cfg, **kw) == getattr(lib, "ERR_" + want), kw
    bad = lib.config_from_workload(synth.WORKLOADS["tiny_f32_L1_N128"])
    bad.vocab = (1 << 24) + 1
    assert verify(lib, bad) == lib.ERR_TOO_LARGE
    bad.vocab = cfg.vocab
    bad.gamma = 17
    assert verify(lib, bad) == lib.ERR_INVALID_ARG


def test_outputs_over_other_operands_are_refused(lib, heads):
    """In place is for rows of one type and stride; an output over another operand's rows is refused."""
    at = [FAKE + (i << 16) for i in range(8)]
    apart = dict(q=at[0], k=at[1], qo=at[2], ko=at[3])
    for kw in (dict(qo=at[0], ldqo=2048), dict(ko=at[1], ldk=512), dict(qo=at[1]), dict(ko=at[0]), dict(ko=at[2]),
               dict(qo=at[0], in_dtype=lib.F32)):
        assert norm_rope(lib, heads, **{**apart, **kw}) == lib.ERR_INVALID_ARG, kw
    assert norm_rope(lib, heads, **apart, T=2 ** 31 - 1) == lib.ERR_TOO_LARGE
    apart = dict(q=at[0], k=at[1], v=at[2], qo=at[3], pages=pages_of(lib, k=at[4], v=at[5]))
    for kw in (dict(qo=at[0]), dict(qo=at[0], in_dtype=lib.BF16, ldqo=2048), dict(qo=at[1]), dict(qo=at[2]),
               dict(pages=pages_of(lib, k=at[4], v=at[4]))):
        assert append(lib, heads, **{**apart, **kw}) == lib.ERR_INVALID_ARG, kw
    assert append(lib, heads, **apart, T=2 ** 31 - 1) == lib.ERR_TOO_LARGE
    assert attend(lib, heads, q=at[0], out=at[0]) == lib.ERR_INVALID_ARG


def test_the_binding_refuses_rows_that_do_not_fit_the_layout(lib, heads):
    bf, ws = torch.bfloat16, None
    q, k = torch.zeros((3, 8, 128), dtype=bf), torch.zeros((3, 2, 128), dtype=bf)
    pages = lib.KvPages(torch.zeros((2, 4, 2, 128, 128), dtype=bf), torch.zeros((2, 4, 2, 128, 128), dtype=bf),
                        torch.zeros((1, 2), dtype=torch.int32))
    cu, ctx = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32)
    for bad in (q[:, :7], q[:, :, :64], q.transpose(0, 1), q[:, ::2]):
        with pytest.raises(lib.DFlashError) as e:
            lib.dflash_attention_chunk_paged(heads, bad, cu, ctx, 3, 0, 0, pages, q, st, ws)
        assert e.value.status == lib.ERR_SHAPE
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_attention_chunk_paged(heads, q.float(), cu, ctx, 3, 0, 0, pages, q, st, ws)
    assert e.value.status == lib.ERR_DTYPE
    with pytest.raises(lib.DFlashError) as e:      # fewer output rows than rows
        lib.dflash_qk_norm_rope(heads, q, k, ctx, None, None, q[:2], k, st)
    assert e.value.status == lib.ERR_SHAPE
    with pytest.raises(lib.DFlashError) as e:      # fp32 values next to bf16 keys
        lib.dflash_kv_append_paged(heads, q, k, k.float(), cu, ctx, 0, pages, None, None, q, st)
    assert e.value.status == lib.ERR_DTYPE
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_qk_norm_rope(heads, None, None, ctx, None, None, None, None, st)
    assert e.value.status == lib.ERR_INVALID_ARG
    with pytest.raises(lib.DFlashError) as e:
        lib.dflash_attention_chunk_paged(heads, None, cu, ctx, 3, 0, 0, pages, q, st, ws)
    assert e.value.status == lib.ERR_INVALID_ARG
    with pytest.raises(lib.DFlashError):
        lib.ChunkWorkspace(lib.make_heads(1, 3, 2, 128), device="cpu")


def test_the_binding_refuses_what_the_library_cannot_see(lib, heads):
    """Types, shapes and layouts behind the pointers: refused before any pointer is passed on."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k = torch.zeros((3, 8, 128), dtype=bf), torch.zeros((3, 2, 128), dtype=bf)
    pool = torch.zeros((2, 4, 2, 128, 128), dtype=bf)
    table, cu, ctx = torch.zeros((1, 2), dtype=i32), torch.tensor([0, 3], dtype=i32), torch.zeros(1, dtype=i32)
    st = torch.zeros(1, dtype=i32)
    good = lib.KvPages(pool, pool, table)
    cos = torch.zeros((8, 64))

    class NoScratch:
        ptr, nbytes = None, 0

    def att(pages=good, cu=cu, ctx=ctx):
        lib.dflash_attention_chunk_paged(heads, q, cu, ctx, 3, 0, 0, pages, q, st, NoScratch())

    def app(g=None, c=cos, s=cos, pages=good):
        lib.dflash_kv_append_paged(heads, q, k, k, cu, ctx, 0, pages, c, s, q, st, g_q=g)

    def fails(f, status):
        with pytest.raises(lib.DFlashError) as e:
            f()
        assert e.value.status == status, f

    fails(att, lib.ERR_WORKSPACE)                                                   # all else is right
    for bad in (lib.KvPages(pool[:1], pool[:1], table), lib.KvPages(pool.float(), pool.float(), table),
                lib.KvPages(pool[:, :, :1].contiguous(), pool[:, :, :1].contiguous(), table),
                lib.KvPages(pool, pool[:, :3], table), lib.KvPages(pool, pool, table.long())):
        fails(lambda: att(pages=bad), lib.ERR_SHAPE)
    fails(lambda: att(cu=cu[:1]), lib.ERR_SHAPE)
    fails(lambda: att(cu=cu.long()), lib.ERR_DTYPE)
    fails(lambda: att(cu=torch.zeros(3, dtype=i32), ctx=torch.zeros(2, dtype=i32)), lib.ERR_SHAPE)   # no table row
    fails(lambda: att(ctx=ctx.float()), lib.ERR_DTYPE)
    fails(lambda: app(g=torch.ones(64, dtype=bf)), lib.ERR_SHAPE)
    fails(lambda: app(g=torch.ones(128)), lib.ERR_DTYPE)
    fails(lambda: app(c=cos[:, :32], s=cos[:, :32]), lib.ERR_SHAPE)
    fails(lambda: app(c=cos.double(), s=cos.double()), lib.ERR_DTYPE)
    fails(lambda: app(s=None), lib.ERR_INVALID_ARG)
    fails(lambda: lib.dflash_qk_norm_rope(heads, q, None, torch.zeros(2, dtype=i32), cos, cos, q, None, st), lib.ERR_SHAPE)

    cfg = lib.config_from_workload(synth.WORKLOADS["tiny_f32_L1_N128"])
    B, m, V = 1, cfg.gamma, cfg.vocab
    p, d = torch.zeros((B, m + 1, V)), torch.zeros((B, m), dtype=i32)
    one, com = torch.zeros(B, dtype=i32), torch.zeros((B, m + 1), dtype=i32)

    def ver(p=p, q=torch.zeros((B, m, V)), d=d, ua=torch.zeros((B, m)), ud=torch.zeros(B), com=com, st=None):
        lib.dflash_verify_probs(cfg, p, q, d, ua, ud, one, com, one, st)

    fails(ver, lib.ERR_INVALID_ARG)                                                 # no status word; all else is right
    for kw, want in [(dict(p=p[:, 1:]), "SHAPE"), (dict(p=p[..., :-1]), "SHAPE"), (dict(p=p.double()), "DTYPE"),
                     (dict(q=torch.zeros((B, m, V), dtype=bf)), "DTYPE"), (dict(q=torch.zeros((B, m + 1, V))), "SHAPE"),
                     (dict(d=d.long()), "DTYPE"), (dict(d=d[:, 1:]), "SHAPE"), (dict(ua=torch.zeros((B, m - 1))), "SHAPE"),
                     (dict(ud=torch.zeros(B).double()), "DTYPE"), (dict(com=com[:, 1:].contiguous()), "SHAPE")]:
        fails(lambda: ver(**kw), getattr(lib, "ERR_" + want))
