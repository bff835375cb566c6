"""GPU: the target-side calls refuse operands that do not lie on the current
device, and status words of another type, before anything is launched."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dfl(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def refused_for_each(dfl, call, operands):
    """The call with each operand in turn on the host, and with an int64 status word."""
    call(**operands)
    torch.cuda.synchronize()
    assert int(operands["dev_status"]) == dfl.OK
    for name, t in operands.items():
        with pytest.raises(dfl.DFlashError) as e:
            call(**{**operands, name: t.cpu()})
        assert e.value.status == dfl.ERR_INVALID_ARG, name
    with pytest.raises(dfl.DFlashError) as e:
        call(**{**operands, "dev_status": operands["dev_status"].long()})
    assert e.value.status == dfl.ERR_DTYPE


def test_operands_on_the_host_are_refused(dfl):
    bf, dev = torch.bfloat16, "cuda"
    heads = dfl.make_heads(1, 4, 2, 64)
    T, n_pos = 5, 160
    q, k, v = (torch.randn((T, h, 64), device=dev).to(bf) for h in (4, 2, 2))
    cos, sin = torch.ones((n_pos, 32), device=dev), torch.zeros((n_pos, 32), device=dev)
    gain = torch.ones(64, dtype=bf, device=dev)
    pool = lambda: torch.zeros((1, 3, 2, 128, 64), dtype=bf, device=dev)  # noqa: E731
    kp, vp, table = pool(), pool(), torch.tensor([[2, 0]], dtype=torch.int32, device=dev)
    cu, ctx = torch.tensor([0, T], dtype=torch.int32, device=dev), torch.tensor([100], dtype=torch.int32, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    positions = torch.arange(T, dtype=torch.int32, device=dev)

    def norm(q, k, positions, cos, sin, q_out, k_out, dev_status, g_q, g_k):
        dfl.dflash_qk_norm_rope(heads, q, k, positions, cos, sin, q_out, k_out, dev_status, g_q=g_q, g_k=g_k)

    refused_for_each(dfl, norm, dict(q=q, k=k, positions=positions, cos=cos, sin=sin, q_out=torch.empty_like(q),
                                     k_out=torch.empty_like(k), dev_status=st, g_q=gain, g_k=gain.clone()))

    def append(q, k, v, cu, ctx, kp, vp, table, cos, sin, q_out, dev_status, g_q, g_k):
        dfl.dflash_kv_append_paged(heads, q, k, v, cu, ctx, 0, dfl.KvPages(kp, vp, table), cos, sin, q_out, dev_status,
                                   g_q=g_q, g_k=g_k)

    refused_for_each(dfl, append, dict(q=q, k=k, v=v, cu=cu, ctx=ctx, kp=kp, vp=vp, table=table, cos=cos, sin=sin,
                                       q_out=torch.empty_like(q), dev_status=st, g_q=gain, g_k=gain.clone()))
    ws = dfl.ChunkWorkspace(heads)

    def attend(q, cu, ctx, kp, vp, table, out, dev_status):
        dfl.dflash_attention_chunk_paged(heads, q, cu, ctx, T, 100, 0, dfl.KvPages(kp, vp, table), out, dev_status, ws)

    refused_for_each(dfl, attend, dict(q=q, cu=cu, ctx=ctx, kp=kp, vp=vp, table=table, out=torch.empty_like(q), dev_status=st))
    with pytest.raises(dfl.DFlashError) as e:
        dfl.dflash_attention_chunk_paged(heads, q, cu, ctx, T, 100, 0, dfl.KvPages(kp, vp, table), torch.empty_like(q), st,
                                         dfl.ChunkWorkspace(heads, device="cpu"))
    assert e.value.status == dfl.ERR_INVALID_ARG
    with pytest.raises(dfl.DFlashError) as e:      # the output over the queries
        dfl.dflash_attention_chunk_paged(heads, q, cu, ctx, T, 100, 0, dfl.KvPages(kp, vp, table), q, st, ws)
    assert e.value.status == dfl.ERR_INVALID_ARG


def test_verification_operands_on_the_host_are_refused(dfl):
    cfg = dfl.config_from_workload(synth.WORKLOADS["tiny_f32_L1_N128"])
    B, m, V, dev = 1, cfg.gamma, cfg.vocab, "cuda"
    p = torch.softmax(torch.randn((B, m + 1, V), device=dev), -1)
    one = lambda: torch.zeros(B, dtype=torch.int32, device=dev)  # noqa: E731

    def verify(**kw):
        dfl.dflash_verify_probs(cfg, **kw)

    refused_for_each(dfl, verify, dict(
        target_probs=p, draft_probs=p[:, :m].contiguous(), draft=torch.zeros((B, m), dtype=torch.int32, device=dev),
        u_accept=torch.rand((B, m), device=dev), u_draw=torch.rand(B, device=dev), tau=one(),
        committed=torch.zeros((B, m + 1), dtype=torch.int32, device=dev), next_anchor=one(), dev_status=one(),
        gamma_b=torch.full((B,), m, dtype=torch.int32, device=dev)))
