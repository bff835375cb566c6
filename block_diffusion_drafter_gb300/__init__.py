"""Python binding of libdflash, the GB300 (sm_103a) DFlash drafting step.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels, reached through its C ABI (include/dflash.h). PyTorch provides the
device memory and streams. Functions keep the C names:
dflash_ctx_fuse, dflash_kv_inject, dflash_draft_block, dflash_verify_accept,
the target-side dflash_qk_norm_rope, dflash_kv_append_paged,
dflash_attention_chunk_paged and dflash_verify_probs, those around drafted trees
(dflash_tree_masks, dflash_attention_tree_paged, dflash_sample,
dflash_verify_tree, dflash_pages_*), plus the sizing / helper calls of the header. There is no CPU fallback: if
the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import _build

F32, BF16 = 0, 1
(OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_DTYPE, ERR_CAPACITY, ERR_ARCH, ERR_CUDA, ERR_TIMEOUT,
 ERR_WORKSPACE, ERR_ALIGN, ERR_TOO_LARGE) = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9, -10
K_GEMM, K_ATTN, K_NORM, K_ARGMAX, K_VERIFY, K_PAGES = range(6)


class DFlashError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "n_layers", "d_target", "n_taps", "d_model", "n_q_heads", "n_kv_heads", "head_dim",
        "d_ffn", "vocab", "gamma", "mask_token_id", "max_batch", "ctx_capacity")] + [
        ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float), ("dtype", ctypes.c_int)]


class WeightsStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_c", "g_c", "embed", "g_final", "lm_head", "g_attn", "w_qkv", "w_o", "g_ffn",
        "w_gateup", "w_down", "rope_cos", "rope_sin")] + [("rope_positions", ctypes.c_int)]


class Trace(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)), ("capacity", ctypes.c_int),
                ("count", ctypes.c_int), ("kinds", ctypes.POINTER(ctypes.c_int)),
                ("bytes", ctypes.POINTER(ctypes.c_double)),
                ("flops", ctypes.POINTER(ctypes.c_double))]


_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
PAGE_KEYS = 128


_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class KvPages(ctypes.Structure):
    """dflash_kv_pages: page pools [L, n_pages, Hkv, 128, Dh] and a device page
    table [max_batch, pages_per_seq] (tensors kept alive by the object)."""
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_int),
                ("pages_per_seq", ctypes.c_int)]

    def __init__(self, k_pool, v_pool, page_table):
        super().__init__(k_pool.data_ptr(), v_pool.data_ptr(), page_table.data_ptr(), k_pool.shape[1],
                         page_table.shape[1])
        self._keep = (k_pool, v_pool, page_table)
        # what the target-side calls compare with their layout: (L, Hkv, Dh, dtype) and the table's sequences
        fits = (k_pool.dim() == 5 and k_pool.shape == v_pool.shape and k_pool.dtype == v_pool.dtype
                and k_pool.shape[3] == PAGE_KEYS and k_pool.is_contiguous() and v_pool.is_contiguous()
                and page_table.dtype == torch.int32 and page_table.is_contiguous())
        self.layout = (k_pool.shape[0], k_pool.shape[2], k_pool.shape[4], _DTYPES.get(k_pool.dtype)) if fits else None
        self.sequences = page_table.shape[0]
        on = {t.get_device() for t in self._keep}
        self.device = on.pop() if len(on) == 1 else None


class Heads(ctypes.Structure):
    """dflash_heads: the attention layout that the target-side calls work on."""
    _fields_ = [("n_layers", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("rms_eps", ctypes.c_float), ("dtype", ctypes.c_int)]


_LL = ctypes.c_longlong
_SIGS = {
    "dflash_abi_version": (_I, []),
    "dflash_status_string": (ctypes.c_char_p, [_I]),
    "dflash_check_config": (_I, [ctypes.POINTER(Config)]),
    "dflash_param_bytes": (_SZ, [ctypes.POINTER(Config), _I]),
    "dflash_kv_cache_bytes": (_SZ, [ctypes.POINTER(Config)]),
    "dflash_workspace_bytes": (_SZ, [ctypes.POINTER(Config), _I]),
    "dflash_workspace_init": (_I, [_P, _SZ, _P]),
    "dflash_ctx_fuse": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _I, _P,
                             _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_kv_inject": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P, _I,
                              _I, _P, _P, _P, _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_draft_block": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P,
                                _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                ctypes.POINTER(Trace), _P]),
    "dflash_verify_accept": (_I, [ctypes.POINTER(Config), _P, _I, _P, _I, _P, _P, _P, _P, _SZ,
                                  ctypes.POINTER(Trace), _P]),
    "dflash_rope_tables": (_I, [ctypes.POINTER(Config), _I, _P, _P]),
    "dflash_linear": (_I, [_I, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dflash_verify_accept_noalloc": (_I, [ctypes.POINTER(Config), _P, _I, _P, _I, _P, _P, _P, _P]),
    "dflash_selftest_wait_timeout": (_I, [_P, _P]),
    "dflash_attention": (_I, [ctypes.POINTER(Config), _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ,
                              ctypes.POINTER(Trace), _P]),
    "dflash_draft_block_dyn": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P, _P,
                                    _I, _I, _P, _P, _P, _P, _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_verify_accept_dyn": (_I, [ctypes.POINTER(Config), _P, _I, _P, _P, _I, _P, _P, _P, _P, _SZ,
                                      ctypes.POINTER(Trace), _P]),
    "dflash_draft_block_ids": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P, _I, _I,
                                    _P, _P, _P, _P, _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_unmask_step": (_I, [ctypes.POINTER(Config), _P, _P, _P, _I, _I, _P, _SZ, ctypes.POINTER(Trace),
                                _P]),
    "dflash_draft_block_iter": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P, _I, _I,
                                     _P, _P, _I, _P, _P, _P, _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_kv_inject_paged": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P, _I, _I, _P,
                                    ctypes.POINTER(KvPages), _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_draft_block_paged": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P, _I, _I,
                                      ctypes.POINTER(KvPages), _P, _P, _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_draft_block_sample": (_I, [ctypes.POINTER(Config), ctypes.POINTER(WeightsStruct), _P, _P,
                                       _I, _I, _P, _P, ctypes.c_float, ctypes.c_uint64, _P, _P, _P,
                                       _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_verify_sample": (_I, [ctypes.POINTER(Config), _P, _I, _P, _P, _I, ctypes.c_float,
                                  ctypes.c_uint64, _P, _P, _P, _P, _SZ, ctypes.POINTER(Trace), _P]),
    "dflash_check_heads": (_I, [ctypes.POINTER(Heads)]),
    "dflash_qk_norm_rope": (_I, [ctypes.POINTER(Heads), _I, _P, _LL, _P, _LL, _P, _P, _P, _P, _P, _I, _I, _P, _LL,
                                 _P, _LL, _P, ctypes.POINTER(Trace), _P]),
    "dflash_kv_append_paged": (_I, [ctypes.POINTER(Heads), _I, _P, _LL, _P, _LL, _P, _LL, _P, _P, _P, _P, _I, _P, _P,
                                    _I, _I, _I, ctypes.POINTER(KvPages), _P, _LL, _P, ctypes.POINTER(Trace), _P]),
    "dflash_attention_chunk_bytes": (_SZ, [ctypes.POINTER(Heads)]),
    "dflash_attention_chunk_paged": (_I, [ctypes.POINTER(Heads), _P, _LL, _P, _P, _I, _I, _I, _I, _I,
                                          ctypes.POINTER(KvPages), _I, ctypes.c_float, _P, _LL, _P, _P, _SZ,
                                          ctypes.POINTER(Trace), _P]),
    "dflash_verify_probs": (_I, [ctypes.POINTER(Config), _P, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P,
                                 ctypes.POINTER(Trace), _P]),
    "dflash_tree_masks": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P, ctypes.POINTER(Trace), _P]),
    "dflash_attention_tree_paged": (_I, [ctypes.POINTER(Heads), _P, _LL, _P, _P, _I, _I, _I, _I, _I,
                                         ctypes.POINTER(KvPages), _P, _I, ctypes.c_float, _P, _LL, _P, _P, _SZ,
                                         ctypes.POINTER(Trace), _P]),
    "dflash_sample": (_I, [_P, _I, _LL, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.POINTER(Trace), _P]),
    "dflash_verify_tree": (_I, [ctypes.POINTER(Heads), _P, _P, _P, _P, _P, _I, _I, _I, ctypes.POINTER(KvPages), _P, _P, _P,
                                _P, _P, ctypes.POINTER(Trace), _P]),
    "dflash_pages_release": (_I, [ctypes.POINTER(KvPages), _P, _P, _I, _P, ctypes.POINTER(Trace), _P]),
    "dflash_pages_reserve": (_I, [ctypes.POINTER(KvPages), _P, _P, _I, _P, ctypes.POINTER(Trace), _P]),
    "dflash_pages_fork": (_I, [ctypes.POINTER(Heads), ctypes.POINTER(KvPages), _P, _P, _I, _P, _P, _I, _P,
                               ctypes.POINTER(Trace), _P]),
}

_lib = None


def lib_path() -> str:
    return _build.LIB


def load(build: bool = True) -> ctypes.CDLL:
    """Loads libdflash.so (building it first when asked and out of date)."""
    global _lib
    if _lib is None:
        if build:
            _build.build_library()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"libdflash.so is not built ({_build.LIB}); run __graft_entry__.build()")
        lib = ctypes.CDLL(_build.LIB)
        for name, (res, args) in _SIGS.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/dflash.h."""
    path = os.path.join(_build.INCLUDE, "dflash.h")
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dflash_[a-z_0-9]+)\s*\(", text)))


def status_string(s: int) -> str:
    return load().dflash_status_string(s).decode()


def _check(fn: str, s: int):
    if s != OK:
        raise DFlashError(fn, s)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


_cuda = None   # whether there is a GPU, asked once


def _stream(stream) -> int | None:
    global _cuda
    if stream is None:
        if _cuda is None:
            _cuda = torch.cuda.is_available()
        # the current stream's handle without a Stream object around it (0.3 instead of 3.6 us a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if _cuda else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def make_config(n_layers, d_target, n_taps, d_model, n_q_heads, n_kv_heads, head_dim, d_ffn,
                vocab, gamma, mask_token_id, max_batch, ctx_capacity, rms_eps=1e-6,
                rope_theta=1e6, dtype=BF16) -> Config:
    return Config(n_layers, d_target, n_taps, d_model, n_q_heads, n_kv_heads, head_dim, d_ffn,
                  vocab, gamma, mask_token_id, max_batch, ctx_capacity, rms_eps, rope_theta, dtype)


def config_from_workload(wl, max_batch=None, ctx_capacity=None) -> Config:
    return make_config(wl.n_layers, wl.d_target, wl.n_taps, wl.d_model, wl.n_q_heads,
                       wl.n_kv_heads, wl.head_dim, wl.d_ffn, wl.vocab, wl.gamma,
                       wl.mask_token_id, max_batch or wl.batch, ctx_capacity or wl.capacity(),
                       wl.rms_eps, wl.rope_theta, BF16 if wl.dtype == "bf16" else F32)


def dflash_check_config(cfg: Config) -> int:
    return load().dflash_check_config(ctypes.byref(cfg))


def dflash_param_bytes(cfg: Config, kind: int) -> int:
    return load().dflash_param_bytes(ctypes.byref(cfg), kind)


def dflash_kv_cache_bytes(cfg: Config) -> int:
    return load().dflash_kv_cache_bytes(ctypes.byref(cfg))


def dflash_workspace_bytes(cfg: Config, max_rows: int) -> int:
    return load().dflash_workspace_bytes(ctypes.byref(cfg), max_rows)


def dflash_rope_tables(cfg: Config, n_pos: int):
    """(cos, sin) fp32 CPU tensors [n_pos, Dh/2] computed by the library in fp64."""
    half = cfg.head_dim // 2
    c = torch.empty((n_pos, half), dtype=torch.float32)
    s = torch.empty((n_pos, half), dtype=torch.float32)
    _check("dflash_rope_tables", load().dflash_rope_tables(ctypes.byref(cfg), n_pos, c.data_ptr(), s.data_ptr()))
    return c, s


class Weights:
    """Device-resident drafter parameters plus the RoPE tables, and the
    dflash_weights struct that points at them."""

    def __init__(self, cfg: Config, tensors: dict, device="cuda"):
        self.cfg = cfg
        self.t = {k: v.to(device).contiguous() for k, v in tensors.items()}
        self.rope_cos = self.rope_sin = None
        n_rope = 0
        if cfg.rope_theta > 0:
            n_rope = cfg.ctx_capacity
            c, s = dflash_rope_tables(cfg, n_rope)
            self.rope_cos, self.rope_sin = c.to(device), s.to(device)
        t = self.t
        self.struct = WeightsStruct(
            _ptr(t["w_c"]), _ptr(t["g_c"]), _ptr(t["embed"]), _ptr(t["g_final"]),
            _ptr(t["lm_head"]), _ptr(t["g_attn"]), _ptr(t["w_qkv"]), _ptr(t["w_o"]),
            _ptr(t["g_ffn"]), _ptr(t["w_gateup"]), _ptr(t["w_down"]), _ptr(self.rope_cos),
            _ptr(self.rope_sin), n_rope)


class Workspace:
    """Caller-owned scratch buffer sized by dflash_workspace_bytes, zeroed once."""

    def __init__(self, cfg: Config, max_rows: int, device="cuda", stream=None):
        n = dflash_workspace_bytes(cfg, max_rows)
        if n == 0:
            raise DFlashError("dflash_workspace_bytes", dflash_check_config(cfg))
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)
        self.nbytes = n
        _check("dflash_workspace_init",
               load().dflash_workspace_init(self.buf.data_ptr(), n, _stream(stream)))

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def _tr(trace):
    return ctypes.byref(trace) if trace is not None else None


def dflash_ctx_fuse(cfg, w: Weights, taps, h_ctx, ws: Workspace, trace=None, stream=None):
    T = taps.shape[0] if taps is not None else 0
    _check("dflash_ctx_fuse", load().dflash_ctx_fuse(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(taps), T, _ptr(h_ctx), ws.ptr, ws.nbytes,
        _tr(trace), _stream(stream)))


def dflash_kv_inject(cfg, w: Weights, h_ctx, n_new, ctx_len, k_cache, v_cache, dev_status,
                     ws: Workspace, trace=None, stream=None):
    B, Tmax = h_ctx.shape[0], h_ctx.shape[1]
    _check("dflash_kv_inject", load().dflash_kv_inject(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(h_ctx), _ptr(n_new), B, Tmax,
        _ptr(ctx_len), _ptr(k_cache), _ptr(v_cache), _ptr(dev_status), ws.ptr, ws.nbytes,
        _tr(trace), _stream(stream)))


def dflash_draft_block(cfg, w: Weights, anchor, ctx_len, max_ctx_hint, k_cache, v_cache, draft,
                       dev_status, ws: Workspace, logits=None, layer_dump=None, trace=None,
                       stream=None):
    B = anchor.shape[0]
    _check("dflash_draft_block", load().dflash_draft_block(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(anchor), _ptr(ctx_len), B,
        int(max_ctx_hint), _ptr(k_cache), _ptr(v_cache), _ptr(draft), _ptr(logits),
        _ptr(layer_dump), _ptr(dev_status), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_verify_accept(cfg, target_logits, draft, tau, committed, next_anchor, ws: Workspace,
                         trace=None, stream=None):
    dt = BF16 if target_logits.dtype == torch.bfloat16 else F32
    B = target_logits.shape[0]
    _check("dflash_verify_accept", load().dflash_verify_accept(
        ctypes.byref(cfg), _ptr(target_logits), dt, _ptr(draft), B, _ptr(tau), _ptr(committed),
        _ptr(next_anchor), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_kv_inject_paged(cfg, w: Weights, h_ctx, n_new, ctx_len, pages: KvPages, dev_status, ws: Workspace,
                           trace=None, stream=None):
    B, Tmax = h_ctx.shape[0], h_ctx.shape[1]
    _check("dflash_kv_inject_paged", load().dflash_kv_inject_paged(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(h_ctx), _ptr(n_new), B, Tmax, _ptr(ctx_len),
        ctypes.byref(pages), _ptr(dev_status), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_draft_block_paged(cfg, w: Weights, anchor, ctx_len, max_ctx_hint, pages: KvPages, draft, dev_status,
                             ws: Workspace, logits=None, trace=None, stream=None):
    B = anchor.shape[0]
    _check("dflash_draft_block_paged", load().dflash_draft_block_paged(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(anchor), _ptr(ctx_len), B, int(max_ctx_hint),
        ctypes.byref(pages), _ptr(draft), _ptr(logits), _ptr(dev_status), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_draft_block_dyn(cfg, w: Weights, anchor, ctx_len, gamma_b, max_ctx_hint, k_cache, v_cache,
                           draft, dev_status, ws: Workspace, logits=None, trace=None, stream=None):
    """Drafting pass with block size gamma_b[b] per sequence (draft[b, j] = -1
    for j >= gamma_b[b])."""
    B = anchor.shape[0]
    _check("dflash_draft_block_dyn", load().dflash_draft_block_dyn(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(anchor), _ptr(ctx_len), _ptr(gamma_b), B,
        int(max_ctx_hint), _ptr(k_cache), _ptr(v_cache), _ptr(draft), _ptr(logits), _ptr(dev_status),
        ws.ptr, ws.nbytes, ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_verify_accept_dyn(cfg, target_logits, draft, gamma_b, tau, committed, next_anchor,
                             ws: Workspace, trace=None, stream=None):
    dt = BF16 if target_logits.dtype == torch.bfloat16 else F32
    B = target_logits.shape[0]
    _check("dflash_verify_accept_dyn", load().dflash_verify_accept_dyn(
        ctypes.byref(cfg), _ptr(target_logits), dt, _ptr(draft), _ptr(gamma_b), B, _ptr(tau),
        _ptr(committed), _ptr(next_anchor), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_draft_block_ids(cfg, w: Weights, ids, ctx_len, max_ctx_hint, k_cache, v_cache, draft, dev_status,
                           ws: Workspace, logits=None, trace=None, stream=None):
    """Drafting pass on explicit block inputs ids [B, R]."""
    B = ids.shape[0]
    _check("dflash_draft_block_ids", load().dflash_draft_block_ids(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(ids), _ptr(ctx_len), B, int(max_ctx_hint),
        _ptr(k_cache), _ptr(v_cache), _ptr(draft), _ptr(logits), _ptr(dev_status), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_unmask_step(cfg, logits, draft, ids, steps_left, ws: Workspace, trace=None, stream=None):
    _check("dflash_unmask_step", load().dflash_unmask_step(
        ctypes.byref(cfg), _ptr(logits), _ptr(draft), _ptr(ids), ids.shape[0], int(steps_left), ws.ptr,
        ws.nbytes, ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_draft_block_iter(cfg, w: Weights, anchor, ctx_len, max_ctx_hint, k_cache, v_cache, n_steps, ids,
                            draft, logits, dev_status, ws: Workspace, trace=None, stream=None):
    """n_steps passes of multi-step confidence unmasking."""
    B = anchor.shape[0]
    _check("dflash_draft_block_iter", load().dflash_draft_block_iter(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(anchor), _ptr(ctx_len), B, int(max_ctx_hint),
        _ptr(k_cache), _ptr(v_cache), int(n_steps), _ptr(ids), _ptr(draft), _ptr(logits), _ptr(dev_status),
        ws.ptr, ws.nbytes, ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_draft_block_sample(cfg, w: Weights, anchor, ctx_len, max_ctx_hint, k_cache, v_cache,
                              temperature, seed, draft, logits, dev_status, ws: Workspace, trace=None,
                              stream=None):
    """Sampling drafting pass: draft j ~ softmax(logits_j / temperature);
    logits [B, gamma, V] fp32 receives the raw logits (the verifier's q)."""
    B = anchor.shape[0]
    _check("dflash_draft_block_sample", load().dflash_draft_block_sample(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(anchor), _ptr(ctx_len), B,
        int(max_ctx_hint), _ptr(k_cache), _ptr(v_cache), float(temperature), int(seed) & (2**64 - 1),
        _ptr(draft), _ptr(logits), _ptr(dev_status), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_verify_sample(cfg, target_logits, draft_logits, draft, temperature, seed, tau, committed,
                         next_anchor, ws: Workspace, trace=None, stream=None):
    """Rejection-acceptance verification at temperature > 0."""
    dt = BF16 if target_logits.dtype == torch.bfloat16 else F32
    B = target_logits.shape[0]
    _check("dflash_verify_sample", load().dflash_verify_sample(
        ctypes.byref(cfg), _ptr(target_logits), dt, _ptr(draft_logits), _ptr(draft), B,
        float(temperature), int(seed) & (2**64 - 1), _ptr(tau), _ptr(committed), _ptr(next_anchor),
        ws.ptr, ws.nbytes, ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_verify_accept_noalloc(cfg, target_logits, draft, tau, committed, next_anchor,
                                 stream=None):
    """dflash_verify_accept with its scratch in the library's own device memory
    (no workspace): for callers that cannot allocate device memory."""
    dt = BF16 if target_logits.dtype == torch.bfloat16 else F32
    B = target_logits.shape[0]
    _check("dflash_verify_accept_noalloc", load().dflash_verify_accept_noalloc(
        ctypes.byref(cfg), _ptr(target_logits), dt, _ptr(draft), B, _ptr(tau), _ptr(committed),
        _ptr(next_anchor), _stream(stream)))


def dflash_attention(cfg, q, ctx_len, max_ctx_hint, layer, k_cache, v_cache, out, dev_status,
                     ws: Workspace, trace=None, stream=None):
    """One layer's context attention (the drafting pass's attention step):
    q, out [B*R, Hq*Dh]; the block's K/V already in cache rows ctx_len.."""
    B = ctx_len.shape[0]
    _check("dflash_attention", load().dflash_attention(
        ctypes.byref(cfg), _ptr(q), _ptr(ctx_len), B, int(max_ctx_hint), int(layer), _ptr(k_cache),
        _ptr(v_cache), _ptr(out), _ptr(dev_status), ws.ptr, ws.nbytes,
        ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def dflash_selftest_wait_timeout(dev_status, stream=None):
    """Launches the bounded-wait self-test: dev_status reads ERR_TIMEOUT after ~1 s."""
    _check("dflash_selftest_wait_timeout", load().dflash_selftest_wait_timeout(_ptr(dev_status), _stream(stream)))


def dflash_linear(x, w, y, ws: Workspace, stream=None):
    dt = BF16 if x.dtype == torch.bfloat16 else F32
    M, K = x.shape
    N = w.shape[0]
    _check("dflash_linear", load().dflash_linear(dt, _ptr(x), _ptr(w), _ptr(y), M, N, K, ws.ptr,
                                                 ws.nbytes, _stream(stream)))


# ---------------------------------------------------------------- target side
def make_heads(n_layers, n_q_heads, n_kv_heads, head_dim, rms_eps=1e-6, dtype=BF16) -> Heads:
    return Heads(n_layers, n_q_heads, n_kv_heads, head_dim, rms_eps, dtype)


def dflash_check_heads(heads: Heads) -> int:
    return load().dflash_check_heads(ctypes.byref(heads))


def dflash_attention_chunk_bytes(heads: Heads) -> int:
    return load().dflash_attention_chunk_bytes(ctypes.byref(heads))


class ChunkWorkspace:
    """Caller-owned scratch of dflash_attention_chunk_paged (any batch of the layout)."""

    def __init__(self, heads: Heads, device="cuda"):
        n = dflash_attention_chunk_bytes(heads)
        if n == 0:
            raise DFlashError("dflash_attention_chunk_bytes", dflash_check_heads(heads))
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)
        self.nbytes = n
        self.ptr = self.buf.data_ptr()


def _here(stream, fn: str, *tensors):
    """The stream's handle, once every operand is known to lie on the current
    device (a kernel that met another's or the host's memory would fault)."""
    handle = _stream(stream)
    if _cuda is None:   # a stream was given: not asked yet
        _stream(None)
    if _cuda:
        device = torch._C._cuda_getDevice()
        at = [t.get_device() for t in tensors if t is not None]
        if at.count(device) != len(at):
            raise DFlashError(fn, ERR_INVALID_ARG)
    return handle


def _rows(t, n_heads: int, head_dim: int, dtype, fn: str):
    """(pointer, row stride, rows) of [T, heads, Dh] rows whose heads lie side by side."""
    if t is None:
        return None, 0, 0
    rows, heads, dh = t.shape
    ld = heads * dh
    whole = t.is_contiguous()
    if not whole:
        ld, hs, es = t.stride()
        whole = es == 1 and (hs == dh or heads == 1)
        if rows <= 1:   # the stride of a single row says nothing
            ld = max(ld, heads * dh)
    if heads != n_heads or dh != head_dim or not whole:
        raise DFlashError(fn, ERR_SHAPE)
    if _DTYPES.get(t.dtype) != dtype:
        raise DFlashError(fn, ERR_DTYPE)
    return t.data_ptr(), ld, rows


def _ints(t, n: int, fn: str):
    """Pointer of a device int32 vector of at least n entries."""
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous():
        raise DFlashError(fn, ERR_SHAPE if t.dtype is torch.int32 else ERR_DTYPE)
    return t.data_ptr()


def _status(t, fn: str):
    return _ints(t, 1, fn) if t is not None else None


def _gain(t, heads: Heads, fn: str):
    if t is None:
        return None
    if t.numel() != heads.head_dim or _DTYPES.get(t.dtype) != heads.dtype or not t.is_contiguous():
        raise DFlashError(fn, ERR_SHAPE if _DTYPES.get(t.dtype) == heads.dtype else ERR_DTYPE)
    return t.data_ptr()


def _tables(c, s, heads: Heads, fn: str):
    """Pointers and rows of the RoPE tables (fp32 [n, Dh/2]), None for no rotation."""
    if c is None or s is None:
        return _ptr(c), _ptr(s), 0
    n, half = c.shape
    if s.numel() != n * half or 2 * half != heads.head_dim or not c.is_contiguous() or not s.is_contiguous():
        raise DFlashError(fn, ERR_SHAPE)
    if c.dtype is not torch.float32 or s.dtype is not torch.float32:
        raise DFlashError(fn, ERR_DTYPE)
    return c.data_ptr(), s.data_ptr(), n


def _view(pages: KvPages, heads: Heads, ctx_len, fn: str):
    """A page view of the layout, with a table row for every sequence, where the lengths lie."""
    if pages.layout != (heads.n_layers, heads.n_kv_heads, heads.head_dim, heads.dtype) or pages.sequences < ctx_len.numel():
        raise DFlashError(fn, ERR_SHAPE)
    if pages.device != ctx_len.get_device():
        raise DFlashError(fn, ERR_INVALID_ARG)
    return ctypes.byref(pages)


def dflash_qk_norm_rope(heads: Heads, q, k, positions, rope_cos, rope_sin, q_out, k_out, dev_status, g_q=None, g_k=None,
                        trace=None, stream=None):
    """Per-head RMSNorm (where a gain is given) and RoPE of q [T, Hq, Dh] and
    k [T, Hkv, Dh] (either may be None) into q_out, k_out."""
    fn = "dflash_qk_norm_rope"
    x = q if q is not None else k
    if x is None:
        raise DFlashError(fn, ERR_INVALID_ARG)
    dt, hq, hk, dh, out = _DTYPES.get(x.dtype, -1), heads.n_q_heads, heads.n_kv_heads, heads.head_dim, heads.dtype
    qp, ldq, n_q = _rows(q, hq, dh, dt, fn)
    kp, ldk, n_k = _rows(k, hk, dh, dt, fn)
    qo, ldqo, n_qo = _rows(q_out if q is not None else None, hq, dh, out, fn)
    ko, ldko, n_ko = _rows(k_out if k is not None else None, hk, dh, out, fn)
    if n_qo < n_q or n_ko < n_k or (q is not None and k is not None and n_q != n_k):
        raise DFlashError(fn, ERR_SHAPE)
    T = n_q if q is not None else n_k
    cos, sin, n = _tables(rope_cos, rope_sin, heads, fn)
    _check(fn, load().dflash_qk_norm_rope(
        ctypes.byref(heads), dt, qp, ldq, kp, ldk, _gain(g_q, heads, fn), _gain(g_k, heads, fn),
        _ints(positions, T, fn) if positions is not None else None, cos, sin, n, T, qo, ldqo, ko, ldko,
        _status(dev_status, fn), _tr(trace),
        _here(stream, fn, q, k, q_out, k_out, positions, rope_cos, rope_sin, g_q, g_k, dev_status)))


def dflash_kv_append_paged(heads: Heads, q, k, v, cu_rows, ctx_len, layer, pages: KvPages, rope_cos, rope_sin, q_out,
                           dev_status, g_q=None, g_k=None, trace=None, stream=None):
    """Appends packed rows k, v [T, Hkv, Dh] to one layer of the paged cache
    (K normed and rotated on the way); q [T, Hq, Dh] (or None) likewise into q_out."""
    fn = "dflash_kv_append_paged"
    dt, hq, hk, dh = _DTYPES.get(k.dtype, -1), heads.n_q_heads, heads.n_kv_heads, heads.head_dim
    qp, ldq, n_q = _rows(q, hq, dh, dt, fn)
    kp, ldk, T = _rows(k, hk, dh, dt, fn)
    vp, ldv, n_v = _rows(v, hk, dh, dt, fn)
    qo, ldqo, n_qo = _rows(q_out if q is not None else None, hq, dh, heads.dtype, fn)
    if n_v != T or (q is not None and (n_q != T or n_qo < T)):
        raise DFlashError(fn, ERR_SHAPE)
    cos, sin, n = _tables(rope_cos, rope_sin, heads, fn)
    B = ctx_len.numel()
    _check(fn, load().dflash_kv_append_paged(
        ctypes.byref(heads), dt, qp, ldq, kp, ldk, vp, ldv, _gain(g_q, heads, fn), _gain(g_k, heads, fn), cos, sin, n,
        _ints(cu_rows, B + 1, fn), _ints(ctx_len, B, fn), B, T, int(layer), _view(pages, heads, ctx_len, fn), qo, ldqo,
        _status(dev_status, fn), _tr(trace),
        _here(stream, fn, k, v, q, q_out, cu_rows, ctx_len, rope_cos, rope_sin, g_q, g_k, dev_status)))


def dflash_attention_chunk_paged(heads: Heads, q, cu_rows, ctx_len, max_rows, max_ctx_hint, layer, pages: KvPages, out,
                                 dev_status, ws: ChunkWorkspace, causal=True, scale=0.0, trace=None, stream=None):
    """Attention of a ragged batch of chunks q [T, Hq, Dh] over the paged cache
    that already holds the chunks' own keys and values."""
    fn = "dflash_attention_chunk_paged"
    hq, dh, dt = heads.n_q_heads, heads.head_dim, heads.dtype
    qp, ldq, T = _rows(q, hq, dh, dt, fn)
    op, ldo, n_out = _rows(out, hq, dh, dt, fn)
    if q is None or n_out < T:
        raise DFlashError(fn, ERR_INVALID_ARG if q is None else ERR_SHAPE)
    B = ctx_len.numel()
    _check(fn, load().dflash_attention_chunk_paged(
        ctypes.byref(heads), qp, ldq, _ints(cu_rows, B + 1, fn), _ints(ctx_len, B, fn), B, T, int(max_rows),
        int(max_ctx_hint), int(layer), _view(pages, heads, ctx_len, fn), 1 if causal else 0, float(scale), op, ldo,
        _status(dev_status, fn), ws.ptr, ws.nbytes, _tr(trace),
        _here(stream, fn, q, out, cu_rows, ctx_len, dev_status, getattr(ws, "buf", None))))


def dflash_verify_probs(cfg, target_probs, draft_probs, draft, u_accept, u_draw, tau, committed, next_anchor,
                        dev_status, gamma_b=None, trace=None, stream=None):
    """Verification against given probabilities from given uniforms; draft_probs
    None for greedy drafts."""
    fn = "dflash_verify_probs"
    B, R, V = target_probs.shape
    dt = _DTYPES.get(target_probs.dtype, -1)
    if R != cfg.gamma + 1 or V != cfg.vocab or not target_probs.is_contiguous() or (
            draft_probs is not None and (draft_probs.shape != (B, R - 1, V) or not draft_probs.is_contiguous())) or (
            u_accept.numel() < B * (R - 1) or u_draw.numel() < B or not u_accept.is_contiguous() or not u_draw.is_contiguous()):
        raise DFlashError(fn, ERR_SHAPE)
    f32 = torch.float32
    if u_accept.dtype is not f32 or u_draw.dtype is not f32 or (draft_probs is not None and draft_probs.dtype is not f32):
        raise DFlashError(fn, ERR_DTYPE)
    _check(fn, load().dflash_verify_probs(
        ctypes.byref(cfg), target_probs.data_ptr(), dt, _ptr(draft_probs), _ints(draft, B * (R - 1), fn),
        _ints(gamma_b, B, fn) if gamma_b is not None else None, u_accept.data_ptr(), u_draw.data_ptr(), B,
        _ints(tau, B, fn), _ints(committed, B * R, fn), _ints(next_anchor, B, fn), _status(dev_status, fn), _tr(trace),
        _here(stream, fn, target_probs, draft_probs, draft, u_accept, u_draw, gamma_b, tau, committed, next_anchor,
              dev_status)))


# ---------------------------------------------------------------- drafted trees
def dflash_tree_masks(parents, cu_rows, ctx_len, mask, positions, dev_status, trace=None, stream=None):
    """Masks [T, words] (int32 bits) and positions [T] (or None) of a ragged batch of
    trees given by every node's parent within its sequence (-1 for none)."""
    fn = "dflash_tree_masks"
    T, B = parents.numel(), cu_rows.numel() - 1
    words = _mask_words(mask, T, fn)
    _check(fn, load().dflash_tree_masks(
        _ints(parents, T, fn), _ints(cu_rows, B + 1, fn), _ints(ctx_len, B, fn) if ctx_len is not None else None, B, T, words,
        mask.data_ptr(), _ints(positions, T, fn) if positions is not None else None, _status(dev_status, fn), _tr(trace),
        _here(stream, fn, parents, cu_rows, ctx_len, mask, positions, dev_status)))


def _mask_words(mask, T: int, fn: str) -> int:
    if mask.dtype is not torch.int32:
        raise DFlashError(fn, ERR_DTYPE)
    if mask.dim() != 2 or mask.shape[0] < T or not mask.is_contiguous():
        raise DFlashError(fn, ERR_SHAPE)
    return mask.shape[1]


def dflash_attention_tree_paged(heads: Heads, q, cu_rows, ctx_len, max_rows, max_ctx_hint, layer, pages: KvPages, mask, out,
                                dev_status, ws: ChunkWorkspace, scale=0.0, trace=None, stream=None):
    """Attention of a ragged batch of trees q [T, Hq, Dh] over the paged cache that
    already holds the nodes' own keys and values; mask [T, words] (int32 bits)."""
    fn = "dflash_attention_tree_paged"
    hq, dh, dt = heads.n_q_heads, heads.head_dim, heads.dtype
    qp, ldq, T = _rows(q, hq, dh, dt, fn)
    op, ldo, n_out = _rows(out, hq, dh, dt, fn)
    if q is None or n_out < T:
        raise DFlashError(fn, ERR_INVALID_ARG if q is None else ERR_SHAPE)
    B, words = ctx_len.numel(), _mask_words(mask, T, fn)
    _check(fn, load().dflash_attention_tree_paged(
        ctypes.byref(heads), qp, ldq, _ints(cu_rows, B + 1, fn), _ints(ctx_len, B, fn), B, T, int(max_rows),
        int(max_ctx_hint), int(layer), _view(pages, heads, ctx_len, fn), mask.data_ptr(), words, float(scale), op, ldo,
        _status(dev_status, fn), ws.ptr, ws.nbytes, _tr(trace),
        _here(stream, fn, q, out, cu_rows, ctx_len, mask, dev_status, getattr(ws, "buf", None))))


def _floats(t, n: int, fn: str):
    """Pointer of a device fp32 vector of at least n entries, None for none."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() < n or not t.is_contiguous():
        raise DFlashError(fn, ERR_SHAPE if t.dtype is torch.float32 else ERR_DTYPE)
    return t.data_ptr()


def dflash_sample(logits, u, tokens, dev_status, temperature=None, top_k=None, top_p=None, min_p=None, probs=None,
                  trace=None, stream=None):
    """Tokens [N] drawn from logits [N, V] by the uniforms u [N] after temperature,
    top-k, top-p and min-p (each a tensor [N] or None), and / or the distributions
    probs [N, V]; u and tokens None: the distributions alone."""
    fn = "dflash_sample"
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise DFlashError(fn, ERR_SHAPE)
    N, V = logits.shape
    ld = max(logits.stride(0), V) if N <= 1 else logits.stride(0)   # the stride of a single row says nothing
    if probs is not None and (probs.shape != (N, V) or not probs.is_contiguous()):
        raise DFlashError(fn, ERR_SHAPE)
    _check(fn, load().dflash_sample(
        logits.data_ptr(), _DTYPES.get(logits.dtype, -1), ld, N, V, _floats(temperature, N, fn),
        _ints(top_k, N, fn) if top_k is not None else None, _floats(top_p, N, fn), _floats(min_p, N, fn), _floats(u, N, fn),
        _ints(tokens, N, fn) if tokens is not None else None, _floats(probs, N * V, fn), _status(dev_status, fn), _tr(trace),
        _here(stream, fn, logits, u, tokens, temperature, top_k, top_p, min_p, probs, dev_status)))


def dflash_verify_tree(tokens, parents, drawn, cu_rows, tau, committed, path, next_anchor, dev_status, heads=None, ctx_len=None,
                       pages=None, trace=None, stream=None):
    """The branch of each tree that the drawn tokens confirm; with heads, ctx_len
    and pages its rows move behind the context in every layer. committed and path
    are [B, max_path]."""
    fn = "dflash_verify_tree"
    T, B = tokens.numel(), cu_rows.numel() - 1
    P = path.shape[-1]
    if committed.shape[-1] != P:
        raise DFlashError(fn, ERR_SHAPE)
    view = None
    if pages is not None:
        if heads is None or ctx_len is None:
            raise DFlashError(fn, ERR_INVALID_ARG)
        if ctx_len.numel() < B:
            raise DFlashError(fn, ERR_SHAPE)
        view = _view(pages, heads, ctx_len, fn)
    _check(fn, load().dflash_verify_tree(
        ctypes.byref(heads) if heads is not None else None, _ints(tokens, T, fn), _ints(parents, T, fn), _ints(drawn, T, fn),
        _ints(cu_rows, B + 1, fn), _ints(ctx_len, B, fn) if ctx_len is not None else None, B, T, P, view, _ints(tau, B, fn),
        _ints(committed, B * P, fn), _ints(path, B * P, fn), _ints(next_anchor, B, fn), _status(dev_status, fn), _tr(trace),
        _here(stream, fn, tokens, parents, drawn, cu_rows, ctx_len, tau, committed, path, next_anchor, dev_status)))


def _book(pages: KvPages, refs, lens, n: int, fn: str):
    """A page view whose table has n rows, and its counts, where the lengths lie."""
    if pages.layout is None or pages.sequences < n:
        raise DFlashError(fn, ERR_SHAPE)
    if pages.device != lens.get_device():
        raise DFlashError(fn, ERR_INVALID_ARG)
    return ctypes.byref(pages), _ints(refs, pages.n_pages, fn)


def dflash_pages_release(pages: KvPages, refs, keep_len, dev_status, trace=None, stream=None):
    """Sequence b keeps the pages of its first keep_len[b] positions."""
    fn = "dflash_pages_release"
    B = keep_len.numel()
    view, counts = _book(pages, refs, keep_len, B, fn)
    _check(fn, load().dflash_pages_release(view, counts, _ints(keep_len, B, fn), B, _status(dev_status, fn), _tr(trace),
                                           _here(stream, fn, refs, keep_len, dev_status)))


def dflash_pages_reserve(pages: KvPages, refs, want_len, dev_status, trace=None, stream=None):
    """Free pages for the missing entries of sequence b's first want_len[b] positions."""
    fn = "dflash_pages_reserve"
    B = want_len.numel()
    view, counts = _book(pages, refs, want_len, B, fn)
    _check(fn, load().dflash_pages_reserve(view, counts, _ints(want_len, B, fn), B, _status(dev_status, fn), _tr(trace),
                                           _here(stream, fn, refs, want_len, dev_status)))


def dflash_pages_fork(heads: Heads, pages: KvPages, refs, ctx_len, src, dst, dev_status, trace=None, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] (ctx_len and the table
    have a row for every sequence)."""
    fn = "dflash_pages_fork"
    n, seqs = src.numel(), ctx_len.numel()
    view = _view(pages, heads, ctx_len, fn)
    _check(fn, load().dflash_pages_fork(
        ctypes.byref(heads), view, _ints(refs, pages.n_pages, fn), _ints(ctx_len, seqs, fn), seqs, _ints(src, n, fn),
        _ints(dst, n, fn), n, _status(dev_status, fn), _tr(trace), _here(stream, fn, refs, ctx_len, src, dst, dev_status)))


class TraceRecorder:
    """Owns CUDA events and host arrays for a dflash_trace."""

    def __init__(self, capacity: int = 512):
        self.capacity = capacity
        self.ev = [torch.cuda.Event(enable_timing=True) for _ in range(2 * capacity)]
        for e in self.ev:      # torch creates the CUDA event on first record
            e.record()
        torch.cuda.synchronize()
        self._events = (ctypes.c_void_p * (2 * capacity))(*[e.cuda_event for e in self.ev])
        self._kinds = (ctypes.c_int * capacity)()
        self._bytes = (ctypes.c_double * capacity)()
        self._flops = (ctypes.c_double * capacity)()
        self.struct = Trace(self._events, capacity, 0, self._kinds, self._bytes, self._flops)

    def reset(self):
        self.struct.count = 0

    def records(self):
        """[(kind, bytes, flops, ms)] of the traced launches (synchronises)."""
        torch.cuda.synchronize()
        out = []
        for i in range(self.struct.count):
            ms = self.ev[2 * i].elapsed_time(self.ev[2 * i + 1])
            out.append((self._kinds[i], self._bytes[i], self._flops[i], ms))
        return out
