// C ABI of the target-side operators: argument validation and launches of
// dflash_qk_norm_rope, dflash_kv_append_paged, dflash_attention_chunk_paged
// and dflash_verify_probs. Host code only.
#include <cmath>
#include <stdint.h>

#include "internal.h"

using namespace dfl;

namespace {

inline int heads_elem_bytes(const dflash_heads* h) { return h->dtype == DFLASH_BF16 ? 2 : 4; }

// A row operand: 16-byte aligned rows of at least `width` elements.
dflash_status rows_ok(const void* p, long long ld, long long width, int es) {
  if (p == nullptr || ld < width) return DFLASH_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || (ld * es) % 16 != 0) return DFLASH_ERR_ALIGN;
  return DFLASH_OK;
}

bool heads_pages_ok(const dflash_kv_pages* p) {
  return p != nullptr && p->k_pool != nullptr && p->v_pool != nullptr && p->page_table != nullptr &&
         p->n_pages >= 1 && p->pages_per_seq >= 1 &&
         static_cast<long long>(p->pages_per_seq) * DFLASH_PAGE_KEYS <= INT32_MAX;
}

constexpr int kMaxRows = INT32_MAX - 1024;   // row indices of the last block stay in 32 bits

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Element types of the row operators' inputs: cfg.dtype, or fp32 rows (a
// projection's output) stored as bf16.
bool in_type_ok(const dflash_heads* h, dflash_dtype in) {
  return (in == DFLASH_F32 || in == DFLASH_BF16) && (in == h->dtype || in == DFLASH_F32);
}

dflash_status rope_args(const float* c, const float* s, int n) {
  if (c == nullptr && s == nullptr) return DFLASH_OK;
  if (c == nullptr || s == nullptr || n < 1) return DFLASH_ERR_INVALID_ARG;
  return aligned16(c) && aligned16(s) ? DFLASH_OK : DFLASH_ERR_ALIGN;
}

}  // namespace

extern "C" {

dflash_status dflash_check_heads(const dflash_heads* h) {
  if (h == nullptr) return DFLASH_ERR_INVALID_ARG;
  if (h->dtype != DFLASH_BF16 && h->dtype != DFLASH_F32) return DFLASH_ERR_DTYPE;
  if (h->n_layers < 1 || h->n_q_heads < 1 || h->n_kv_heads < 1 || !(h->rms_eps >= 0.f) || !std::isfinite(h->rms_eps))
    return DFLASH_ERR_INVALID_ARG;
  if (h->head_dim != 64 && h->head_dim != 128) return DFLASH_ERR_SHAPE;
  if (h->n_q_heads % h->n_kv_heads != 0 || h->n_q_heads / h->n_kv_heads > DFLASH_MAX_GROUP) return DFLASH_ERR_SHAPE;
  if (h->n_q_heads > 4096 || h->n_layers > 65536) return DFLASH_ERR_SHAPE;
  return DFLASH_OK;
}

dflash_status dflash_qk_norm_rope(const dflash_heads* h, dflash_dtype in_dtype, const void* q, long long ld_q,
                                  const void* k, long long ld_k, const void* g_q, const void* g_k,
                                  const int32_t* positions, const float* rope_cos, const float* rope_sin,
                                  int rope_positions, int T, void* q_out, long long ld_qo, void* k_out,
                                  long long ld_ko, int32_t* dev_status, dflash_trace* trace,
                                  dflash_stream_t stream) {
  dflash_status st = dflash_check_heads(h);
  if (st != DFLASH_OK) return st;
  if (!in_type_ok(h, in_dtype)) return DFLASH_ERR_DTYPE;
  if (T < 0) return DFLASH_ERR_INVALID_ARG;
  if (T == 0) return DFLASH_OK;
  if ((q == nullptr && k == nullptr) || dev_status == nullptr || !trace_ok(trace)) return DFLASH_ERR_INVALID_ARG;
  if ((st = rope_args(rope_cos, rope_sin, rope_positions)) != DFLASH_OK) return st;
  if (rope_cos != nullptr && positions == nullptr) return DFLASH_ERR_INVALID_ARG;
  const int es = heads_elem_bytes(h), is = in_dtype == DFLASH_BF16 ? 2 : 4;
  const long long wq = static_cast<long long>(h->n_q_heads) * h->head_dim, wk = static_cast<long long>(h->n_kv_heads) * h->head_dim;
  if (q != nullptr && ((st = rows_ok(q, ld_q, wq, is)) != DFLASH_OK || (st = rows_ok(q_out, ld_qo, wq, es)) != DFLASH_OK))
    return st;
  if (k != nullptr && ((st = rows_ok(k, ld_k, wk, is)) != DFLASH_OK || (st = rows_ok(k_out, ld_ko, wk, es)) != DFLASH_OK))
    return st;
  if (!aligned16(g_q) || !aligned16(g_k)) return DFLASH_ERR_ALIGN;
  if (T > kMaxRows) return DFLASH_ERR_TOO_LARGE;
  // in place: the same rows; no output over another part's rows
  if ((q != nullptr && q_out == q && (in_dtype != h->dtype || ld_q != ld_qo)) ||
      (k != nullptr && k_out == k && (in_dtype != h->dtype || ld_k != ld_ko)) ||
      (q != nullptr && k != nullptr && (q_out == k || k_out == q || q_out == k_out)))
    return DFLASH_ERR_INVALID_ARG;
  if ((st = check_arch()) != DFLASH_OK) return st;
  RowArgs a{};
  a.q = q; a.k = k; a.ldq = ld_q; a.ldk = ld_k;
  a.q_out = q_out; a.k_out = k_out; a.ldqo = ld_qo; a.ldko = ld_ko;
  a.g_q = g_q; a.g_k = g_k; a.eps = h->rms_eps;
  a.rope_cos = rope_cos; a.rope_sin = rope_sin; a.rope_positions = rope_positions;
  a.T = T; a.n_q_heads = h->n_q_heads; a.n_kv_heads = h->n_kv_heads; a.head_dim = h->head_dim;
  a.in_bf16 = in_dtype == DFLASH_BF16; a.out_bf16 = h->dtype == DFLASH_BF16;
  a.dev_status = dev_status;
  a.positions = positions;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  const double width = static_cast<double>((q != nullptr ? wq : 0) + (k != nullptr ? wk : 0));
  tr.before(DFLASH_K_NORM, T * (width * (is + es) + (rope_cos != nullptr ? 4.0 * h->head_dim : 0.0)), 0);
  const cudaError_t e = launch_target_rows(a, false, s, use_pdl());
  tr.after();
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

dflash_status dflash_kv_append_paged(const dflash_heads* h, dflash_dtype in_dtype, const void* q, long long ld_q,
                                     const void* k, long long ld_k, const void* v, long long ld_v, const void* g_q,
                                     const void* g_k, const float* rope_cos, const float* rope_sin, int rope_positions,
                                     const int32_t* cu_rows, const int32_t* ctx_len, int B, int T, int layer,
                                     const dflash_kv_pages* pages, void* q_out, long long ld_qo, int32_t* dev_status,
                                     dflash_trace* trace, dflash_stream_t stream) {
  dflash_status st = dflash_check_heads(h);
  if (st != DFLASH_OK) return st;
  if (!in_type_ok(h, in_dtype)) return DFLASH_ERR_DTYPE;
  if (T < 0 || B < 0 || layer < 0 || layer >= h->n_layers) return DFLASH_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return DFLASH_OK;
  if (k == nullptr || v == nullptr || cu_rows == nullptr || ctx_len == nullptr || dev_status == nullptr ||
      !heads_pages_ok(pages) || !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  if ((st = rope_args(rope_cos, rope_sin, rope_positions)) != DFLASH_OK) return st;
  const int es = heads_elem_bytes(h), is = in_dtype == DFLASH_BF16 ? 2 : 4;
  const long long wq = static_cast<long long>(h->n_q_heads) * h->head_dim, wk = static_cast<long long>(h->n_kv_heads) * h->head_dim;
  if (q != nullptr && ((st = rows_ok(q, ld_q, wq, is)) != DFLASH_OK || (st = rows_ok(q_out, ld_qo, wq, es)) != DFLASH_OK))
    return st;
  if ((st = rows_ok(k, ld_k, wk, is)) != DFLASH_OK || (st = rows_ok(v, ld_v, wk, is)) != DFLASH_OK) return st;
  if (!aligned16(g_q) || !aligned16(g_k) || !aligned16(pages->k_pool) || !aligned16(pages->v_pool))
    return DFLASH_ERR_ALIGN;
  if (T > kMaxRows) return DFLASH_ERR_TOO_LARGE;
  if (pages->k_pool == pages->v_pool ||
      (q != nullptr && ((q_out == q && (in_dtype != h->dtype || ld_q != ld_qo)) || q_out == k || q_out == v)))
    return DFLASH_ERR_INVALID_ARG;
  if ((st = check_arch()) != DFLASH_OK) return st;
  RowArgs a{};
  a.q = q; a.k = k; a.v = v; a.ldq = ld_q; a.ldk = ld_k; a.ldv = ld_v;
  a.q_out = q_out; a.ldqo = ld_qo;
  a.g_q = g_q; a.g_k = g_k; a.eps = h->rms_eps;
  a.rope_cos = rope_cos; a.rope_sin = rope_sin; a.rope_positions = rope_positions;
  a.T = T; a.n_q_heads = h->n_q_heads; a.n_kv_heads = h->n_kv_heads; a.head_dim = h->head_dim;
  a.in_bf16 = in_dtype == DFLASH_BF16; a.out_bf16 = h->dtype == DFLASH_BF16;
  a.dev_status = dev_status;
  a.cu_rows = cu_rows; a.ctx_len = ctx_len; a.B = B; a.layer = layer;
  a.k_pool = pages->k_pool; a.v_pool = pages->v_pool;
  a.pages = PageView{pages->page_table, pages->n_pages, pages->pages_per_seq};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  const double width = static_cast<double>((q != nullptr ? wq : 0) + 2 * wk);
  tr.before(DFLASH_K_NORM, T * (width * (is + es) + (rope_cos != nullptr ? 4.0 * h->head_dim : 0.0)), 0);
  const cudaError_t e = launch_target_rows(a, true, s, use_pdl());
  tr.after();
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

size_t dflash_attention_chunk_bytes(const dflash_heads* h) {
  if (dflash_check_heads(h) != DFLASH_OK) return 0;
  return kChunkSlots * chunk_slot_floats(h->head_dim) * sizeof(float) +
         static_cast<size_t>(kChunkDescs) * kChunkDescInts * sizeof(int32_t);
}

dflash_status dflash_attention_chunk_paged(const dflash_heads* h, const void* q, long long ld_q,
                                           const int32_t* cu_rows, const int32_t* ctx_len, int B, int T, int max_rows,
                                           int max_ctx_hint, int layer, const dflash_kv_pages* pages, int causal,
                                           float scale, void* out, long long ld_o, int32_t* dev_status, void* ws,
                                           size_t ws_bytes, dflash_trace* trace, dflash_stream_t stream) {
  dflash_status st = dflash_check_heads(h);
  if (st != DFLASH_OK) return st;
  if (T < 0 || B < 0 || max_rows < 0 || max_ctx_hint < 0 || layer < 0 || layer >= h->n_layers || !std::isfinite(scale) ||
      scale < 0.f || (causal != 0 && causal != 1))
    return DFLASH_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return DFLASH_OK;
  if (cu_rows == nullptr || ctx_len == nullptr || dev_status == nullptr || !heads_pages_ok(pages) || !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  const int es = heads_elem_bytes(h);
  const long long wq = static_cast<long long>(h->n_q_heads) * h->head_dim;
  if ((st = rows_ok(q, ld_q, wq, es)) != DFLASH_OK || (st = rows_ok(out, ld_o, wq, es)) != DFLASH_OK) return st;
  if (!aligned16(pages->k_pool) || !aligned16(pages->v_pool) || !aligned16(ws)) return DFLASH_ERR_ALIGN;
  // tensor-map coordinates are 32-bit
  if (static_cast<double>(h->n_layers) * pages->n_pages * h->n_kv_heads > 2147483647.0 ||
      static_cast<long long>(T) * (h->n_q_heads / h->n_kv_heads) > INT32_MAX / 2 || B > INT32_MAX / 256)
    return DFLASH_ERR_TOO_LARGE;
  if (ws == nullptr || ws_bytes < dflash_attention_chunk_bytes(h)) return DFLASH_ERR_WORKSPACE;
  if (q == out) return DFLASH_ERR_INVALID_ARG;
  if ((st = check_arch()) != DFLASH_OK) return st;
  ChunkArgs a{};
  a.q = q; a.out = out; a.ldq = ld_q; a.ldo = ld_o;
  a.cu_rows = cu_rows; a.ctx_len = ctx_len;
  a.B = B; a.T = T; a.layer = layer; a.n_layers = h->n_layers; a.causal = causal;
  // bounds that size the grid; no result depends on them
  const int capacity = pages->pages_per_seq * DFLASH_PAGE_KEYS;
  a.max_rows = max_rows < T ? max_rows : T;
  a.max_ctx = max_ctx_hint < capacity ? max_ctx_hint : capacity;
  a.n_q_heads = h->n_q_heads; a.n_kv_heads = h->n_kv_heads; a.head_dim = h->head_dim;
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(h->head_dim));
  a.k_pool = pages->k_pool; a.v_pool = pages->v_pool;
  a.pages = PageView{pages->page_table, pages->n_pages, pages->pages_per_seq};
  a.dev_status = dev_status;
  a.partials = static_cast<float*>(ws);
  a.desc = reinterpret_cast<int32_t*>(static_cast<float*>(ws) + kChunkSlots * chunk_slot_floats(h->head_dim));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  // as if every sequence had max_ctx_hint context keys (the lengths are on the device)
  const double keys = static_cast<double>(B) * a.max_ctx + T;
  const double bytes = 2.0 * keys * h->n_kv_heads * h->head_dim * es + 2.0 * T * static_cast<double>(wq) * es;
  const double flops = 4.0 * T * static_cast<double>(wq) * (a.max_ctx + (causal ? 0.5 : 1.0) * a.max_rows);
  const cudaError_t e = launch_attention_chunk(a, h->dtype == DFLASH_BF16, s, use_pdl(), tr, bytes, flops);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

dflash_status dflash_verify_probs(const dflash_config* c, const void* target_probs, dflash_dtype probs_dtype,
                                  const float* draft_probs, const int32_t* draft, const int32_t* gamma_b,
                                  const float* u_accept, const float* u_draw, int B, int32_t* tau,
                                  int32_t* committed, int32_t* next_anchor, int32_t* dev_status, dflash_trace* trace,
                                  dflash_stream_t stream) {
  dflash_status st = dflash_check_config(c);
  if (st != DFLASH_OK) return st;
  if (probs_dtype != DFLASH_BF16 && probs_dtype != DFLASH_F32) return DFLASH_ERR_DTYPE;
  if (B < 1 || B > c->max_batch || target_probs == nullptr || draft == nullptr || u_accept == nullptr ||
      u_draw == nullptr || tau == nullptr || committed == nullptr || next_anchor == nullptr || dev_status == nullptr ||
      !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  if (B > (1 << 24) || c->vocab > (1 << 24)) return DFLASH_ERR_TOO_LARGE;
  if ((st = check_arch()) != DFLASH_OK) return st;
  ProbsArgs a{target_probs, probs_dtype == DFLASH_BF16, draft_probs, draft, gamma_b, u_accept, u_draw, B, c->gamma,
              c->vocab, tau, committed, next_anchor, dev_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  const int es = probs_dtype == DFLASH_BF16 ? 2 : 4;
  // the row of the draw, and the drafts' own entries
  const double bytes = static_cast<double>(B) * (c->vocab + c->gamma) * (es + (draft_probs != nullptr ? 4 : 0));
  tr.before(DFLASH_K_VERIFY, bytes, 0);
  const cudaError_t e = launch_verify_probs(a, s, use_pdl());
  tr.after();
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
