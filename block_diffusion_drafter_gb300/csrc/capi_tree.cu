// C ABI of the operators around a drafted tree: argument validation and launches
// of dflash_tree_masks, dflash_sample, dflash_verify_tree and dflash_pages_*
// (dflash_attention_tree_paged stands beside the chunk attention in
// capi_target.cu). Host code only.
#include <stdint.h>

#include "internal.h"

using namespace dfl;

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A page view whose table and counts are written.
dflash_status book_ok(const dflash_kv_pages* p, const int32_t* refs) {
  if (p == nullptr || p->page_table == nullptr || refs == nullptr || p->n_pages < 1 || p->pages_per_seq < 1 ||
      static_cast<long long>(p->pages_per_seq) * DFLASH_PAGE_KEYS > INT32_MAX || p->n_pages > INT32_MAX - 8192)
    return DFLASH_ERR_INVALID_ARG;
  return DFLASH_OK;
}

PagesArgs book_args(const dflash_kv_pages* p, int32_t* refs, int32_t* status) {
  PagesArgs a{};
  a.table = const_cast<int32_t*>(p->page_table);
  a.refs = refs;
  a.n_pages = p->n_pages;
  a.pages_per_seq = p->pages_per_seq;
  a.dev_status = status;
  return a;
}

dflash_status pools_ok(const dflash_kv_pages* p) {
  if (p->k_pool == nullptr || p->v_pool == nullptr || p->k_pool == p->v_pool) return DFLASH_ERR_INVALID_ARG;
  return aligned(p->k_pool, 16) && aligned(p->v_pool, 16) ? DFLASH_OK : DFLASH_ERR_ALIGN;
}

int row_bytes(const dflash_heads* h) { return h->head_dim * (h->dtype == DFLASH_BF16 ? 2 : 4); }

dflash_status answer(cudaError_t e) { return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA; }

}  // namespace

extern "C" {

dflash_status dflash_tree_masks(const int32_t* parents, const int32_t* cu_rows, const int32_t* ctx_len, int B, int T,
                                int mask_words, uint32_t* mask, int32_t* positions, int32_t* dev_status,
                                dflash_trace* trace, dflash_stream_t stream) {
  if (T < 0 || B < 0 || mask_words < 0) return DFLASH_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return DFLASH_OK;   // a mask of no words, too
  if (mask_words < 1 || parents == nullptr || cu_rows == nullptr || mask == nullptr || dev_status == nullptr ||
      (positions != nullptr && ctx_len == nullptr) || !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  if (T > INT32_MAX - 1024 || mask_words > INT32_MAX / 32) return DFLASH_ERR_TOO_LARGE;
  const dflash_status st = check_arch();
  if (st != DFLASH_OK) return st;
  const MaskArgs a{parents, cu_rows, ctx_len, B, T, mask_words, mask, positions, dev_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  tr.before(DFLASH_K_NORM, T * (4.0 + 4.0 * mask_words + (positions != nullptr ? 4.0 : 0.0)), 0);
  const cudaError_t e = launch_tree_masks(a, s, use_pdl());
  tr.after();
  return answer(e);
}

dflash_status dflash_sample(const void* logits, dflash_dtype logits_dtype, long long ld, int N, int V,
                            const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                            const float* u, int32_t* tokens, float* probs, int32_t* dev_status, dflash_trace* trace,
                            dflash_stream_t stream) {
  if (logits_dtype != DFLASH_BF16 && logits_dtype != DFLASH_F32) return DFLASH_ERR_DTYPE;
  if (N < 0 || V < 1 || ld < V) return DFLASH_ERR_INVALID_ARG;
  if (N == 0) return DFLASH_OK;
  if (logits == nullptr || dev_status == nullptr || (tokens == nullptr) != (u == nullptr) ||
      (tokens == nullptr && probs == nullptr) || !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  const int es = logits_dtype == DFLASH_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(probs, 4)) return DFLASH_ERR_ALIGN;
  if (N > (1 << 20) || V > kDrawMaxVocab) return DFLASH_ERR_TOO_LARGE;
  if (probs != nullptr) {   // rows of logits are read again after others' distributions are written
    const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(probs);
    if (y < x + (static_cast<uintptr_t>(N - 1) * ld + V) * es && x < y + static_cast<uintptr_t>(N) * V * 4) return DFLASH_ERR_INVALID_ARG;
  }
  const dflash_status st = check_arch();
  if (st != DFLASH_OK) return st;
  const DrawArgs a{logits, ld, es == 2, N, V, temperature, top_k, top_p, min_p, u, tokens, probs, dev_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  tr.before(DFLASH_K_VERIFY, static_cast<double>(N) * V * (es + (probs != nullptr ? 4 : 0)), 0);
  const cudaError_t e = launch_sample_logits(a, s, use_pdl());
  tr.after();
  return answer(e);
}

dflash_status dflash_verify_tree(const dflash_heads* h, const int32_t* tokens, const int32_t* parents,
                                 const int32_t* drawn, const int32_t* cu_rows, const int32_t* ctx_len, int B, int T,
                                 int max_path, const dflash_kv_pages* pages, int32_t* tau, int32_t* committed,
                                 int32_t* path, int32_t* next_anchor, int32_t* dev_status, dflash_trace* trace,
                                 dflash_stream_t stream) {
  dflash_status st;
  if (pages != nullptr && (st = dflash_check_heads(h)) != DFLASH_OK) return st;
  if (B < 0 || T < 0 || max_path < 1) return DFLASH_ERR_INVALID_ARG;
  if (B == 0) return DFLASH_OK;
  if ((T > 0 && (tokens == nullptr || parents == nullptr || drawn == nullptr)) || cu_rows == nullptr || tau == nullptr ||
      committed == nullptr || path == nullptr || next_anchor == nullptr || dev_status == nullptr || !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  if (pages != nullptr) {
    if (ctx_len == nullptr || pages->page_table == nullptr || pages->n_pages < 1 || pages->pages_per_seq < 1 ||
        static_cast<long long>(pages->pages_per_seq) * DFLASH_PAGE_KEYS > INT32_MAX)
      return DFLASH_ERR_INVALID_ARG;
    if ((st = pools_ok(pages)) != DFLASH_OK) return st;
  }
  if ((st = check_arch()) != DFLASH_OK) return st;
  TreeArgs a{tokens, parents, drawn, cu_rows, ctx_len, B, T, max_path, tau, committed, path, next_anchor, dev_status};
  if (pages != nullptr) {
    a.k_pool = pages->k_pool;
    a.v_pool = pages->v_pool;
    a.pages = PageView{pages->page_table, pages->n_pages, pages->pages_per_seq};
    a.n_layers = h->n_layers;
    a.n_kv_heads = h->n_kv_heads;
    a.row_bytes = row_bytes(h);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  // as if every sequence confirmed one node behind its root (the paths are on the device)
  const double moved = pages != nullptr ? 4.0 * B * h->n_layers * h->n_kv_heads * row_bytes(h) : 0.0;
  tr.before(DFLASH_K_VERIFY, 12.0 * T + 8.0 * B * max_path + moved, 0);
  const cudaError_t e = launch_verify_tree(a, s, use_pdl());
  tr.after();
  return answer(e);
}

dflash_status dflash_pages_release(const dflash_kv_pages* pages, int32_t* refs, const int32_t* keep_len, int B,
                                   int32_t* dev_status, dflash_trace* trace, dflash_stream_t stream) {
  dflash_status st = book_ok(pages, refs);
  if (st != DFLASH_OK) return st;
  if (B < 0) return DFLASH_ERR_INVALID_ARG;
  if (B == 0) return DFLASH_OK;
  if (keep_len == nullptr || dev_status == nullptr || !trace_ok(trace)) return DFLASH_ERR_INVALID_ARG;
  if ((st = check_arch()) != DFLASH_OK) return st;
  PagesArgs a = book_args(pages, refs, dev_status);
  a.len = keep_len;
  a.B = B;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  tr.before(DFLASH_K_PAGES, 4.0 * B * pages->pages_per_seq, 0);
  const cudaError_t e = launch_pages_release(a, s, use_pdl());
  tr.after();
  return answer(e);
}

dflash_status dflash_pages_reserve(const dflash_kv_pages* pages, int32_t* refs, const int32_t* want_len, int B,
                                   int32_t* dev_status, dflash_trace* trace, dflash_stream_t stream) {
  dflash_status st = book_ok(pages, refs);
  if (st != DFLASH_OK) return st;
  if (B < 0) return DFLASH_ERR_INVALID_ARG;
  if (B == 0) return DFLASH_OK;
  if (want_len == nullptr || dev_status == nullptr || !trace_ok(trace)) return DFLASH_ERR_INVALID_ARG;
  // missing entries are summed in 32 bits
  if (B > kMaxReserve || static_cast<long long>(B) * pages->pages_per_seq > INT32_MAX) return DFLASH_ERR_TOO_LARGE;
  if ((st = check_arch()) != DFLASH_OK) return st;
  PagesArgs a = book_args(pages, refs, dev_status);
  a.len = want_len;
  a.B = B;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  tr.before(DFLASH_K_PAGES, 4.0 * B * pages->pages_per_seq + 4.0 * pages->n_pages, 0);
  const cudaError_t e = launch_pages_reserve(a, s, use_pdl());
  tr.after();
  return answer(e);
}

dflash_status dflash_pages_fork(const dflash_heads* h, const dflash_kv_pages* pages, int32_t* refs, int32_t* ctx_len,
                                int seqs, const int32_t* src, const int32_t* dst, int n, int32_t* dev_status,
                                dflash_trace* trace, dflash_stream_t stream) {
  dflash_status st = dflash_check_heads(h);
  if (st != DFLASH_OK) return st;
  if ((st = book_ok(pages, refs)) != DFLASH_OK) return st;
  if (n < 0 || seqs < 0) return DFLASH_ERR_INVALID_ARG;
  if (n == 0) return DFLASH_OK;
  if (ctx_len == nullptr || src == nullptr || dst == nullptr || dev_status == nullptr || !trace_ok(trace))
    return DFLASH_ERR_INVALID_ARG;
  if ((st = pools_ok(pages)) != DFLASH_OK) return st;
  if (n > kMaxForks) return DFLASH_ERR_TOO_LARGE;
  if ((st = check_arch()) != DFLASH_OK) return st;
  PagesArgs a = book_args(pages, refs, dev_status);
  a.ctx_len = ctx_len;
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.seqs = seqs;
  a.k_pool = pages->k_pool;
  a.v_pool = pages->v_pool;
  a.n_layers = h->n_layers;
  a.n_kv_heads = h->n_kv_heads;
  a.row_bytes = row_bytes(h);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Tracer tr{trace, s};
  tr.before(DFLASH_K_PAGES, 8.0 * n * pages->pages_per_seq + 4.0 * pages->n_pages, 0);
  cudaError_t e = launch_pages_fork(a, s, use_pdl());
  tr.after();
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  // as if half a page were copied a pair (the lengths are on the device)
  tr.before(DFLASH_K_PAGES, 2.0 * DFLASH_PAGE_KEYS * n * h->n_layers * h->n_kv_heads * row_bytes(h), 0);
  e = launch_pages_copy(a, s, use_pdl());
  tr.after();
  return answer(e);
}

}  // extern "C"
