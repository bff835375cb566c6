// Page bookkeeping of a paged cache: which sequence holds which page. The count
// of a page is the number of table entries that name it; 0 is free.
//
// Counts change by atomic additions of whole numbers, whose order does not show.
// Free pages are given out in ascending order to the entries in the order of
// sequences (or pairs), found by prefix sums in one block, so that the result is
// a function of the inputs alone. All of it is a few thousand integers: bound by
// latency, a handful of dependent passes. 128 sequences of up to 4000 positions:
// release 1.4 us, reserve 3.6, a fork of 24 pairs with its copy (8 layers, 8 heads of
// 128, 101 MB read and written) 23.5; 4 sequences of 1000: 1.2, 1.7, and 16.5 for 3
// pairs (36 layers, 57 MB).
#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kListTile = 4 * kThreads;          // counts that a pass over refs looks at
constexpr int kListMax = 2 * kListTile;          // free pages listed at once

__device__ __forceinline__ int pages_of(long long len) { return static_cast<int>((len + kPageKeys - 1) / kPageKeys); }
__device__ __forceinline__ bool is_page(const PagesArgs& p, int e) { return e >= 0 && e < p.n_pages; }

// Entries from `keep` on of a table row become -1 and their pages' counts go down. One warp.
__device__ __forceinline__ void drop_entries(const PagesArgs& p, int32_t* row, int keep, int lane) {
  for (int j = keep + lane; j < p.pages_per_seq; j += 32) {
    const int e = row[j];
    if (e == -1) continue;
    row[j] = -1;
    if (is_page(p, e) && atomicSub(&p.refs[e], 1) <= 0) {
      atomicAdd(&p.refs[e], 1);
      report(p.dev_status, DFLASH_ERR_INVALID_ARG);
    }
  }
}

__global__ void __launch_bounds__(128) pages_release_kernel(const PagesArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (b >= p.B) return;
  drop_entries(p, p.table + static_cast<size_t>(b) * p.pages_per_seq, pages_of(max(p.len[b], 0)), threadIdx.x & 31);
}

// Inclusive sum over the block's threads; `sums` holds kWarps ints.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  int w = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  return v + (warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// Lists the free pages from page *at on, in ascending order, until `want` are
// found, the list may overflow with the next tile, or the pages end. The whole block.
__device__ __forceinline__ int list_free(const PagesArgs& p, int& at, int want, int* list, int* sums) {
  int found = 0;
  while (at < p.n_pages && found < want && found <= kListMax - kListTile) {
    const int i0 = at + 4 * threadIdx.x;
    bool free[4];
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      free[k] = i0 + k < p.n_pages && __ldcg(p.refs + i0 + k) <= 0;
      n += free[k];
    }
    int total;
    int rank = found + block_scan(n, sums, total) - n;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (free[k]) list[rank++] = i0 + k;
    found += total;
    at += kListTile;
  }
  __syncthreads();
  return found;
}

// ------------------------------------------------------------------ reserve
__global__ void __launch_bounds__(kThreads) pages_reserve_kernel(const PagesArgs p) {
  __shared__ int s_off[kMaxReserve + 1];   // missing entries of the sequences before
  __shared__ int s_list[kListMax];
  __shared__ int s_sums[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto wanted = [&](int b) {
    const int n = pages_of(max(p.len[b], 0));
    if (n > p.pages_per_seq && lane == 0) report(p.dev_status, DFLASH_ERR_CAPACITY);
    return min(n, p.pages_per_seq);
  };
  for (int b = warp; b < p.B; b += kWarps) {
    const int32_t* row = p.table + static_cast<size_t>(b) * p.pages_per_seq;
    const int n = wanted(b);
    int missing = 0;
    for (int j = lane; j < n; j += 32) missing += !is_page(p, row[j]);
    missing = __reduce_add_sync(0xffffffffu, missing);
    if (lane == 0) s_off[b + 1] = missing;
  }
  if (threadIdx.x == 0) s_off[0] = 0;
  __syncthreads();
  int need = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int total;
    const int sum = block_scan(b < p.B ? s_off[b + 1] : 0, s_sums, total);
    if (b < p.B) s_off[b + 1] = need + sum;
    need += total;
  }
  __syncthreads();
  int at = 0, base = 0;   // pages looked at, pages given out
  while (base < need) {
    const int found = min(list_free(p, at, need - base, s_list, s_sums), need - base);
    for (int b = warp; b < p.B && found > 0; b += kWarps) {
      const int lo = max(s_off[b], base);   // rank of the first entry of this row that is still missing
      if (s_off[b + 1] <= base || lo >= base + found) continue;
      int32_t* row = p.table + static_cast<size_t>(b) * p.pages_per_seq;
      const int n = min(pages_of(max(p.len[b], 0)), p.pages_per_seq);
      int rank = lo - base;
      for (int j0 = 0; j0 < n && rank < found; j0 += 32) {
        const bool miss = j0 + lane < n && !is_page(p, row[j0 + lane]);
        const unsigned all = __ballot_sync(0xffffffffu, miss);
        const int r = rank + __popc(all & ((1u << lane) - 1u));
        if (miss && r < found) {
          row[j0 + lane] = s_list[r];
          p.refs[s_list[r]] = 1;
        }
        rank += __popc(all);
      }
    }
    base += found;
    __syncthreads();   // the list is read; counts are written before they are looked at again
    if (at >= p.n_pages) break;
  }
  if (base < need && threadIdx.x == 0) report(p.dev_status, DFLASH_ERR_CAPACITY);
}

// ------------------------------------------------------------------ fork
// Whether pair i may be taken: numbers inside the table, a length that fits, a
// target that is no pair's source and no earlier pair's target.
__device__ __forceinline__ bool pair_ok(const PagesArgs& p, const int32_t* src, const int32_t* dst, int i) {
  const int s = src[i], d = dst[i];
  if (s < 0 || s >= p.seqs || d < 0 || d >= p.seqs) return false;
  for (int j = 0; j < p.n; ++j)
    if (src[j] == d || (j < i && dst[j] == d)) return false;
  const int len = p.ctx_len[s];   // no pair's target: not written by this call
  return len >= 0 && len <= static_cast<long long>(p.pages_per_seq) * kPageKeys;
}

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const PagesArgs p) {
  __shared__ int32_t s_src[kMaxForks], s_dst[kMaxForks];
  __shared__ int s_page[kMaxForks];        // the pair's own page; -1 none is needed, -2 left out, -3 not to be had
  __shared__ int s_list[kListMax];
  __shared__ int s_sums[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = threadIdx.x;
  if (i < p.n) {
    s_src[i] = p.src[i];
    s_dst[i] = p.dst[i];
  }
  __syncthreads();
  const bool ok = i < p.n && pair_ok(p, s_src, s_dst, i);
  const int len = ok ? p.ctx_len[s_src[i]] : 0;
  if (i < p.n) s_page[i] = ok ? -1 : -2;
  if (i < p.n && !ok) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
  __syncthreads();
  for (int k = warp; k < p.n; k += kWarps) {
    if (s_page[k] == -2) continue;
    drop_entries(p, p.table + static_cast<size_t>(s_dst[k]) * p.pages_per_seq, 0, lane);
    // a source without one of its pages
    const int32_t* row = p.table + static_cast<size_t>(s_src[k]) * p.pages_per_seq;
    const int n = pages_of(p.ctx_len[s_src[k]]);
    bool whole = true;
    for (int j = lane; j < n; j += 32) whole = whole && is_page(p, row[j]);
    if (!__all_sync(0xffffffffu, whole) && lane == 0) s_page[k] = -3;
  }
  __syncthreads();
  int need;
  const bool part = ok && s_page[i] == -1 && len % kPageKeys != 0;
  const int rank = block_scan(part, s_sums, need) - 1;
  int at = 0;
  const int found = need > 0 ? list_free(p, at, need, s_list, s_sums) : 0;
  if (part) {
    s_page[i] = rank < found ? s_list[rank] : -3;
    if (rank < found) p.refs[s_list[rank]] = 1;
  }
  __syncthreads();
  for (int k = warp; k < p.n; k += kWarps) {
    const int own = s_page[k];
    if (own == -2) continue;
    const int n = own == -3 ? 0 : p.ctx_len[s_src[k]];
    const int32_t* from = p.table + static_cast<size_t>(s_src[k]) * p.pages_per_seq;
    int32_t* to = p.table + static_cast<size_t>(s_dst[k]) * p.pages_per_seq;
    for (int j = lane; j < n / kPageKeys; j += 32) {
      const int e = from[j];
      to[j] = e;
      atomicAdd(&p.refs[e], 1);
    }
    if (lane == 0) {
      if (own >= 0) to[n / kPageKeys] = own;
      p.ctx_len[s_dst[k]] = n;
      if (own == -3) report(p.dev_status, DFLASH_ERR_CAPACITY);
    }
  }
}

// The rows of the forked sequences' last pages: block (slab, pair), a slab the
// rows of one (layer, head, keys or values), which lie side by side. Bound by the
// bytes, read and written once.
constexpr int kCopyThreads = 256, kCopyBatch = 8;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagesArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.y;
  const int s = p.src[i], d = p.dst[i];
  if (s < 0 || s >= p.seqs || d < 0 || d >= p.seqs) return;
  bool clash = false;   // as pair_ok: such a pair was left out
  for (int j = threadIdx.x; j < p.n; j += kCopyThreads) clash = clash || p.src[j] == d || (j < i && p.dst[j] == d);
  const int len = p.ctx_len[s];
  const long long most = static_cast<long long>(p.pages_per_seq) * kPageKeys;
  clash = clash || len < 0 || len > most || p.ctx_len[d] != len;   // or the target was left empty
  if (__syncthreads_or(clash)) return;
  const int rows = len % kPageKeys;
  if (rows == 0) return;
  const int from = p.table[static_cast<size_t>(s) * p.pages_per_seq + len / kPageKeys];
  const int to = p.table[static_cast<size_t>(d) * p.pages_per_seq + len / kPageKeys];
  if (!is_page(p, from) || !is_page(p, to) || from == to) return;
  const int vecs = rows * (p.row_bytes / 16);
  const size_t page_vecs = static_cast<size_t>(kPageKeys) * (p.row_bytes / 16);
  const int slabs = p.n_layers * p.n_kv_heads * 2;
  for (int q = blockIdx.x; q < slabs; q += gridDim.x) {
    const int head = (q >> 1) % p.n_kv_heads, layer = (q >> 1) / p.n_kv_heads;
    uint4* pool = static_cast<uint4*>(q & 1 ? p.v_pool : p.k_pool);
    const size_t base = static_cast<size_t>(layer) * p.n_pages;
    const uint4* x = pool + ((base + from) * p.n_kv_heads + head) * page_vecs;
    uint4* y = pool + ((base + to) * p.n_kv_heads + head) * page_vecs;
    for (int v0 = threadIdx.x; v0 < vecs; v0 += kCopyThreads * kCopyBatch) {
      uint4 t[kCopyBatch];
#pragma unroll
      for (int k = 0; k < kCopyBatch; ++k)
        if (v0 + k * kCopyThreads < vecs) t[k] = __ldcs(x + v0 + k * kCopyThreads);
#pragma unroll
      for (int k = 0; k < kCopyBatch; ++k)
        if (v0 + k * kCopyThreads < vecs) __stcs(y + v0 + k * kCopyThreads, t[k]);
    }
  }
}

template <typename K>
cudaError_t launch_pages(K kernel, dim3 grid, int threads, const PagesArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_pages_release(const PagesArgs& a, cudaStream_t s, bool pdl) {
  return launch_pages(pages_release_kernel, dim3((a.B + 3) / 4), 128, a, s, pdl);
}
cudaError_t launch_pages_reserve(const PagesArgs& a, cudaStream_t s, bool pdl) {
  return launch_pages(pages_reserve_kernel, dim3(1), kThreads, a, s, pdl);
}
cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t s, bool pdl) {
  return launch_pages(pages_fork_kernel, dim3(1), kThreads, a, s, pdl);
}
cudaError_t launch_pages_copy(const PagesArgs& a, cudaStream_t s, bool pdl) {
  return launch_pages(pages_copy_kernel, dim3(2 * a.n_layers * a.n_kv_heads, a.n), kCopyThreads, a, s, pdl);
}

}  // namespace dfl
