// Shared by the chunk attention kernels: how a ragged batch of chunks is cut
// into units of packed rows, and where a unit's keys and pages lie.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {

struct ChunkUnit {
  int b;       // sequence
  int row0;    // its first packed row
  int n;       // its rows (new tokens)
  int ctx;     // its context length
  int tok0;    // the unit's first token of the chunk
};

// Partial rows in a slot: 8 rows x 4 columns are 128 contiguous bytes, so that
// the kernel that holds a row a thread stores, and the merge that takes 8 rows
// of 16 columns a load reads, whole lines. Index of columns 4c .. 4c+3 of row r.
template <int DH>
__device__ __forceinline__ size_t partial_at(int r, int c) {
  return static_cast<size_t>(((r >> 3) * (DH / 4) + c) * 8 + (r & 7)) * 4;
}

// Rows [first, last) of sequence b, kept inside the T rows of q whatever
// cu_rows holds.
__device__ __forceinline__ void chunk_rows(const ChunkArgs& p, int b, int& first, int& n) {
  first = min(max(p.cu_rows[b], 0), p.T);
  n = max(min(p.cu_rows[b + 1], p.T) - first, 0);
}

// Keys that the row of token i sees: positions 0 .. ctx + i, or all of the
// chunk's when not causal, inside the sequence's page table.
__device__ __forceinline__ int row_keys(const ChunkArgs& p, const ChunkUnit& u, int i) {
  const int seen = u.ctx + (p.causal ? i + 1 : u.n);
  return max(0, min(seen, p.pages.pages_per_seq * kPageKeys));
}
// Keys of the unit's last row.
__device__ __forceinline__ int unit_keys(const ChunkArgs& p, const ChunkUnit& u, int n_tok) {
  return row_keys(p, u, u.tok0 + n_tok - 1);
}

// Unit i of tok tokens each, sequences in order; false when there are fewer.
// Called by a converged warp; every lane gets the answer.
__device__ __forceinline__ bool find_unit(const ChunkArgs& p, int tok, int i, int lane, ChunkUnit& u) {
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int first = 0, n = 0;
    if (b0 + lane < p.B) chunk_rows(p, b0 + lane, first, n);
    const int mine = (n + tok - 1) / tok;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    if (i < all) {
      const int src = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, incl > i))) - 1;
      u.b = b0 + src;
      u.row0 = __shfl_sync(0xffffffffu, first, src);
      u.n = __shfl_sync(0xffffffffu, n, src);
      u.tok0 = (i - __shfl_sync(0xffffffffu, incl - mine, src)) * tok;
      u.ctx = p.ctx_len[u.b];
      return true;
    }
    i -= all;
  }
  return false;
}

// Bits off .. off + 15 of a row's mask over the chunk's keys: word off / 32 on,
// nothing behind the last word, and ones below bit 0 (the context, which all see).
__device__ __forceinline__ uint32_t mask_window16(const uint32_t* row, int words, int off) {
  const int at = max(off, 0) >> 5;
  const uint32_t lo = at < words ? __ldg(row + at) : 0u;
  if (off < 0) return off <= -16 ? 0xFFFFu : (lo << -off | ((1u << -off) - 1u)) & 0xFFFFu;
  const uint32_t hi = at + 1 < words ? __ldg(row + at + 1) : 0u;
  return __funnelshift_r(lo, hi, off & 31) & 0xFFFFu;
}

// Reports a sequence whose keys do not fit its page table (they are cut there).
__device__ __forceinline__ void check_capacity(const ChunkArgs& p, const ChunkUnit& u) {
  if (static_cast<long long>(u.ctx) + u.n > static_cast<long long>(p.pages.pages_per_seq) * kPageKeys)
    report(p.dev_status, DFLASH_ERR_CAPACITY);
}

// Pool page of key k of sequence b; an entry outside the pool is reported and
// reads page 0 instead.
__device__ __forceinline__ int page_of(const ChunkArgs& p, int b, int k) {
  const int pg = p.pages.table[static_cast<size_t>(b) * p.pages.pages_per_seq + k / kPageKeys];
  if (pg >= 0 && pg < p.pages.n_pages) return pg;
  report(p.dev_status, DFLASH_ERR_CAPACITY);
  return 0;
}

}  // namespace dfl
