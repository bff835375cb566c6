// Drafted trees: the masks and positions that follow from the nodes' parents,
// and the branch that the target's own tokens confirm, with its rows of the
// paged cache.
#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

// ------------------------------------------------------------------ masks
// One thread a node: it walks up its branch and writes its row of bits word by
// word (numbers fall on the way, so no word is met twice). Bound by latency: the
// offsets, the parents, then a step a generation. A block keeps the parents of its
// nodes' sequences in shared memory where they fit, and the offsets of up to kMaskSeqs
// sequences. 64 nodes of some 20 generations 2.6 us; with the tests for words and bad
// parents inside the loop 4.8.
constexpr int kMaskThreads = 128, kMaskSeqs = 512, kMaskNodes = 2048;

__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(const MaskArgs p) {
  __shared__ int s_cu[kMaskSeqs + 1], s_parents[kMaskNodes];
  __shared__ int s_from;
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * kMaskThreads, t = t0 + threadIdx.x;
  const bool few = p.B <= kMaskSeqs;
  if (few)
    for (int i = threadIdx.x; i <= p.B; i += kMaskThreads) s_cu[i] = p.cu_rows[i];
  __syncthreads();
  const int* cu = few ? s_cu : p.cu_rows;
  const int last = min(p.T, cu[p.B]);
  // the sequence of a node: the last one that begins at or before it
  int b = 0, end = p.B;
  while (end - b > 1) {
    const int mid = (b + end) >> 1;
    if (cu[mid] <= t) b = mid; else end = mid;
  }
  const int first = max(cu[b], 0);
  const bool node_is = t < last && t >= first;
  const int ctx = p.positions != nullptr && node_is ? p.ctx_len[b] : 0;
  if (threadIdx.x == 0) s_from = first;
  __syncthreads();
  // parents of the nodes from the first one's sequence on
  const int from = min(s_from, t0), upto = min(last, t0 + kMaskThreads);
  const bool near = upto - from <= kMaskNodes;
  if (near)
    for (int i = from + threadIdx.x; i < upto; i += kMaskThreads) s_parents[i - from] = p.parents[i];
  __syncthreads();
  if (!node_is) return;
  uint32_t* row = p.mask + static_cast<size_t>(t) * p.words;
  int depth = 0;
  // 64 bits at a time, so that the loop is a load, a shift and a test
  auto walk = [&](auto parent_of) {
    int node = t - first, part = node >> 6, up;
    unsigned long long bits = 0ull;
    for (int i = 2 * part + 2; i < p.words; ++i) row[i] = 0u;
    auto flush = [&]() {
      if (2 * part < p.words) row[2 * part] = static_cast<uint32_t>(bits);
      if (2 * part + 1 < p.words) row[2 * part + 1] = static_cast<uint32_t>(bits >> 32);
      bits = 0ull;
    };
    while (true) {
      bits |= 1ull << (node & 63);
      up = parent_of(node);
      if (up < 0 || up >= node) break;
      ++depth;
      node = up;
      if (node >> 6 != part) {
        for (; part > node >> 6; --part) flush();   // parts passed over: zeros
      }
    }
    for (; part >= 0; --part) flush();
    if (up >= node || t - first >= 32 * p.words) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
  };
  if (near && first >= from) walk([&](int node) { return s_parents[first - from + node]; });
  else walk([&](int node) { return __ldg(p.parents + first + node); });
  if (p.positions != nullptr) p.positions[t] = ctx + depth;
}

// ------------------------------------------------------------------ the confirmed branch
// Block (b, y): every block of a sequence finds the branch for itself. All nodes
// are tested at once (a node counts where its token is the one drawn behind its
// parent), each tells its parent of itself, the lowest number wins, and the walk
// is one shared-memory read a node. Then each warp moves the branch's rows in one
// (layer, head, keys or values) after another. Rows only move down: path[j] >= j,
// and a row's source lies above every row written before, so kBatch rounds of rows
// are read, then written, with nothing kept aside. Bound by latency for one sequence
// (36 layers, 8 heads of 128: 2.1 us); 32 of them move 19 MB in 8.6 us, a third of a
// copy's rate: each block first goes through offsets, tokens, path and pages.
constexpr int kTreeThreads = 256, kTreeWarps = kTreeThreads / 32;
constexpr int kMaxPath = DFLASH_MAX_TREE;
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kTreeThreads) verify_tree_kernel(const TreeArgs p) {
  __shared__ int s_child[DFLASH_MAX_TREE];          // the lowest confirmed child of a node
  __shared__ int s_path[kMaxPath];
  __shared__ int s_len;
  __shared__ long long s_from[kMaxPath], s_to[kMaxPath];   // rows in a layer's pool, head 0; -1: stays
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x;
  const int first = min(max(p.cu_rows[b], 0), p.T);
  int n = max(min(p.cu_rows[b + 1], p.T) - first, 0);
  const int32_t *tokens = p.tokens + first, *parents = p.parents + first, *drawn = p.drawn + first;
  const bool writes = blockIdx.y == 0;
  if (n > DFLASH_MAX_TREE || (n > 0 && parents[0] >= 0)) {
    if (threadIdx.x == 0 && writes) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
    n = 0;
  }
  for (int i = threadIdx.x; i < n; i += kTreeThreads) s_child[i] = INT32_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kTreeThreads) {
    const int up = parents[i];
    if (up >= i) {
      if (writes) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
    } else if (up >= 0 && tokens[i] == drawn[up]) {
      atomicMin(&s_child[up], i);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int len = 0;
    for (int at = 0; n > 0 && at != INT32_MAX && len < p.max_path && len < kMaxPath; at = s_child[at]) s_path[len++] = at;
    s_len = len;
  }
  __syncthreads();
  const int len = s_len;
  if (writes) {
    const int last = len > 0 ? drawn[s_path[len - 1]] : -1;
    for (int j = threadIdx.x; j < p.max_path; j += kTreeThreads) {
      p.path[static_cast<size_t>(b) * p.max_path + j] = j < len ? s_path[j] : -1;
      p.committed[static_cast<size_t>(b) * p.max_path + j] = j + 1 < len ? tokens[s_path[j + 1]] : j + 1 == len ? last : -1;
    }
    if (threadIdx.x == 0) {
      p.tau[b] = len;
      p.next_anchor[b] = last;
    }
  }
  if (p.k_pool == nullptr || len < 2) return;
  const int32_t* table = p.pages.table + static_cast<size_t>(b) * p.pages.pages_per_seq;
  const long long ctx = p.ctx_len[b];
  // the row of a position in a layer's pool, head 0; -1 where it has no page
  auto row_at = [&](long long pos) -> long long {
    if (pos >= 0 && pos < static_cast<long long>(p.pages.pages_per_seq) * kPageKeys) {
      const int page = table[pos / kPageKeys];
      if (page >= 0 && page < p.pages.n_pages) return static_cast<long long>(page) * p.n_kv_heads * kPageKeys + pos % kPageKeys;
    }
    if (writes) report(p.dev_status, DFLASH_ERR_CAPACITY);
    return -1;
  };
  for (int j = threadIdx.x; j < len; j += kTreeThreads) {
    const int i = s_path[j];
    const long long from = i == j ? -1 : row_at(ctx + i), to = i == j ? -1 : row_at(ctx + j);
    s_from[j] = to < 0 ? -1 : from;
    s_to[j] = to;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes_row = p.row_bytes / 16, rows = 32 / lanes_row;   // 8, 16 or 32 lanes a row
  const int piece = lane % lanes_row, mine = lane / lanes_row;
  const int slabs = p.n_layers * p.n_kv_heads * 2;
  const size_t layer_rows = static_cast<size_t>(p.pages.n_pages) * p.n_kv_heads * kPageKeys;
  for (int s = blockIdx.y * kTreeWarps + warp; s < slabs; s += gridDim.y * kTreeWarps) {
    const int head = (s >> 1) % p.n_kv_heads, layer = (s >> 1) / p.n_kv_heads;
    uint4* pool = static_cast<uint4*>(s & 1 ? p.v_pool : p.k_pool) +
                  (layer * layer_rows + static_cast<size_t>(head) * kPageKeys) * lanes_row + piece;
    for (int j0 = 0; j0 < len; j0 += kBatch * rows) {
      uint4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int j = j0 + k * rows + mine;
        if (j < len && s_from[j] >= 0) x[k] = pool[s_from[j] * lanes_row];
      }
      __syncwarp();   // all lanes have read before any writes
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int j = j0 + k * rows + mine;
        if (j < len && s_from[j] >= 0) pool[s_to[j] * lanes_row] = x[k];
      }
      __syncwarp();
    }
  }
}

template <typename K, typename A>
cudaError_t launch_one(K kernel, dim3 grid, int threads, cudaStream_t s, bool pdl, const A& a) {
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

cudaError_t launch_tree_masks(const MaskArgs& a, cudaStream_t s, bool pdl) {
  return launch_one(tree_masks_kernel, dim3((a.T + kMaskThreads - 1) / kMaskThreads), kMaskThreads, s, pdl, a);
}

cudaError_t launch_verify_tree(const TreeArgs& a, cudaStream_t s, bool pdl) {
  // a warp a (layer, head, keys or values) while that leaves at most four blocks an SM; then several
  int y = 1;
  if (a.k_pool != nullptr) {
    const long long slabs = 2LL * a.n_layers * a.n_kv_heads, all = 4LL * num_sms_of_current_device();
    const long long want = (slabs + kTreeWarps - 1) / kTreeWarps, room = (all + a.B - 1) / a.B;
    y = static_cast<int>(want < room ? want : room);
  }
  return launch_one(verify_tree_kernel, dim3(a.B, y), kTreeThreads, s, pdl, a);
}

}  // namespace dfl
