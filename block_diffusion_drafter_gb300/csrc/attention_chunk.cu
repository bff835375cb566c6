// Attention of a ragged batch of chunks of new tokens over a paged KV cache:
// row i of sequence b's chunk (position ctx_len[b] + i) attends to keys
// 0 .. ctx_len[b] + i (causal) or to all ctx_len[b] + n_b keys.
//
// The rows of one KV head's G query heads are packed as r = i * G + g, so
// that a key and value tile is read once for all of them, whether the chunk
// has one token or thousands. This file holds the CUDA-core kernel of fp32
// models and the merge of split results; the tcgen05 kernel of bf16 models
// shares the packing and the partial format.
#include "chunk.cuh"

namespace dfl {
namespace {

constexpr float kLog2eC = 1.4426950408889634f;

// ------------------------------------------------------------------ fp32
// One CTA per (unit of 16 RT packed rows, KV head, split). Keys in tiles of
// kSimtKeys through shared memory; thread (ty, tx) of 16 x 16 holds an RT x 4 piece
// of the score tile and rows RT ty.. x columns 4 tx + 64 c .. + 3 of the output. RT is 4,
// or less where the chunks are hinted to have fewer rows (a drafted block of 17
// rows of one head each: 32 rows a unit instead of 64), or 8. Bound by the shared
// memory's bandwidth: 20 16-byte reads for 192 multiply-adds a thread (RT 4, four
// columns of the scores and four keys of the products). Values are on their way
// during the scores and the next keys during the products: 10 sequences of 47 rows
// of 10 heads behind 6681 keys 677 -> 461 us, with 8 rows a thread and the splits
// chosen for whole waves (35 TFLOP/s of fp32).
constexpr int kSimtKeys = 64, kSimtThreads = 256;

template <int DH, int RT>
constexpr size_t simt_smem() {
  return sizeof(float) * (static_cast<size_t>(16 * RT + 2 * kSimtKeys) * (DH + 4) + 16 * RT * (kSimtKeys + 4));
}

// CTAs an SM that leave each variant registers enough to keep its loads together
// (the compiler's own choice, three of 80 registers, spilled: three ragged blocks
// of the tiny shape 14.3 instead of 12.6 us).
template <int DH, int RT>
constexpr int simt_ctas() { return RT == 1 || (DH == 64 && RT <= 4) ? 2 : 1; }

template <int DH, int RT>
__global__ void __launch_bounds__(kSimtThreads, (simt_ctas<DH, RT>())) chunk_simt_kernel(const ChunkArgs p, int splits) {
  extern __shared__ __align__(16) float sm[];
  constexpr int kSimtRows = 16 * RT;
  constexpr int LD = DH + 4, LP = kSimtKeys + 4, DC = DH / 16, D4 = DH / 4;
  float* sq = sm;
  float* sk = sq + kSimtRows * LD;
  float* sv = sk + kSimtKeys * LD;
  float* sp = sv + kSimtKeys * LD;
  pdl_launch_dependents();
  pdl_wait();
  const int G = p.n_q_heads / p.n_kv_heads, tok = kSimtRows / G;
  const int kvh = blockIdx.y, sp_i = blockIdx.z;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  ChunkUnit u;
  const bool have = find_unit(p, tok, static_cast<int>(blockIdx.x), threadIdx.x & 31, u);   // every warp alike
  const int unit = blockIdx.x * p.n_kv_heads + kvh;
  if (splits > 1 && sp_i == 0 && threadIdx.x == 0) {
    int* d = p.desc + unit * kChunkDescInts;
    d[0] = have ? splits : 0;
    d[1] = have ? u.row0 + u.tok0 : 0;
    d[2] = have ? min(tok, u.n - u.tok0) : 0;
    d[3] = kvh;
    d[4] = unit * splits;
    d[5] = unit * splits + 1;
    d[6] = 1;
  }
  if (!have) return;
  if (threadIdx.x == 0) check_capacity(p, u);
  const int n_tok = min(tok, u.n - u.tok0), rows = n_tok * G;
  const int keys = unit_keys(p, u, n_tok);
  // this split's keys: whole tiles
  const int tiles = (keys + kSimtKeys - 1) / kSimtKeys;
  const int t0 = static_cast<int>(static_cast<long long>(tiles) * sp_i / splits);
  const int t1 = static_cast<int>(static_cast<long long>(tiles) * (sp_i + 1) / splits);
  const float* q = static_cast<const float*>(p.q);
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = threadIdx.x; i < kSimtRows * D4; i += kSimtThreads) {
    const int r = i / D4, d = i % D4 * 4;
    *reinterpret_cast<float4*>(&sq[r * LD + d]) =
        r < rows ? *reinterpret_cast<const float4*>(&q[(u.row0 + u.tok0 + r / G) * p.ldq + (kvh * G + r % G) * DH + d]) : none;
  }
  int lim[RT];     // keys that row RT ty + i sees
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = RT * ty + i;
    lim[i] = r < rows ? row_keys(p, u, u.tok0 + r / G) : 0;
  }
  float m[RT], l[RT], o[RT][DC];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DC; ++c) o[i][c] = 0.f;
  }
  const float scale = p.scale * kLog2eC;
  // rows of a tile to shared memory, zeros behind the last key (the rows there may hold anything)
  auto fetch = [&](const void* pool, float* dst, int t) {
    const int k0 = t * kSimtKeys;
    // a tile lies inside one page
    const int page = page_of(p, u.b, k0);
    const size_t base = ((static_cast<size_t>(p.layer) * p.pages.n_pages + page) * p.n_kv_heads + kvh) *
                            static_cast<size_t>(kPageKeys) + k0 % kPageKeys;
    const float* g = static_cast<const float*>(pool) + base * DH;
#pragma unroll
    for (int i = threadIdx.x; i < kSimtKeys * D4; i += kSimtThreads) {
      const int r = i / D4, d = i % D4 * 4;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(&dst[r * LD + d])), "l"(g + r * DH + d),
                   "r"(k0 + r < keys ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (t0 < t1) fetch(p.k_pool, sk, t0);
  for (int t = t0; t < t1; ++t) {   // values come during the scores, the next keys during the products
    const int k0 = t * kSimtKeys;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    fetch(p.v_pool, sv, t);
    float s[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DH; d += 4) {
      float4 a[RT], b[4];
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i] = *reinterpret_cast<const float4*>(&sq[(RT * ty + i) * LD + d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sk[(tx + 16 * j) * LD + d]);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = k0 + tx + 16 * j < lim[i] ? s[i][j] * scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: every term is 0
      const float al = exp2f(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - ref);
        sum += e;
        sp[(RT * ty + i) * LP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * al + sum;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < DC; ++c) o[i][c] *= al;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // also: all threads have left the keys
    if (t + 1 < t1) fetch(p.k_pool, sk, t + 1);
#pragma unroll 2
    for (int j = 0; j < kSimtKeys; j += 4) {
      float pr[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float4 e = *reinterpret_cast<const float4*>(&sp[(RT * ty + i) * LP + j]);
        pr[i][0] = e.x; pr[i][1] = e.y; pr[i][2] = e.z; pr[i][3] = e.w;
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int c = 0; c < DC; c += 4) {
          const float4 v = *reinterpret_cast<const float4*>(&sv[(j + jj) * LD + 4 * tx + 16 * c]);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            o[i][c] += pr[i][jj] * v.x;
            o[i][c + 1] += pr[i][jj] * v.y;
            o[i][c + 2] += pr[i][jj] * v.z;
            o[i][c + 3] += pr[i][jj] * v.w;
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = RT * ty + i;
    if (r >= rows) continue;
    if (splits == 1) {
      const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
      float* y = static_cast<float*>(p.out) + (u.row0 + u.tok0 + r / G) * p.ldo + (kvh * G + r % G) * DH;
#pragma unroll
      for (int c = 0; c < DC; c += 4)
        *reinterpret_cast<float4*>(&y[4 * tx + 16 * c]) = make_float4(o[i][c] * inv, o[i][c + 1] * inv, o[i][c + 2] * inv, o[i][c + 3] * inv);
    } else {
      float* slot = p.partials + static_cast<size_t>(unit * splits + sp_i) * (kSimtRows * (DH + 2));
#pragma unroll
      for (int c = 0; c < DC; c += 4)
        *reinterpret_cast<float4*>(slot + partial_at<DH>(r, tx + 4 * c)) = make_float4(o[i][c], o[i][c + 1], o[i][c + 2], o[i][c + 3]);
      if (tx == 0)
        reinterpret_cast<float2*>(slot + kSimtRows * DH)[r] = make_float2(m[i], l[i]);
    }
  }
}

// ------------------------------------------------------------------ merge
// Joins the partial rows of split units: CTA (unit, x) takes packed rows
// 8x .. 8x+7, a warp a quarter of the columns, a lane four columns of one row.
// The parts' rows, maxima and sums of BATCH splits are requested at once;
// they are added in ascending split order (a batch at a time, under the
// running maximum), so a result does not depend on timing. SLOT_ROWS: rows that a
// part's slot holds.
__device__ __forceinline__ void store_out(float* y, float4 v) { *reinterpret_cast<float4*>(y) = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* y, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(y) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
template <typename T, int DH, int BATCH, int SLOT_ROWS>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const ChunkArgs p) {
  constexpr int NL = DH / 64;   // loads of 16 columns a warp
  pdl_launch_dependents();
  pdl_wait();
  const int* d = p.desc + blockIdx.x * kChunkDescInts;
  const int S = d[0];
  if (S == 0) return;
  const int G = p.n_q_heads / p.n_kv_heads, rows = d[2] * G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = blockIdx.y; g * 8 < rows; g += gridDim.y) {
    const int first = d[4], rest = d[5], step = d[6];
    const int r = g * 8 + (lane & 7), c0 = warp * NL * 4 + (lane >> 3);
    float M = -INFINITY, L = 0.f;
    float4 acc[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += BATCH) {
      float2 ml[BATCH];
      float4 x[BATCH][NL];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (s0 + k < S) {
          const int at = s0 + k == 0 ? first : rest + (s0 + k - 1) * step;
          const float* slot = p.partials + static_cast<size_t>(at) * (SLOT_ROWS * (DH + 2));
          ml[k] = __ldcg(reinterpret_cast<const float2*>(slot + SLOT_ROWS * DH) + r);
#pragma unroll
          for (int i = 0; i < NL; ++i) x[k][i] = __ldcg(reinterpret_cast<const float4*>(slot + partial_at<DH>(r, c0 + 4 * i)));
        }
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
      const float ref = top == -INFINITY ? 0.f : top;
      const float f = exp2f(M - ref);
      L *= f;
#pragma unroll
      for (int i = 0; i < NL; ++i) { acc[i].x *= f; acc[i].y *= f; acc[i].z *= f; acc[i].w *= f; }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (s0 + k < S) {
          const float w = exp2f(ml[k].x - ref);
          L += ml[k].y * w;
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            acc[i].x += x[k][i].x * w; acc[i].y += x[k][i].y * w; acc[i].z += x[k][i].z * w; acc[i].w += x[k][i].w * w;
          }
        }
      }
      M = top;
    }
    if (r < rows) {
      const float inv = L > 0.f ? 1.f / L : 0.f;
      T* y = static_cast<T*>(p.out) + (d[1] + r / G) * p.ldo + (d[3] * G + r % G) * DH;
#pragma unroll
      for (int i = 0; i < NL; ++i)
        store_out(y + (c0 + 4 * i) * 4, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
    }
  }
}

template <typename K, typename... Args>
cudaError_t launch_plain(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, bool pdl, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// How a batch is cut for units of 16 RT rows: units (at most: every sequence's
// last one holds one row), and the splits of their keys that leave the fewest
// tiles one after another, the merge counted as one. cost: in hundredths of the
// time of a tile of 64 rows.
struct SimtPlan {
  long long units, work, cost;
  int splits;
};
template <int DH, int RT>
SimtPlan plan_simt(const ChunkArgs& a) {
  const int tok = 16 * RT / (a.n_q_heads / a.n_kv_heads);
  SimtPlan r{};
  r.units = (static_cast<long long>(a.T) + static_cast<long long>(a.B) * (tok - 1)) / tok;
  r.work = r.units * a.n_kv_heads;
  r.splits = 1;
  const long long hinted = static_cast<long long>(a.B) * ((a.max_rows + tok - 1) / tok) * a.n_kv_heads;
  const long long busy = hinted > 0 && hinted < r.work ? hinted : r.work;   // the rest of the grid finds no unit
  const long long slots = static_cast<long long>(num_sms_of_current_device()) * simt_ctas<DH, RT>();
  const long long tiles = (static_cast<long long>(a.max_ctx) + a.max_rows + kSimtKeys - 1) / kSimtKeys;
  // the workspace holds this many parts of 16 RT rows, and a descriptor a unit
  const long long parts = r.work <= kChunkDescs ? static_cast<long long>(kChunkSlots) * (kChunkRows / (16 * RT)) : 0;
  for (int n = 1; n == 1 || (n <= 64 && n <= tiles && n * r.work <= parts); ++n) {
    const long long waves = (busy * n + slots - 1) / slots;
    const long long cost = waves * ((tiles + n - 1) / n) * (RT == 8 ? 173 : 100) + (n > 1 ? 100 : 0);
    if (n == 1 || cost < r.cost) {
      r.cost = cost;
      r.splits = n;
    }
  }
  return r;
}

template <int DH, int RT>
cudaError_t launch_simt(const ChunkArgs& a, const SimtPlan& plan, cudaStream_t s, bool pdl, Tracer& tr, double bytes,
                        double flops) {
  constexpr int rows = 16 * RT;
  const long long units = plan.units, work = plan.work;
  const int splits = plan.splits;
  constexpr size_t smem = simt_smem<DH, RT>();
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!done[dev & 63]) {
    const cudaError_t e = cudaFuncSetAttribute(chunk_simt_kernel<DH, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    done[dev & 63] = true;
  }
  tr.before(DFLASH_K_ATTN, bytes, flops);
  cudaError_t e = launch_plain(chunk_simt_kernel<DH, RT>,
                               dim3(static_cast<unsigned>(units), a.n_kv_heads, splits), kSimtThreads, smem, s, pdl, a,
                               splits);
  tr.after();
  if (e != cudaSuccess || splits == 1) return e;
  tr.before(DFLASH_K_ATTN, 0.0, 0.0);
  e = launch_plain(chunk_merge_kernel<float, DH, 8, rows>, dim3(static_cast<unsigned>(work), rows / 8), 128, 0, s, pdl, a);
  tr.after();
  return e;
}

template <int DH>
cudaError_t launch_f32(const ChunkArgs& a, cudaStream_t s, bool pdl, Tracer& tr, double bytes, double flops) {
  const int G = a.n_q_heads / a.n_kv_heads;
  const long long rows = static_cast<long long>(a.max_rows) * G;
  if (rows <= 16 && G <= 16) return launch_simt<DH, 1>(a, plan_simt<DH, 1>(a), s, pdl, tr, bytes, flops);
  if (rows <= 32 && G <= 32) return launch_simt<DH, 2>(a, plan_simt<DH, 2>(a), s, pdl, tr, bytes, flops);
  // 128 rows a unit read the shared tiles half as often for their products (2 x 64
  // rows of 28 heads behind 9000 keys 609 -> 529 us), where that leaves CTAs enough.
  const SimtPlan flat = plan_simt<DH, 4>(a);
  if constexpr (DH == 128) {
    if (rows > 64) {
      const SimtPlan tall = plan_simt<DH, 8>(a);
      if (tall.cost < flat.cost) return launch_simt<DH, 8>(a, tall, s, pdl, tr, bytes, flops);
    }
  }
  return launch_simt<DH, 4>(a, flat, s, pdl, tr, bytes, flops);
}

template <int DH>
cudaError_t launch_merge(const ChunkArgs& a, int ctas, int y, cudaStream_t s, bool pdl) {
  // Long chunks have many units, each in two or three parts: two requested at
  // once leave room for more warps than eight (with eight, a 2048-token chunk's
  // merge took 12 us). Few rows behind a long context have one unit in up to 19
  // parts: ten at once, two round trips (17 rows behind 32768 keys, batches of
  // 6 / 8 / 10: 32.6 / 33.1 / 32.5 us; 16 leave too few warps, 35.6).
  return y == kChunkRows / 8 ? launch_plain(chunk_merge_kernel<__nv_bfloat16, DH, 2, kChunkRows>, dim3(ctas, y), 128, 0, s, pdl, a)
                             : launch_plain(chunk_merge_kernel<__nv_bfloat16, DH, 10, kChunkRows>, dim3(ctas, y), 128, 0, s, pdl, a);
}

}  // namespace

// Over few pages units stay whole, each with the CTA in whose range it starts:
// the merge of split ones is a launch of its own and costs more than the pages
// one after another. The hints tell what the longest unit costs (in the ranges'
// measure, 0.39 us each) and the least that equal ranges could take; partial rows
// and merge cost about 35 beside two tiles of rows, 25 beside one, 19 for a token.
// Split / whole, 32 heads over 8, in us: 1 row, 101 keys 9.1 / 7.9, 701 keys 10.5 /
// 13.5; 8 x 17 rows, 317 keys 15.6 / 11.9, 717 keys 17.7 / 15.4; one of them, 717 keys
// 11.7 / 13.8; prompts of 256 / 512 / 1000 tokens 15.8 / 10.6, 18.2 / 13.9, 25.7 / 20.5;
// 300 rows behind 900 keys 21.0 / 27.4. With more units than CTAs some take two:
// whole up to 3 pages, and 6 where the chunk fills a unit (4 x 300 rows behind 300
// keys 29.2 / 24.5, 20 x 2 rows, 702 keys 22.4 / 26.4). Lengths far below the hints
// cost at most the longest unit, so that has 8 pages at most. The figures are those
// of 32 heads over 8 of 128; other layouts follow the same rule.
bool keep_whole(const ChunkArgs& a) {
  const int G = a.n_q_heads / a.n_kv_heads, tok = kChunkRows / G, sms = num_sms_of_current_device();
  const long long rows = static_cast<long long>(a.max_rows) * G;
  const long long pages = (static_cast<long long>(a.max_ctx) + a.max_rows + kPageKeys - 1) / kPageKeys;
  if (pages > 8) return false;
  const long long most = (static_cast<long long>(a.T) + static_cast<long long>(a.B) * (tok - 1)) / tok;
  const long long hinted = static_cast<long long>(a.B) * ((a.max_rows + tok - 1) / tok);
  const long long units = (hinted < most ? hinted : most) * a.n_kv_heads;
  if (units > sms) return pages <= (rows > kChunkRows ? 6 : 3);
  const bool two = rows > kChunkRows / 2;
  const int share = two ? 15 : rows > 32 ? 12 : 9, page = two ? 5 : 4, merge = two ? 35 : rows > 8 ? 25 : 19;
  const long long before = a.causal ? a.max_rows / (2 * kPageKeys) : 0;   // pages that a unit sees less, on average
  return share + page * pages <= units * (share + page * (pages - before)) / sms + merge;
}

cudaError_t launch_attention_chunk(const ChunkArgs& args, int bf16, cudaStream_t s, bool pdl, Tracer& tr, double bytes,
                                   double flops) {
  ChunkArgs a = args;
  if (a.head_dim != 64 && a.head_dim != 128) return cudaErrorInvalidValue;
  if (!bf16)
    return a.head_dim == 128 ? launch_f32<128>(a, s, pdl, tr, bytes, flops) : launch_f32<64>(a, s, pdl, tr, bytes, flops);
  int ctas = 0;
  a.whole_units = keep_whole(a);
  tr.before(DFLASH_K_ATTN, bytes, flops);
  cudaError_t e = launch_chunk_tc(a, &ctas, s, pdl);
  tr.after();
  if (e != cudaSuccess || a.whole_units) return e;
  // the merge's grid covers the rows of the hinted chunk; its CTAs walk on over further rows
  const int G = a.n_q_heads / a.n_kv_heads;
  const long long rows = static_cast<long long>(a.max_rows) * G;
  const int y = static_cast<int>(rows < 8 ? 1 : rows >= kChunkRows ? kChunkRows / 8 : (rows + 7) / 8);
  tr.before(DFLASH_K_ATTN, 0.0, 0.0);
  e = a.head_dim == 128 ? launch_merge<128>(a, ctas, y, s, pdl) : launch_merge<64>(a, ctas, y, s, pdl);
  tr.after();
  return e;
}

}  // namespace dfl
