// Per-head RMSNorm of queries and keys with the position rotation in the same
// pass, and the same on the way into a paged KV cache.
//
//   y = R_p( g (.) x / sqrt(mean(x^2) + eps) )     x one head's Dh values
//   R_p: (x_j, x_{j+Dh/2}) turned by the angle p * theta^(-2j/Dh)
//
// A group of Dh/16 lanes takes one (row, head): each lane holds elements
// 8l .. 8l+7 of the first half and the same of the second in 16-byte accesses,
// so a rotation's two values sit in one thread and only the sum of squares
// crosses lanes (a fixed shuffle tree). A block of 128 threads takes the heads
// of a few rows: a row's position, its page and its cos / sin values are
// fetched once for all its heads, while the first heads are already on
// their way. Statistics and the rotation are fp32; each output is rounded once,
// to its storage type. Bound by the rows' bytes for many rows, by three
// dependent loads (sequence, lengths or page, tables) for few.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kRowThreads = 128;

// Eight elements as they lie in memory. Rows are read and written once
// (load_once, store8: streaming accesses); gains and tables stay in the caches.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_once(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // bf16 is the upper half of an fp32
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 r[2];
  __device__ __forceinline__ void load(const float* p) {
    r[0] = *reinterpret_cast<const float4*>(p);
    r[1] = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void load_once(const float* p) {
    r[0] = __ldcs(reinterpret_cast<const float4*>(p));
    r[1] = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) { v[4 * i] = r[i].x; v[4 * i + 1] = r[i].y; v[4 * i + 2] = r[i].z; v[4 * i + 3] = r[i].w; }
  }
};
__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p + 4), make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]), two_bf16(v[4], v[5]), two_bf16(v[6], v[7])));
}

// The number of entries of cu[1..B] that are <= t, i.e. the sequence of packed
// row t (B when t lies behind the last one): a 32-ary search by one warp.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, hi = B;   // the count lies in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;   // cu[i] <= t: the count is at least i
    const bool le = i <= hi && cu[i] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    lo += n * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <typename TI, typename TO, int DH, bool APPEND>
__global__ void __launch_bounds__(kRowThreads, sizeof(TI) == 4 ? 7 : 8) target_rows_kernel(const RowArgs p, int groups_per_row) {
  constexpr int GL = DH / 16;                   // lanes per (row, head)
  constexpr int NG = kRowThreads / GL;          // groups per block
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int group = threadIdx.x / GL, gl = threadIdx.x % GL;
  const int rows_per_block = NG / groups_per_row;
  // groups_per_row is a power of two; a warp's groups may span several rows
  const int t = blockIdx.x * rows_per_block + group / groups_per_row;
  // a group's heads: first, first + step, ... (several blocks share a row where there are few)
  const int sub = group % groups_per_row, head0 = sub + blockIdx.y * groups_per_row, step = groups_per_row * gridDim.y;
  const int hq = p.q != nullptr ? p.n_q_heads : 0, hk = p.k != nullptr ? p.n_kv_heads : 0;
  const int heads = hq + hk + (APPEND ? p.n_kv_heads : 0);
  const TI* xq = static_cast<const TI*>(p.q) + t * p.ldq;
  const TI* xk = static_cast<const TI*>(p.k) + t * p.ldk;
  const TI* xv = static_cast<const TI*>(p.v) + t * p.ldv;
  Eight<TI> lo, hi;
  auto fetch = [&](int h) {
    const TI* x = h < hq ? xq + h * DH : h < hq + hk ? xk + (h - hq) * DH : xv + (h - hq - hk) * DH;
    lo.load_once(x + 8 * gl);
    hi.load_once(x + DH / 2 + 8 * gl);
  };
  bool live = t < p.T;
  if (live && head0 < heads) fetch(head0);   // on its way while the row's place is looked up

  int pos = 0, page_row = 0;
  size_t page_base = 0;
  if (APPEND) {
    const int t_first = __shfl_sync(0xffffffffu, t, 0), t_last = __shfl_sync(0xffffffffu, t, 31);
    int b = 0;
    for (int tt = t_first; tt <= t_last; ++tt) {   // warp-uniform bounds
      const int f = find_sequence(p.cu_rows, p.B, tt, lane);
      if (tt == t) b = f;
    }
    live = live && b < p.B;
    if (live) {
      const int first = p.cu_rows[b];
      live = t >= first;
      pos = p.ctx_len[b] + (t - first);
      if (live) {
        int page = -1;
        const int at = pos / kPageKeys;
        if (pos >= 0 && at < p.pages.pages_per_seq)
          page = p.pages.table[static_cast<size_t>(b) * p.pages.pages_per_seq + at];
        if (page < 0 || page >= p.pages.n_pages) {
          if (gl == 0 && head0 == 0) report(p.dev_status, DFLASH_ERR_CAPACITY);
          live = false;
        } else if (p.rope_cos != nullptr && pos >= p.rope_positions) {
          if (gl == 0 && head0 == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
          live = false;
        } else {
          page_row = pos % kPageKeys;
          page_base = (static_cast<size_t>(p.layer) * p.pages.n_pages + page) * p.n_kv_heads;
        }
      }
    }
  } else if (live && p.rope_cos != nullptr) {
    pos = p.positions[t];
    if (pos < 0 || pos >= p.rope_positions) {
      if (gl == 0 && head0 == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
      live = false;
    }
  }
  const unsigned group_mask = ((1u << GL) - 1u) << (lane / GL * GL);
  if (!live) return;   // whole groups leave together

  float cs[8], sn[8];
  const bool turn = p.rope_cos != nullptr;
  if (turn) {
    Eight<float> c, s;
    c.load(p.rope_cos + static_cast<size_t>(pos) * (DH / 2) + 8 * gl);
    s.load(p.rope_sin + static_cast<size_t>(pos) * (DH / 2) + 8 * gl);
    c.get(cs);
    s.get(sn);
  }
  // bf16 rows: the next head's 32 bytes are requested as soon as this one's are in
  // fp32 registers, which costs no register beyond the 64 of eight blocks an SM
  // (32768 rows of 40 heads 117 -> 112 us; three heads in flight took 117
  // registers, half the warps, and 167 us). fp32 rows have 64 bytes a thread in
  // flight and run at 0.97 - 0.99 of a copy without, at seven blocks (eight spill).
  constexpr bool kAhead = sizeof(TI) == 2;
  for (int h = head0; h < heads; h += step) {
    if (!kAhead && h != head0) fetch(h);
    float a[8], b[8];
    lo.get(a);
    hi.get(b);
    if (kAhead && h + step < heads) fetch(h + step);
    const bool is_v = APPEND && h >= hq + hk;
    if (!is_v) {
      const TO* gain = static_cast<const TO*>(h < hq ? p.g_q : p.g_k);
      if (gain != nullptr) {
        Eight<TO> ga, gb;
        ga.load(gain + 8 * gl);
        gb.load(gain + DH / 2 + 8 * gl);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
#pragma unroll
        for (int o = GL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group_mask, ss, o);
        const float r = rsqrtf(ss * (1.0f / DH) + p.eps);
        float g[8];
        ga.get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= r * g[j];
        gb.get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] *= r * g[j];
      }
      if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = a[j], w = b[j];
          a[j] = u * cs[j] - w * sn[j];
          b[j] = w * cs[j] + u * sn[j];
        }
      }
    }
    TO* y;
    if (h < hq) {
      y = static_cast<TO*>(p.q_out) + t * p.ldqo + h * DH;
    } else if (APPEND) {
      const int g = is_v ? h - hq - hk : h - hq;
      y = static_cast<TO*>(is_v ? p.v_pool : p.k_pool) + ((page_base + g) * kPageKeys + page_row) * DH;
    } else {
      y = static_cast<TO*>(p.k_out) + t * p.ldko + (h - hq) * DH;
    }
    store8(y + 8 * gl, a);
    store8(y + DH / 2 + 8 * gl, b);
  }
}

template <typename TI, typename TO, int DH, bool APPEND>
cudaError_t launch_rows(const RowArgs& a, cudaStream_t s, bool pdl) {
  constexpr int NG = kRowThreads / (DH / 16);
  const int heads = (a.q != nullptr ? a.n_q_heads : 0) + (a.k != nullptr ? a.n_kv_heads : 0) +
                    (APPEND ? a.n_kv_heads : 0);
  // Groups of a row. Few rows: as many as the row has heads, for the most loads
  // at once. Many rows: the split that leaves the fewest groups idle in a row's
  // last round (40 heads: 8 groups in 5 rounds, not 32 in 2), of those the one
  // with the most rounds for the row's place and its tables: bf16 down to 4
  // groups, fp32 to 8 (48 heads of a bf16 append 16 / 8 / 4 / 2 groups 62.2 / 60.2
  // / 59.7 / 67.5 us, 40 of an fp32 call 8 / 4 / 2 groups 102.4 / 104.7 / 110.7).
  int gpr = 1;
  while (gpr < NG && gpr < heads) gpr *= 2;
  if (static_cast<long long>(a.T) * gpr > 2LL * NG * 8 * num_sms_of_current_device()) {
    int best = gpr;
    for (int g = gpr; g >= (sizeof(TI) == 2 ? 4 : 8); g /= 2)
      if ((heads + g - 1) / g * g <= (heads + best - 1) / best * best) best = g;
    gpr = best;
  }
  const int rpb = NG / gpr;
  const unsigned blocks = static_cast<unsigned>((a.T + rpb - 1) / rpb);
  // few rows: a head a group, the rest of a row's heads in other blocks
  const unsigned slices = blocks <= 2u * num_sms_of_current_device() ? (heads + gpr - 1) / gpr : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, slices);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, target_rows_kernel<TI, TO, DH, APPEND>, a, gpr);
}

template <typename TI, typename TO>
cudaError_t launch_typed(const RowArgs& a, bool append, cudaStream_t s, bool pdl) {
  if (a.head_dim == 128)
    return append ? launch_rows<TI, TO, 128, true>(a, s, pdl) : launch_rows<TI, TO, 128, false>(a, s, pdl);
  return append ? launch_rows<TI, TO, 64, true>(a, s, pdl) : launch_rows<TI, TO, 64, false>(a, s, pdl);
}

}  // namespace

cudaError_t launch_target_rows(const RowArgs& a, bool append, cudaStream_t s, bool pdl) {
  if (a.head_dim != 64 && a.head_dim != 128) return cudaErrorInvalidValue;
  if (a.in_bf16 && a.out_bf16) return launch_typed<__nv_bfloat16, __nv_bfloat16>(a, append, s, pdl);
  if (!a.in_bf16 && a.out_bf16) return launch_typed<float, __nv_bfloat16>(a, append, s, pdl);
  if (!a.in_bf16 && !a.out_bf16) return launch_typed<float, float>(a, append, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace dfl
