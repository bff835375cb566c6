// Per-head RMSNorm of queries and keys with the position rotation in the same
// pass, and the same on the way into a paged KV cache.
//
//   y = R_p( g (.) x / sqrt(mean(x^2) + eps) )     x one head's Dh values
//   R_p: (x_j, x_{j+Dh/2}) turned by the angle p * theta^(-2j/Dh)
//
// A group of Dh/8 lanes takes one (row, head): each lane holds elements
// 4l..4l+3 of the first half and the same of the second, so a rotation's two
// values sit in one thread and only the sum of squares crosses lanes (a fixed
// shuffle tree). A block of 256 threads takes the heads of one row (of two to
// four rows where there are few heads): the row's position, its page and its
// cos / sin values are fetched once for all its heads. Statistics and the
// rotation are fp32; each output is rounded once, to its storage type.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kRowThreads = 256;
constexpr int kHeadsInFlight = 4;   // heads whose loads a group has in flight

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
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
__global__ void __launch_bounds__(kRowThreads) target_rows_kernel(const RowArgs p, int groups_per_row) {
  constexpr int GL = DH / 8;                    // lanes per (row, head)
  constexpr int NG = kRowThreads / GL;          // groups per block
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int group = threadIdx.x / GL, gl = threadIdx.x % GL;
  const int rows_per_block = NG / groups_per_row;
  // groups_per_row is a power of two and a warp's groups may span two rows:
  // the search below runs once per distinct row of the warp
  const int t = blockIdx.x * rows_per_block + group / groups_per_row;
  const int sub = group % groups_per_row;
  bool live = t < p.T;
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
          if (gl == 0 && sub == 0) report(p.dev_status, DFLASH_ERR_CAPACITY);
          live = false;
        } else if (p.rope_cos != nullptr && pos >= p.rope_positions) {
          if (gl == 0 && sub == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
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
      if (gl == 0 && sub == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
      live = false;
    }
  }
  const unsigned group_mask = GL == 32 ? 0xffffffffu : ((1u << GL) - 1u) << (lane / GL * GL);
  if (!live) return;   // whole groups leave together

  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.rope_cos != nullptr) {
    cs = load4(p.rope_cos + static_cast<size_t>(pos) * (DH / 2) + 4 * gl);
    sn = load4(p.rope_sin + static_cast<size_t>(pos) * (DH / 2) + 4 * gl);
  }
  const int hq = p.q != nullptr ? p.n_q_heads : 0, hk = p.k != nullptr ? p.n_kv_heads : 0;
  const int hv = APPEND ? p.n_kv_heads : 0;
  const TI* xq = static_cast<const TI*>(p.q) + t * p.ldq;
  const TI* xk = static_cast<const TI*>(p.k) + t * p.ldk;
  const TI* xv = static_cast<const TI*>(p.v) + t * p.ldv;
  for (int h0 = sub; h0 < hq + hk + hv; h0 += kHeadsInFlight * groups_per_row) {
    float4 lo[kHeadsInFlight], hi[kHeadsInFlight];
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int h = h0 + i * groups_per_row;
      if (h < hq + hk + hv) {
        const TI* x = h < hq ? xq + h * DH : h < hq + hk ? xk + (h - hq) * DH : xv + (h - hq - hk) * DH;
        lo[i] = load4(x + 4 * gl);
        hi[i] = load4(x + DH / 2 + 4 * gl);
      }
    }
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int h = h0 + i * groups_per_row;
      if (h >= hq + hk + hv) break;   // uniform in the group
      float4 a = lo[i], b = hi[i];
      const bool is_v = h >= hq + hk;
      const TO* gain = static_cast<const TO*>(h < hq ? p.g_q : p.g_k);
      if (!is_v) {
        if (gain != nullptr) {
          float ss = a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w;
#pragma unroll
          for (int o = GL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group_mask, ss, o);
          const float r = 1.0f / sqrtf(ss * (1.0f / DH) + p.eps);
          const float4 ga = load4(gain + 4 * gl), gb = load4(gain + DH / 2 + 4 * gl);
          a.x *= r * ga.x; a.y *= r * ga.y; a.z *= r * ga.z; a.w *= r * ga.w;
          b.x *= r * gb.x; b.y *= r * gb.y; b.z *= r * gb.z; b.w *= r * gb.w;
        }
        const float4 u = a, w = b;
        a = make_float4(u.x * cs.x - w.x * sn.x, u.y * cs.y - w.y * sn.y, u.z * cs.z - w.z * sn.z, u.w * cs.w - w.w * sn.w);
        b = make_float4(w.x * cs.x + u.x * sn.x, w.y * cs.y + u.y * sn.y, w.z * cs.z + u.z * sn.z, w.w * cs.w + u.w * sn.w);
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
      store4(y + 4 * gl, a);
      store4(y + DH / 2 + 4 * gl, b);
    }
  }
}

template <typename TI, typename TO, int DH, bool APPEND>
cudaError_t launch_rows(const RowArgs& a, cudaStream_t s, bool pdl) {
  constexpr int NG = kRowThreads / (DH / 8);
  const int heads = (a.q != nullptr ? a.n_q_heads : 0) + (a.k != nullptr ? a.n_kv_heads : 0) +
                    (APPEND ? a.n_kv_heads : 0);
  // groups of a row: as many as it has heads, up to the block's
  int gpr = 1;
  while (gpr < NG && gpr < heads) gpr *= 2;
  const int rpb = NG / gpr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T + rpb - 1) / rpb));
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
