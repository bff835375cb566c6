// Verification of drafted tokens against the target's probabilities from
// given random numbers (the rejection-acceptance rule that keeps speculative
// decoding lossless in distribution, "DFlash 블록 확산 디코딩" lossless paragraph):
//   draft j is kept while u_j * q_j(x_j) < p_j(x_j);
//   w = max(p_a - q_a, 0) at the first rejection a (p_a where that has no
//   mass), p_gamma after gamma kept drafts;
//   y = min { v : w_0 + ... + w_v > u * (w_0 + ... + w_{V-1}) }.
// A drafter that draws nothing (greedy drafts, q_j one token) has
// w = p_a without token x_a.
//
// The draw compares a prefix sum over the vocabulary with a threshold, so the
// order and the rounding of the sum would decide which token a border case
// gives. Probabilities are therefore summed as integers, each truncated to a
// multiple of 2^-62 (exact for p >= 2^-38): the sums are exact and do not
// depend on their order, and the threshold floor(u * total) is an exact
// 128-bit product. The acceptance products u * q are exact in 64-bit floats.
//
// One launch: a cluster of kParts CTAs takes a sequence, each a contiguous
// part of its vocabulary, each warp a contiguous part of that. Every CTA runs
// the acceptance test for itself (gamma independent lookups); the parts'
// sums meet through distributed shared memory; the warp whose range holds the
// threshold walks it once more (from L2) to the token.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kParts = 8;            // CTAs of a cluster: the portable maximum
constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kVec = 4;              // entries of a lane's step

// floor(x * 2^62) for 0 <= x <= 1; NaN and negative values count as 0, values
// above 1 as 1.
__device__ __forceinline__ unsigned long long fixed62(float x) {
  const uint32_t u = __float_as_uint(fminf(fmaxf(x, 0.f), 1.f));
  const int e = static_cast<int>(u >> 23);   // 0 .. 127
  const unsigned long long m = static_cast<unsigned long long>((u & 0x7FFFFFu) | 0x800000u) << 39;   // 1.0 = 2^62
  return e == 0 ? 0ull : m >> min(127 - e, 63);
}
// floor(u * total), u clamped to [0, 1 - 2^-24].
__device__ __forceinline__ unsigned long long threshold(float u, unsigned long long total) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(u, 0.f), 0.99999994f));
  const int e = static_cast<int>(b >> 23);   // 0 .. 126
  if (e == 0) return 0ull;                   // below 2^-126
  const unsigned long long m = (b & 0x7FFFFFu) | 0x800000u;   // u = m * 2^(e - 150)
  const unsigned long long hi = __umul64hi(total, m), lo = total * m;
  const int sh = 150 - e;                    // 24 .. 149
  if (sh >= 128) return 0ull;
  if (sh >= 64) return hi >> (sh - 64);
  return (hi << (64 - sh)) | (lo >> sh);     // hi < 2^24: the quotient fits
}
__device__ __forceinline__ float prob_at(const float* p) { return *p; }
__device__ __forceinline__ float prob_at(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long ld_dsmem_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

template <typename TT>
__global__ void __cluster_dims__(kParts, 1, 1) __launch_bounds__(kProbThreads)
    verify_probs_kernel(const ProbsArgs p) {
  __shared__ int s_a;
  __shared__ unsigned long long s_left[kProbWarps], s_all[kProbWarps];   // sums of w and of p_a
  __shared__ unsigned long long s_part[2];
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.x % kParts, b = blockIdx.x / kParts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int V = p.V, R = p.gamma + 1;
  const int g = p.gamma_b == nullptr ? p.gamma : min(max(p.gamma_b[b], 1), p.gamma);
  const TT* target = static_cast<const TT*>(p.target) + static_cast<size_t>(b) * R * V;
  const float* drafter = p.draft_probs == nullptr ? nullptr : p.draft_probs + static_cast<size_t>(b) * p.gamma * V;
  const int32_t* draft = p.draft + static_cast<size_t>(b) * p.gamma;

  if (warp == 0) {
    bool keep = false;
    if (lane < g) {
      const int x = draft[lane];
      if (x >= 0 && x < V) {   // not a token: rejected
        const float pj = prob_at(target + static_cast<size_t>(lane) * V + x);
        const float qj = drafter == nullptr ? 1.f : drafter[static_cast<size_t>(lane) * V + x];
        const float u = p.u_accept[static_cast<size_t>(b) * p.gamma + lane];
        keep = static_cast<double>(u) * static_cast<double>(qj) < static_cast<double>(pj);
      }
    }
    const unsigned no = ~__ballot_sync(0xffffffffu, keep);   // lane g is never kept (g <= 16)
    if (lane == 0) s_a = __ffs(static_cast<int>(no)) - 1;
  }
  __syncthreads();
  const int a = s_a;
  const TT* row = target + static_cast<size_t>(a) * V;
  const float* qrow = a < g && drafter != nullptr ? drafter + static_cast<size_t>(a) * V : nullptr;
  const int out_token = a < g && drafter == nullptr ? draft[a] : -1;   // greedy drafter's rejected token

  // entries [begin, end) of this warp: whole steps of 32 * kVec
  constexpr int kStep = 32 * kVec;
  const int steps = (V + kStep - 1) / kStep, shares = kParts * kProbWarps;
  const int id = part * kProbWarps + warp;
  const int begin = static_cast<int>(static_cast<long long>(steps) * id / shares) * kStep;
  const int end = min(V, static_cast<int>(static_cast<long long>(steps) * (id + 1) / shares) * kStep);
  // weights of the kVec entries from v on: w (left) and p_a (all)
  auto weights = [&](int v, unsigned long long* left, unsigned long long* all) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      left[i] = all[i] = 0ull;
      if (v + i < end) {
        all[i] = fixed62(prob_at(row + v + i));
        const unsigned long long q = qrow != nullptr ? fixed62(qrow[v + i]) : (v + i == out_token ? all[i] : 0ull);
        left[i] = all[i] > q ? all[i] - q : 0ull;
      }
    }
  };
  unsigned long long sum_left = 0ull, sum_all = 0ull;
  for (int v0 = begin; v0 < end; v0 += kStep) {
    unsigned long long l[kVec], w[kVec];
    weights(v0 + lane * kVec, l, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) { sum_left += l[i]; sum_all += w[i]; }
  }
  sum_left = warp_sum(sum_left);
  sum_all = warp_sum(sum_all);
  if (lane == 0) { s_left[warp] = sum_left; s_all[warp] = sum_all; }
  __syncthreads();
  if (threadIdx.x < 2) {
    const unsigned long long* s = threadIdx.x == 0 ? s_left : s_all;
    unsigned long long t = 0ull;
    for (int w = 0; w < kProbWarps; ++w) t += s[w];
    s_part[threadIdx.x] = t;
  }
  cluster_sync();
  // the parts' sums in vocabulary order
  unsigned long long before[2] = {0ull, 0ull}, total[2] = {0ull, 0ull};
#pragma unroll
  for (int r = 0; r < kParts; ++r) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned long long t = ld_dsmem_u64(mapa_shared(smem_u32(&s_part[k]), r));
      if (r < part) before[k] += t;
      total[k] += t;
    }
  }
  cluster_arrive();   // this CTA's reads of its peers are done
  const int k = total[0] > 0ull ? 0 : 1;   // no residual mass: p_a itself
  const unsigned long long thr = threshold(p.u_draw[b], total[k]);
  unsigned long long cum = before[k];
  for (int w = 0; w < warp; ++w) cum += k == 0 ? s_left[w] : s_all[w];
  const unsigned long long mine = k == 0 ? sum_left : sum_all;
  int y = -1;
  if (total[k] == 0ull) {   // nothing to draw from
    if (id == 0 && lane == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
    if (id == 0) y = 0;
  } else if (cum <= thr && thr - cum < mine) {
    for (int v0 = begin; v0 < end; v0 += kStep) {
      unsigned long long l[kVec], w[kVec], c[kVec];
      weights(v0 + lane * kVec, l, w);
      unsigned long long s = 0ull;
#pragma unroll
      for (int i = 0; i < kVec; ++i) { s += k == 0 ? l[i] : w[i]; c[i] = s; }
      unsigned long long incl = s;   // inclusive prefix over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > thr);
      if (hit != 0u) {
        const int src = __ffs(static_cast<int>(hit)) - 1;
        int at = 0;
#pragma unroll
        for (int i = kVec - 1; i >= 0; --i)
          if (cum + (incl - s) + c[i] > thr) at = i;
        y = __shfl_sync(0xffffffffu, v0 + lane * kVec + at, src);
        break;
      }
      cum += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (y >= 0) {   // one warp of the cluster
    if (lane <= p.gamma)
      p.committed[static_cast<size_t>(b) * R + lane] = lane < a ? draft[lane] : (lane == a ? y : -1);
    if (lane == 0) {
      p.tau[b] = a + 1;
      p.next_anchor[b] = y;
    }
  }
  cluster_wait();     // no peer reads this CTA's sums any more
}

template <typename TT>
cudaError_t launch_probs(const ProbsArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * kParts);
  cfg.blockDim = dim3(kProbThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, verify_probs_kernel<TT>, a);
}

}  // namespace

cudaError_t launch_verify_probs(const ProbsArgs& a, cudaStream_t s, bool pdl) {
  if (a.gamma > DFLASH_MAX_GAMMA) return cudaErrorInvalidValue;
  return a.target_bf16 ? launch_probs<__nv_bfloat16>(a, s, pdl) : launch_probs<float>(a, s, pdl);
}

}  // namespace dfl
