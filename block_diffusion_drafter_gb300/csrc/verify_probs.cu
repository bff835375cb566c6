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
// One launch: a cluster of CTAs takes a sequence, each a contiguous part of its
// vocabulary, each warp a contiguous part of that, in rows of 32 entries of
// which eight are in flight (and the next eight requested). Every CTA runs the
// acceptance test for itself (gamma independent lookups); the parts' sums meet
// through distributed shared memory; the warp whose range holds the threshold
// knows its groups' sums and reads one group once more (from L2) to find the
// token. Bound by latency for few sequences (the drafts, their probabilities, the
// rows, the cluster's join, the group once more: 7 us). For many by no single
// thing: 64 sequences of 151936 entries take 22 us, of which the bytes are 11.6 us at
// a copy's rate and the instructions (20 an entry and its draft's probability) 5 us
// of issue. The chain at both ends is not covered by other CTAs (all are in the same
// phase), and 512 CTAs do not divide over 152 SMs (some hold four, others three).
// Each further 64 sequences take 16.6 us, 4.7 TB/s; the same kernel with one integer
// operation a weight took 19.6 instead of 22 us.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kRows = 8;             // rows of 32 entries that a warp loads at once
constexpr int kOver = 4 << 23;       // 4 in units of 2^-23; 32 of them fit an int
constexpr int kGroups = 8;           // groups of rows whose sums a warp keeps, while no group is longer than
constexpr int kGroupRows = 248;      // rows: the parts of so many entries' sums fit 32 bits
constexpr int kMaxGroups = 40;       // 2^24 entries, 64 warps: 8192 rows, 34 groups

// floor(x * 2^62) for 0 <= x <= 1; NaN and negative values count as 0, values
// above 1 as 1 (a saturating move). The mantissa, 1.0 = 2^62, shifted right by
// 127 - exponent (PTX shifts by 32 and more give 0).
struct Fixed {
  uint32_t lo, hi;
  __device__ __forceinline__ unsigned long long value() const { return static_cast<unsigned long long>(hi) << 32 | lo; }
};
__device__ __forceinline__ Fixed fixed62(float x) {
  const uint32_t u = __float_as_uint(__saturatef(x));
  const uint32_t n = 127u - (u >> 23);
  const uint32_t m = ((u & 0x7FFFFFu) | 0x800000u) << 7;
  Fixed f;
  asm("{\n\t.reg .u32 t, k;\n\t"
      "max.u32 k, %3, 32;\n\tsub.u32 k, k, 32;\n\tshr.u32 t, %2, k;\n\t"
      "shf.r.clamp.b32 %0, 0, t, %3;\n\tshr.u32 %1, %2, %3;\n\t}"
      : "=r"(f.lo), "=r"(f.hi)
      : "r"(m), "r"(n));
  return f;
}
// max(a - b, 0)
__device__ __forceinline__ Fixed minus(Fixed a, Fixed b) {
  Fixed d;
  asm("{\n\t.reg .u32 m;\n\tsub.cc.u32 %0, %2, %4;\n\tsubc.cc.u32 %1, %3, %5;\n\tsubc.u32 m, 0, 0;\n\t"
      "not.b32 m, m;\n\tand.b32 %0, %0, m;\n\tand.b32 %1, %1, m;\n\t}"
      : "=&r"(d.lo), "=&r"(d.hi)
      : "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi));
  return d;
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
__device__ __forceinline__ float prob_at(const float* p) { return __ldg(p); }
__device__ __forceinline__ float prob_at(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

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

// The kRows rows of 32 entries from entry v0 on, this lane's of each: p_a and,
// where the drafter drew (DREW), q_a.
template <typename TT, bool DREW>
struct Chunk {
  float p[kRows], q[DREW ? kRows : 1];
  __device__ __forceinline__ void load(const TT* row, const float* qrow, int v0, int end, int lane) {
    const TT* a = row + v0 + lane;
    const float* b = qrow + v0 + lane;
    if (v0 + 32 * kRows <= end) {   // offsets known at compile time, nothing to test
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        p[i] = prob_at(a + 32 * i);
        if (DREW) q[i] = __ldg(b + 32 * i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool in = v0 + 32 * i + lane < end;
        p[i] = in ? prob_at(a + 32 * i) : 0.f;
        if (DREW) q[i] = in ? __ldg(b + 32 * i) : 0.f;
      }
    }
  }
  // The sum of this lane's weights: w, or p_a itself where the draft is a greedy
  // drafter's and is not `out`. The integers of fixed62 by additions of floats: x
  // = h1 + h2 + r with h1 the multiple of 2^-23 and h2 that of 2^-46 that adding
  // 1 under rounding towards zero cuts off (the bits of the sums count them), and
  // the multiples of 2^-62 in r likewise. Each step is exact, and the bits' offsets
  // cancel between p and q or are taken off. Added to s1, s2, s3 in units of 2^-23,
  // 2^-46 and 2^-62, at most 2^23 an entry (s1 of an entry of one; 248 rows of them
  // fit an int). 20 instructions an entry where
  // fixed62 and minus take 30 (64 sequences: 26.6 -> 22.0 us).
  __device__ __forceinline__ void add(int v0, int lane, int out, int& s1, int& s2, int& s3) const {
    constexpr float kUp = 8388608.f;   // 2^23
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float a = __saturatef(p[i]);
      if (DREW) {
        const float b = fminf(__saturatef(q[i]), a);   // max(a - q, 0) = a - min(q, a)
        const float a1 = __fadd_rz(a, 1.f), b1 = __fadd_rz(b, 1.f);
        s1 += __float_as_int(a1) - __float_as_int(b1);
        const float ra = __fsub_rn(a, __fsub_rn(a1, 1.f)), rb = __fsub_rn(b, __fsub_rn(b1, 1.f));   // < 2^-23
        const float a2 = __fmaf_rz(ra, kUp, 1.f), b2 = __fmaf_rz(rb, kUp, 1.f);
        s2 += __float_as_int(a2) - __float_as_int(b2);
        const float ta = __fmaf_rn(ra, kUp, __fsub_rn(1.f, a2)), tb = __fmaf_rn(rb, kUp, __fsub_rn(1.f, b2));
        s3 += __float_as_int(__fmaf_rz(ta, kUp, 128.f)) - __float_as_int(__fmaf_rz(tb, kUp, 128.f));   // steps of 2^-16
      } else {
        if (v0 + 32 * i + lane == out) a = 0.f;
        const float a1 = __fadd_rz(a, 1.f);
        s1 += __float_as_int(a1) - 0x3F800000;
        const float ra = __fsub_rn(a, __fsub_rn(a1, 1.f));
        const float a2 = __fmaf_rz(ra, kUp, 1.f);
        s2 += __float_as_int(a2) - 0x3F800000;
        const float ta = __fmaf_rn(ra, kUp, __fsub_rn(1.f, a2));
        s3 += __float_as_int(__fmaf_rz(ta, kUp, 128.f)) - 0x43000000;
      }
    }
  }
};

// This warp's entries [begin, end) in groups of whole chunks: the sum of the
// weights of the range, and of each group into sums[]; all ones where the range's
// sum may not fit 64 bits.
template <typename TT, bool DREW>
__device__ __forceinline__ unsigned long long sum_range(const TT* row, const float* qrow, int begin, int end, int group,
                                                        int out, int lane, unsigned long long* sums) {
  constexpr int kChunk = 32 * kRows;
  unsigned long long* next = sums;
  int left = group, s1 = 0, s2 = 0, s3 = 0;
  int coarse = 0;   // this lane's sum in units of 2^-23, less than one off an entry
  Chunk<TT, DREW> even, odd;
  auto take = [&](const Chunk<TT, DREW>& c, int v0) {
    c.add(v0, lane, out, s1, s2, s3);
    left -= kChunk;
    if (left == 0 || v0 + kChunk >= end) {
      const long long x1 = s1, x2 = s2, x3 = s3;   // x2 and x3 may be negative where DREW
      const unsigned long long sum = warp_sum((static_cast<unsigned long long>(x1) << 39) +
                                              (static_cast<unsigned long long>(x2) << 16) +
                                              static_cast<unsigned long long>(x3));
      if (lane == 0) *next = sum;
      ++next;
      coarse = min(coarse + min(s1, kOver), kOver);
      left = group;
      s1 = s2 = s3 = 0;
    }
  };
  if (begin < end) even.load(row, qrow, begin, end, lane);
  for (int v0 = begin; v0 < end; v0 += 2 * kChunk) {   // the next chunk is on its way while one is taken
    const bool two = v0 + kChunk < end;
    if (two) odd.load(row, qrow, v0 + kChunk, end, lane);
    take(even, v0);
    if (v0 + 2 * kChunk < end) even.load(row, qrow, v0 + 2 * kChunk, end, lane);
    if (two) take(odd, v0 + kChunk);
  }
  if (__reduce_add_sync(0xffffffffu, coarse) >= kOver - (end - begin)) return ~0ull;
  unsigned long long all = 0ull;
  __syncwarp();
  for (const unsigned long long* s = sums + lane; s < next; s += 32) all += *s;
  return warp_sum(all);
}

// The first entry of [v0, end) at which the running sum, cum before it, exceeds
// thr, or -1. A lane takes eight neighbouring entries.
template <typename TT>
__device__ __forceinline__ int find_entry(const TT* row, const float* qrow, int v0, int end, int out, int lane,
                                          unsigned long long cum, unsigned long long thr) {
  for (; v0 < end; v0 += 256) {
    const int v = v0 + 8 * lane;
    float p[8], q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = v + i < end && v + i != out ? prob_at(row + v + i) : 0.f;
      q[i] = v + i < end && qrow != nullptr ? __ldg(qrow + v + i) : 0.f;
    }
    unsigned long long w[8], mine = 0ull;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = minus(fixed62(p[i]), fixed62(q[i])).value();
      mine += w[i];
    }
    unsigned long long incl = mine;   // inclusive prefix over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > thr);
    if (hit != 0u) {
      unsigned long long c = cum + incl - mine;
      int n = 0;                      // entries of this lane before the first that exceeds
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c += w[i];
        n += c <= thr;
      }
      return __shfl_sync(0xffffffffu, v + n, __ffs(static_cast<int>(hit)) - 1);
    }
    cum += __shfl_sync(0xffffffffu, incl, 31);
  }
  return -1;
}

template <typename TT, int PARTS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) verify_probs_kernel(const ProbsArgs p) {
  constexpr int kProbWarps = THREADS / 32;
  __shared__ int s_a;
  __shared__ unsigned long long s_warp[2][kProbWarps];   // sums of w and, where w has no mass, of p_a
  __shared__ unsigned long long s_group[kProbWarps][kMaxGroups];
  __shared__ unsigned long long s_part[2];
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.x % PARTS, b = blockIdx.x / PARTS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int V = p.V, R = p.gamma + 1;
  const int g = p.gamma_b == nullptr ? p.gamma : min(max(p.gamma_b[b], 1), p.gamma);
  const TT* target = static_cast<const TT*>(p.target) + static_cast<size_t>(b) * R * V;
  const float* drafter = p.draft_probs == nullptr ? nullptr : p.draft_probs + static_cast<size_t>(b) * p.gamma * V;
  const int32_t* draft = p.draft + static_cast<size_t>(b) * p.gamma;
  const float u_draw = p.u_draw[b];

  if (warp == 0) {
    bool keep = false;
    if (lane < g) {
      const int x = draft[lane];
      const float u = p.u_accept[static_cast<size_t>(b) * p.gamma + lane];
      if (x >= 0 && x < V) {   // not a token: rejected
        // saturated as the draw's weights are: NaN and negative entries are 0, larger ones 1
        const float pj = __saturatef(prob_at(target + static_cast<size_t>(lane) * V + x));
        const float qj = drafter == nullptr ? 1.f : __saturatef(__ldg(drafter + static_cast<size_t>(lane) * V + x));
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
  int out = a < g && drafter == nullptr ? draft[a] : -1;   // greedy drafter's rejected token

  // this warp's entries [begin, end), in groups of whole chunks
  const int rows = (V + 31) / 32, shares = PARTS * kProbWarps, id = part * kProbWarps + warp;
  const int begin = static_cast<int>(static_cast<long long>(rows) * id / shares) * 32;
  const int end = min(V, static_cast<int>(static_cast<long long>(rows) * (id + 1) / shares) * 32);
  const int group = min((((end - begin + 31) / 32 + kGroups - 1) / kGroups + kRows - 1) / kRows * kRows, kGroupRows) * 32;   // entries
  // The sums of this warp, of the warps before it in the part, of the parts before
  // and of all. A sum that may not fit 64 bits is all ones, at each level: seen in
  // its upper 24 bits.
  auto fits = [](unsigned long long t) {
    return __reduce_add_sync(0xffffffffu, static_cast<unsigned>(t >> 40)) < (1u << 24) - 64u;
  };
  unsigned long long mine, before, total;
  bool valid;
  auto join = [&](int k) {
    if (lane == 0) s_warp[k][warp] = mine;
    __syncthreads();
    const unsigned long long w = lane < kProbWarps ? s_warp[k][lane] : 0ull;
    if (warp == 0) {
      const unsigned long long t = fits(w) ? warp_sum(w) : ~0ull;
      if (lane == 0) s_part[k] = t;
    }
    cluster_sync();
    const unsigned long long t = lane < PARTS ? ld_dsmem_u64(mapa_shared(smem_u32(&s_part[k]), lane)) : 0ull;
    valid = fits(t);
    total = warp_sum(t);
    before = warp_sum((lane < part ? t : 0ull) + (lane < warp ? w : 0ull));
  };
  mine = qrow != nullptr ? sum_range<TT, true>(row, qrow, begin, end, group, -1, lane, s_group[warp])
                           : sum_range<TT, false>(row, nullptr, begin, end, group, out, lane, s_group[warp]);
  join(0);
  if (total == 0ull && valid) {   // no residual mass anywhere: p_a itself (the whole cluster goes this way)
    qrow = nullptr;
    out = -1;
    mine = sum_range<TT, false>(row, nullptr, begin, end, group, -1, lane, s_group[warp]);
    join(1);
  }
  cluster_arrive();      // this CTA's reads of its peers are done
  const unsigned long long thr = threshold(u_draw, total);
  unsigned long long cum = before;
  int y = -1;
  if (total == 0ull || !valid) {   // nothing to draw from, or weights that sum to 4 and more
    if (id == 0 && lane == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
    if (id == 0) y = 0;
  } else if (cum <= thr && thr - cum < mine) {
    int v0 = begin;
    for (int at = 0; thr - cum >= s_group[warp][at]; ++at, v0 += group) cum += s_group[warp][at];
    y = find_entry(row, qrow, v0, end, out, lane, cum, thr);
  }
  if (y >= 0) {   // one warp of the cluster
    if (lane <= p.gamma)
      p.committed[static_cast<size_t>(b) * R + lane] = lane < a ? draft[lane] : (lane == a ? y : -1);
    if (lane == 0) {
      p.tau[b] = a + 1;
      p.next_anchor[b] = y;
    }
  }
  cluster_wait();        // no peer reads this CTA's sums any more
}

template <typename TT, int PARTS, int THREADS>
cudaError_t launch_probs(const ProbsArgs& a, cudaStream_t s, bool pdl) {
  if (PARTS > 8) {
    static bool done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!done[dev & 63]) {
      const cudaError_t e =
          cudaFuncSetAttribute(verify_probs_kernel<TT, PARTS, THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      done[dev & 63] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * PARTS);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PARTS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, verify_probs_kernel<TT, PARTS, THREADS>, a);
}

template <typename TT>
cudaError_t launch_typed(const ProbsArgs& a, cudaStream_t s, bool pdl) {
  // CTAs a sequence while two of each SM's slots hold them all: 16 of 256 threads
  // (four slots an SM), then 8 of 512 (two slots), then 8 of 256. Us for 1 / 8 / 16 /
  // 32 / 64 sequences that drew: 16 of 256 6.9 / 8.2 / 11.8 / 17.9 / 28.9, 8 of 512
  // 7.7 / 8.9 / 11.8 / 13.8 / 26.2, 8 of 256 8.9 / 9.8 / 11.9 / 17.5 / 21.9; four of
  // 512 and CTAs of 128 were never the fastest by more than noise.
  const long long slots = 2LL * num_sms_of_current_device();
  if (16LL * a.B <= slots) return launch_probs<TT, 16, 256>(a, s, pdl);
  return 8LL * a.B <= slots ? launch_probs<TT, 8, 512>(a, s, pdl) : launch_probs<TT, 8, 256>(a, s, pdl);
}

}  // namespace

cudaError_t launch_verify_probs(const ProbsArgs& a, cudaStream_t s, bool pdl) {
  if (a.gamma > DFLASH_MAX_GAMMA) return cudaErrorInvalidValue;
  return a.target_bf16 ? launch_typed<__nv_bfloat16>(a, s, pdl) : launch_typed<float>(a, s, pdl);
}

}  // namespace dfl
