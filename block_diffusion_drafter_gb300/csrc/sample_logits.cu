// Rows of logits to shaped distributions (temperature, top-k, top-p, min-p) and
// to tokens from given random numbers.
//
//   w_v = exp((x_v - max x) / T), tokens ordered by (x descending, v ascending);
//   top-k keeps the first k, top-p of these the ones with less than p of their
//   weight before them, min-p those with w >= min_p: each a first part of the one
//   order, so all together is a border (a value and, among entries equal to it, a
//   last index);
//   y = min { v : sum of the kept weights up to v > u * their sum }.
//
// Which token a border case gives must not depend on rounding or on an order of
// summation: weights are integers W = floor(w 2^43), computed to about 2^-31 of
// themselves by a function of (x, max, T) alone, and every sum of them is exact.
// At V entries of random weights the drawn token differs from that of exact
// weights with a probability of about sqrt(V) 2^-31 (2^-31 errors add at random
// along the prefix), 2e-7 for 151936 entries; fp32 weights would give 1e-3 from
// the exponent's rounding alone.
//
// A row belongs to a cluster of CTAs, each of which keeps a contiguous part of it
// in shared memory, each warp a contiguous part of that: logits are read from
// HBM once. Borders are found without sorting: a histogram over the candidates
// (a count or a weight a bin), the clusters' bins added through distributed
// shared memory, the border's bin taken apart further. The first level's bins
// are linear in max - x, the further ones cut the range of the values' ordered
// bit patterns, 11 or 10 bits a level, until a bin holds one entry or one value.
// Candidates are few: for top-k, k threads hold an entry of the k-th largest
// thread maximum or more; for top-p, entries below max - T ln(V / (1 - p)) weigh
// less than 1 - p together.
#include <cuda_bf16.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxParts = 16;
constexpr int kCountBins = 2048, kMassBins = 1024;
constexpr int kHistInts = 4096;      // 16 KB: counts, or counts and three parts of a weight
constexpr int kInFlight = 5;         // 16-byte loads a thread
constexpr int kOne = 43;             // the largest weight is 2^43
typedef unsigned long long u64;
constexpr unsigned kAll = 0xffffffffu;

// 2^(j/32), j = 0 .. 31, in two floats (from the exponential's definition).
__device__ const float kPow2[32][2] = {
    {1.0f, 0.0f}, {1.0218971967697144f, -4.811559861650494e-08f}, {1.0442737340927124f, 4.8334701574503924e-08f},
    {1.0671404600143433f, -5.9337519786595294e-08f}, {1.0905077457427979f, -1.3077539939843064e-08f}, {1.114386796951294f, -5.435540018083884e-08f},
    {1.1387885808944702f, 5.386222312608879e-08f}, {1.1637248992919922f, -4.051441493402308e-08f}, {1.1892070770263672f, 3.797635272917432e-08f},
    {1.215247392654419f, -3.267394887984665e-08f}, {1.2418577671051025f, 4.496838101886169e-08f}, {1.2690509557724f, 1.419333317542737e-09f},
    {1.2968395948410034f, -4.018999533172973e-08f}, {1.3252366781234741f, -3.496373324196611e-08f}, {1.3542555570602417f, -1.0123349269974824e-08f},
    {1.3839099407196045f, -5.875577357983275e-08f}, {1.4142135381698608f, 2.4203234971764687e-08f}, {1.4451807737350464f, 3.324199937537742e-08f},
    {1.4768261909484863f, -4.500898853621038e-08f}, {1.5091644525527954f, -2.4959373234878512e-08f}, {1.5422108173370361f, 8.070904833346049e-09f},
    {1.5759809017181396f, -5.661025426206834e-08f}, {1.610490322113037f, 9.836217174097328e-09f}, {1.6457555294036865f, -5.124972091152813e-08f},
    {1.6817928552627563f, -2.4755326677450284e-08f}, {1.7186193466186523f, -4.8496175963919086e-08f}, {1.7562521696090698f, -9.235770370707996e-09f},
    {1.7947090864181519f, -1.141504490931311e-08f}, {1.8340080976486206f, -1.1239277952768134e-08f}, {1.8741676807403564f, -4.663005626071026e-08f},
    {1.9152065515518188f, 9.845328108326612e-09f}, {1.9571441411972046f, -1.7021804410433106e-08f}
};

// A value's place in the order: larger float, larger key; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
__device__ __forceinline__ u64 ld_peer_u64(const void* p, int rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_peer_v4(const void* p, int rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(mapa_shared(smem_u32(p), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void st_peer_u32(const void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "r"(v) : "memory");
}

template <typename TT>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int N = 4;
  static constexpr int kFinal = 0;          // values' keys differ by at least 2^kFinal
  static __device__ __forceinline__ void get(const uint4& q, float* x) {
    x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y); x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 put(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float largest() { return FLT_MAX; }
  static __device__ __forceinline__ uint32_t at_or_below(uint32_t key) { return key; }   // the next value's key
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr int kFinal = 16;
  static __device__ __forceinline__ void get(const uint4& q, float* x) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float* x) {   // of bf16 values
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xFFFF0000u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float largest() { return __uint_as_float(0x7F7F0000u); }
  static __device__ __forceinline__ uint32_t at_or_below(uint32_t key) {
    if (key & 0x80000000u) return key & 0xFFFF0000u;                 // positive: 0x....0000, negative: 0x....FFFF
    return (key & 0xFFFFu) == 0xFFFFu ? key : (key & 0xFFFF0000u) - 1u;
  }
};

// The weight's function: 2^43 exp((x - m) / T), with c = log2(e) / T in two floats.
// s + e = m - x exactly; y = (s + e) c = p + pe; y = i / 32 - r with |r| <= 1/64 + |pe|;
// 2^-y = 2^(-i/32) 2^r, the first factor from the table (a lane an entry, so a
// shuffle is the lookup: no bank conflicts, where a table in shared memory has three
// lanes a bank), the second 1 + q by the exponential's series to r^4 (r^5 term
// below 2^-39). The table's high part, 24 bits, is kept as an integer and only the
// rest is rounded: hi q + lo, below 2^-5, to 2^-36.
struct Weigh {
  float m, ch, cl;
  float hi, lo;              // this lane's table entry
  __device__ __forceinline__ void set(float top, float T, int lane) {
    m = top;
    T = fminf(fmaxf(T, 0x1p-100f), 0x1p100f);
    constexpr float kLh = 1.44269502162933349609375f, kLl = 1.92596303350e-8f;   // log2(e)
    ch = __fdiv_rn(kLh, T);
    cl = __fdiv_rn(__fmaf_rn(-ch, T, kLh) + kLl, T);
    hi = kPow2[lane][0];
    lo = kPow2[lane][1];
  }
  // Called by a whole warp.
  __device__ __forceinline__ u64 operator()(float x) const {
    const float s = __fsub_rn(m, x), bb = __fsub_rn(s, m);
    const float e = __fadd_rn(__fsub_rn(m, __fsub_rn(s, bb)), __fsub_rn(-x, bb));
    float p = __fmul_rn(s, ch);
    float pe = __fmaf_rn(e, ch, __fmaf_rn(s, cl, __fmaf_rn(s, ch, -p)));
    const bool in = p < static_cast<float>(kOne + 1);   // false for -inf (and where s c overflows)
    p = in ? p : 0.f;
    pe = in ? pe : 0.f;
    const float t = __fmaf_rn(p, 32.f, 12582912.f);     // 1.5 2^23: the low bits are round(32 p)
    const int i = 0x4B400000 - __float_as_int(t);       // -round(32 p)
    const float r = __fsub_rn(__fmaf_rn(__fsub_rn(t, 12582912.f), 0.03125f, -p), pe);
    float q = __fmaf_rn(r, 9.618129e-3f, 5.5504109e-2f);
    q = __fmaf_rn(r, q, 0.24022651f);
    q = __fmul_rn(r, __fmaf_rn(r, q, 0.69314718f));
    const float th = __shfl_sync(kAll, hi, i & 31), tl = __shfl_sync(kAll, lo, i & 31);
    const int rest = __float2int_rn(__fmul_rn(__fmaf_rn(th, q, tl), 0x1p36f));
    const u64 mant = (static_cast<u64>((__float_as_uint(th) & 0x7FFFFFu) | 0x800000u) << 13) + static_cast<long long>(rest);
    return in ? (mant << (kOne - 36)) >> (-(i >> 5)) : 0ull;
  }
};

// What stays: entries above `thr`, and of those equal to it the ones up to index `cut`.
struct Border {
  float thr;
  int cut;
  __device__ __forceinline__ bool keeps(float x, int v) const { return x > thr || (x == thr && v <= cut); }
};

struct Shared {
  float warp_f[2][kWarps];
  float2 part_f;                   // the CTA's largest entry, and the least thread maximum
  u64 warp[2][kWarps];             // warps' sums, and the CTA's: two joins in turn
  u64 part[2];
  u64 scan[kWarps];
  u64 above;
  unsigned bin, count;
  int tie;
  double min_log;                  // T ln(min_p)
};

template <typename TT>
__global__ void __launch_bounds__(kThreads, 2) sample_logits_kernel(const DrawArgs p, const int parts, const int rows) {
  using P = Pack<TT>;
  constexpr int VEC = P::N;
  extern __shared__ __align__(16) uint4 s_data[];          // [kWarps][rows][32]
  __shared__ Shared sh;
  unsigned* hist = reinterpret_cast<unsigned*>(s_data + kWarps * rows * 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x / parts, part = blockIdx.x % parts, V = p.V;
  pdl_launch_dependents();
  pdl_wait();

  // ---------------------------------------------------------------- the row
  // 16-byte pieces of the aligned span around the row; entries outside it are -inf.
  const TT* row = static_cast<const TT*>(p.logits) + static_cast<size_t>(n) * p.ld;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(TT));
  const uint4* base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row) & ~static_cast<uintptr_t>(15));
  const int pieces = (shift + V + VEC - 1) / VEC;
  const int first = (part * kWarps + warp) * rows * 32;    // this warp's first piece
  uint4* mine = s_data + warp * rows * 32;
  float top = -INFINITY;
  {
    const float none[8] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
    for (int r0 = 0; r0 < rows; r0 += kInFlight) {
      uint4 q[kInFlight];
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int at = first + (r0 + k) * 32 + lane;
        q[k] = r0 + k < rows && at < pieces ? __ldcs(base + at) : P::put(none);
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        if (r0 + k >= rows) break;
        const int at = first + (r0 + k) * 32 + lane;
        float x[VEC];
        P::get(q[k], x);
        bool odd = at * VEC < shift || (at + 1) * VEC > shift + V;   // also pieces behind the row: -inf already
#pragma unroll
        for (int i = 0; i < VEC; ++i) odd = odd || !(x[i] <= FLT_MAX);   // NaN or +inf
        if (odd) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int v = at * VEC + i - shift;
            if (v < 0 || v >= V || x[i] != x[i]) x[i] = -INFINITY;
            x[i] = fminf(x[i], P::largest());
          }
          q[k] = P::put(x);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) top = fmaxf(top, x[i]);
        mine[(r0 + k) * 32 + lane] = q[k];
      }
    }
  }
  const float thread_top = top;
  const float T_in = p.temperature != nullptr ? p.temperature[n] : 1.f;
  const int k_in = p.top_k != nullptr ? p.top_k[n] : 0;
  const float p_in = p.top_p != nullptr ? p.top_p[n] : 1.f;
  const float min_p = p.min_p != nullptr ? p.min_p[n] : 0.f;
  const bool has_min = min_p > 0.f;
  if (has_min && threadIdx.x == 0) sh.min_log = static_cast<double>(T_in) * log(static_cast<double>(fminf(min_p, 1.f)));

  // f(value, index) of this warp's entries, all lanes together
  auto each = [&](auto f) {
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
      float x[VEC];
      P::get(mine[r * 32 + lane], x);
      const int v0 = (first + r * 32 + lane) * VEC - shift;
#pragma unroll
      for (int i = 0; i < VEC; ++i) f(x[i], v0 + i);
    }
  };
  // Cluster barriers: after reading its peers' memory a CTA tells so (left) and
  // nobody writes there again before all have (settle).
  bool pending = false;
  auto settle = [&]() {
    if (pending) cluster_wait();
    pending = false;
  };
  auto left = [&]() {
    cluster_arrive();
    pending = true;
  };
  auto meet = [&]() {
    settle();
    cluster_sync();
  };

  // ---------------------------------------------------------------- maximum
  float least = thread_top > -INFINITY ? thread_top : INFINITY;   // of the threads' maxima
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    least = fminf(least, __shfl_xor_sync(kAll, least, o));
  }
  if (lane == 0) {
    sh.warp_f[0][warp] = top;
    sh.warp_f[1][warp] = least;
  }
  __syncthreads();
  if (warp == 0) {
    float a = sh.warp_f[0][lane % kWarps], b = sh.warp_f[1][lane % kWarps];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
      b = fminf(b, __shfl_xor_sync(kAll, b, o));
    }
    if (lane == 0) sh.part_f = make_float2(a, b);
  }
  meet();
  {
    const u64 t = ld_peer_u64(&sh.part_f, lane % parts);   // parts divides 32
    top = __uint_as_float(static_cast<uint32_t>(t));
    least = __uint_as_float(static_cast<uint32_t>(t >> 32));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      least = fminf(least, __shfl_xor_sync(kAll, least, o));
    }
  }
  left();
  const float m = top;
  const bool bad = m == -INFINITY || !(T_in >= 0.f);
  float* probs = p.probs != nullptr ? p.probs + static_cast<size_t>(n) * V : nullptr;

  // A sum over the cluster of one value a warp: what lies before this warp, and all.
  int turn = 0;
  auto join = [&](u64 v, u64& before, u64& total) {
    turn ^= 1;
    if (lane == 0) sh.warp[turn][warp] = v;
    __syncthreads();
    const u64 w = lane < kWarps ? sh.warp[turn][lane] : 0ull;
    const u64 all = warp_sum(w);
    if (threadIdx.x == 0) sh.part[turn] = all;
    meet();
    const u64 t = lane < parts ? ld_peer_u64(&sh.part[turn], lane) : 0ull;
    total = warp_sum(t);
    before = warp_sum((lane < part ? t : 0ull) + (lane < warp ? w : 0ull));
    left();
  };
  // The index of the r-th entry (from 1) equal to x, in every CTA.
  auto find_tie = [&](float x, unsigned r) -> int {
    unsigned c = 0;
    each([&](float y, int) { c += y == x; });
    const u64 all = __reduce_add_sync(kAll, c);
    u64 before, total;
    join(all, before, total);
    if (before < r && r <= before + all) {
      unsigned cum = static_cast<unsigned>(before);
      int found = -1;
#pragma unroll 1
      for (int i = 0; i < rows && found < 0; ++i) {
        float y[VEC];
        P::get(mine[i * 32 + lane], y);
        unsigned k = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) k += y[j] == x;
        const unsigned incl = static_cast<unsigned>(warp_scan(k, lane));
        const unsigned hit = __ballot_sync(kAll, cum + incl >= r);
        if (hit != 0u) {
          unsigned at = cum + incl - k;
          int v = (first + i * 32 + lane) * VEC - shift, is = -1;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            at += y[j] == x;
            if (is < 0 && at >= r) is = v + j;
          }
          found = __shfl_sync(kAll, is, __ffs(static_cast<int>(hit)) - 1);
        }
        cum += __shfl_sync(kAll, incl, 31);
      }
      settle();   // nobody reads behind the join any more
      if (lane < parts) st_peer_u32(&sh.tie, lane, static_cast<uint32_t>(found));
    }
    meet();
    return sh.tie;
  };
  auto clear = [&](int ints) {
    settle();
    __syncthreads();
    for (int i = threadIdx.x; i < ints / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  };
  // The bin in which the running sum over the bins (of all CTAs, largest values
  // first) reaches `need` (from 1): sh.bin, what lies above it and the entries in
  // it (0 where not counted); false where the sum stays below.
  auto find_bin = [&](bool mass, bool counted, u64 need) -> bool {
    meet();
    const int per = mass ? 2 : 4, b0 = threadIdx.x * per;
    u64 v[4] = {0ull, 0ull, 0ull, 0ull};
    unsigned cnt[2] = {0u, 0u};
    if (!mass) {
      for (int r = 0; r < parts; ++r) {
        const uint4 c = ld_peer_v4(hist + b0, r);
        v[0] += c.x; v[1] += c.y; v[2] += c.z; v[3] += c.w;
      }
    } else {
#pragma unroll 4
      for (int r = 0; r < parts; ++r) {
        const u64 c = counted ? ld_peer_u64(hist + b0, r) : 0ull;
        const u64 a0 = ld_peer_u64(hist + kMassBins + b0, r), a1 = ld_peer_u64(hist + 2 * kMassBins + b0, r),
                  a2 = ld_peer_u64(hist + 3 * kMassBins + b0, r);
        cnt[0] += static_cast<unsigned>(c);
        cnt[1] += static_cast<unsigned>(c >> 32);
        v[0] += (a0 & kAll) + ((a1 & kAll) << 14) + ((a2 & kAll) << 29);
        v[1] += (a0 >> 32) + ((a1 >> 32) << 14) + ((a2 >> 32) << 29);
      }
    }
    left();
    const u64 own = v[0] + v[1] + v[2] + v[3];
    u64 incl = warp_scan(own, lane);
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    u64 total = 0ull, before = 0ull;
    {
      const u64 w = lane < kWarps ? sh.scan[lane] : 0ull;
      total = warp_sum(w);
      before = warp_sum(lane < warp ? w : 0ull);
    }
    incl += before;
    if (total >= need && incl - own < need && need <= incl) {
      u64 cum = incl - own;
      int b = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (b == k && k + 1 < per && cum + v[k] < need) {
          cum += v[k];
          ++b;
        }
      }
      sh.bin = b0 + b;
      sh.above = cum;
      sh.count = mass ? cnt[b & 1] : static_cast<unsigned>(b == 0 ? v[0] : b == 1 ? v[1] : b == 2 ? v[2] : v[3]);
    }
    __syncthreads();
    return total >= need;
  };
  // Linear bins of 2^-s below m, and the range of keys of one of them: with the
  // difference rounded down and b 2^-s exact, entry x is in bin b just where
  // m - (b + 1) 2^-s < x <= m - b 2^-s.
  auto linear_scale = [&](float lowest, int bins) -> float {
    const float range = fminf(__fsub_ru(m, lowest), FLT_MAX);
    const int e = range > 0.f ? max(ilogbf(range) + 1, -100) : -100;   // a difference rounded down is below 2^e
    return ldexpf(static_cast<float>(bins), -e);                       // bins is a power of two
  };
  auto linear_bin = [&](float x, float scale) { return __float2uint_rz(__fsub_rd(m, x) * scale); };
  auto linear_edge = [&](int b, float scale) { return __fsub_rd(m, static_cast<float>(b) / scale); };   // exact quotient

  Border keep{-FLT_MAX, INT32_MAX};
  const bool greedy = T_in == 0.f || k_in == 1;
  Weigh weigh;
  weigh.set(m, greedy ? 1.f : T_in, lane);
  int token = 0;
  u64 total = 0ull;
  if (bad) {
    if (part == 0 && threadIdx.x == 0) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
    keep = Border{FLT_MAX, -1};   // nothing stays
  } else if (greedy) {
    token = find_tie(m, 1u);
    keep = Border{m, token};
    total = 1ull << kOne;
  } else {
    // -------------------------------------------------------------- top-k
    if (k_in > 1 && k_in < V) {
      u64 need = static_cast<u64>(k_in);
      uint32_t lo = key_of(-FLT_MAX), hi = key_of(m);
      float scale = 0.f;
      // k threads have a maximum in or above this bin
      if (k_in <= parts * kThreads) {
        scale = linear_scale(least, kCountBins);
        clear(kCountBins);
        const unsigned b = linear_bin(thread_top, scale);
        if (b < kCountBins) atomicAdd(&hist[b], 1u);
        const bool found = find_bin(false, true, need);
        if (found) lo = max(lo, key_of(linear_edge(static_cast<int>(sh.bin) + 1, scale)) + 1u);
        scale = found ? linear_scale(value_of(lo), kCountBins) : 0.f;
      }
      while (true) {
        const float flo = value_of(lo), fhi = value_of(hi);
        const uint32_t range = hi - lo;
        int step = max(0, 32 - __clz(range) - 11);
        if (step <= P::kFinal) step = P::kFinal;
        const bool linear = scale > 0.f;
        clear(kCountBins);
        each([&](float x, int) {
          if (x >= flo && x <= fhi) {
            const unsigned b = linear ? linear_bin(x, scale) : (hi - key_of(x)) >> step;
            if (b < kCountBins) atomicAdd(&hist[b], 1u);
          }
        });
        if (!find_bin(false, true, need)) break;        // fewer finite entries than k: all stay
        need -= sh.above;
        const unsigned bin = sh.bin, count = sh.count;
        uint32_t next_lo, next_hi;
        if (linear) {
          next_hi = min(hi, key_of(linear_edge(static_cast<int>(bin), scale)));
          next_lo = max(lo, key_of(linear_edge(static_cast<int>(bin) + 1, scale)) + 1u);
        } else {
          next_hi = hi - (bin << step);
          next_lo = max(lo, next_hi - ((1u << step) - 1u));
        }
        if (need == count) {
          keep.thr = value_of(next_lo);
          break;
        }
        if (!linear && step == P::kFinal) {             // one value
          keep.thr = value_of(P::at_or_below(next_hi));
          keep.cut = find_tie(keep.thr, static_cast<unsigned>(need));
          break;
        }
        lo = next_lo;
        hi = next_hi;
        scale = 0.f;
      }
    }
    // -------------------------------------------------------------- top-p
    if (p_in < 1.f) {
      const Border from = keep;
      // entries below weigh less than 1 - p together, the largest alone weighs 1
      const float y0 = log2f(static_cast<float>(V) / (1.f - fmaxf(p_in, 0.f))) + 0.25f;
      float cut = fmaxf(__fsub_rd(m, y0 / weigh.ch * 1.0001f), -FLT_MAX);
      cut = fmaxf(cut, from.thr);
      uint32_t lo = key_of(cut), hi = key_of(m);
      float scale = linear_scale(cut, kMassBins);
      u64 need = 0ull, base = 0ull;
      bool once = true;
      while (true) {
        const float flo = value_of(lo), fhi = value_of(hi);
        const uint32_t range = hi - lo;
        int step = max(0, 32 - __clz(range) - 10);
        if (step <= P::kFinal) step = P::kFinal;
        const bool linear = once;
        clear(kHistInts);
        u64 sum = 0ull;
        each([&](float x, int v) {
          const bool in = once ? from.keeps(x, v) : x >= flo && x <= fhi && from.keeps(x, v);
          if (__any_sync(kAll, in)) {
            const u64 w = weigh(x);
            if (in) {
              sum += w;
              if (x >= flo) {
                const unsigned b = linear ? linear_bin(x, scale) : (hi - key_of(x)) >> step;
                if (b < kMassBins) {
                  if (!once) atomicAdd(&hist[b], 1u);
                  atomicAdd(&hist[kMassBins + b], static_cast<unsigned>(w) & 0x3FFFu);
                  atomicAdd(&hist[2 * kMassBins + b], static_cast<unsigned>(w >> 14) & 0x7FFFu);
                  atomicAdd(&hist[3 * kMassBins + b], static_cast<unsigned>(w >> 29));
                }
              }
            }
          }
        });
        if (once) {   // the weight of all that top-k left, and how much of it has to lie up to the border
          u64 before, all;
          join(warp_sum(sum), before, all);
          bool whole;
          need = draw_threshold(fmaxf(p_in, 0.f), all, whole);
          if (!whole || need == 0ull) ++need;
        }
        if (!find_bin(true, !once, need - base)) break;    // not reached: rounding of the cut; all stay
        base += sh.above;
        const unsigned bin = sh.bin, count = sh.count;
        uint32_t next_lo, next_hi;
        if (linear) {
          next_hi = min(hi, key_of(linear_edge(static_cast<int>(bin), scale)));
          next_lo = max(lo, key_of(linear_edge(static_cast<int>(bin) + 1, scale)) + 1u);
        } else {
          next_hi = hi - (bin << step);
          next_lo = max(lo, next_hi - ((1u << step) - 1u));
        }
        if (!once && count == 1u) {
          const float x = value_of(next_lo);
          keep = x <= from.thr ? from : Border{x, INT32_MAX};
          break;
        }
        if (!linear && step == P::kFinal) {                // one value
          const float x = value_of(P::at_or_below(next_hi));
          const u64 w = weigh(x), left_over = need - base;   // w > 0: the sum reaches past `base` in this bin
          const u64 r = (left_over + w - 1ull) / w;
          if (r < count) keep = Border{x, find_tie(x, static_cast<unsigned>(r))};
          else keep = x == from.thr ? from : Border{x, INT32_MAX};
          break;
        }
        lo = next_lo;
        hi = next_hi;
        once = false;
      }
    }
    // -------------------------------------------------------------- min-p
    if (has_min) {
      const float x = fminf(__double2float_ru(static_cast<double>(m) + sh.min_log), m);
      if (x > keep.thr) keep = Border{x, INT32_MAX};
    }
    // -------------------------------------------------------------- draw
    u64 sum = 0ull;
    each([&](float x, int v) {
      const bool in = keep.keeps(x, v);
      if (__any_sync(kAll, in)) {
        const u64 w = weigh(x);
        if (in) sum += w;
      }
    });
    sum = warp_sum(sum);
    u64 cum;
    join(sum, cum, total);
    if (p.tokens != nullptr) {
      bool whole;
      const u64 thr = draw_threshold(p.u[n], total, whole);
      if (cum <= thr && thr - cum < sum) {   // one warp of the cluster
#pragma unroll 1
        for (int r = 0; r < rows; ++r) {
          float x[VEC];
          P::get(mine[r * 32 + lane], x);
          const int v0 = (first + r * 32 + lane) * VEC - shift;
          u64 w[VEC], own = 0ull;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const u64 t = weigh(x[i]);
            w[i] = keep.keeps(x[i], v0 + i) ? t : 0ull;
            own += w[i];
          }
          const u64 incl = warp_scan(own, lane);
          const unsigned hit = __ballot_sync(kAll, cum + incl > thr);
          if (hit != 0u) {
            u64 c = cum + incl - own;
            int k = 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              c += w[i];
              k += c <= thr;
            }
            token = __shfl_sync(kAll, v0 + k, __ffs(static_cast<int>(hit)) - 1);
            if (lane == 0) p.tokens[n] = token;
            break;
          }
          cum += __shfl_sync(kAll, incl, 31);
        }
      }
    }
  }
  if ((bad || greedy) && p.tokens != nullptr && part == 0 && threadIdx.x == 0) p.tokens[n] = token;
  // ---------------------------------------------------------------- distribution
  if (probs != nullptr) {
    const float inv = total > 0ull ? 1.f / __ull2float_rn(total) : 0.f;
    float* out = probs - shift;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
      const int at = first + r * 32 + lane, v0 = at * VEC - shift;
      float x[VEC], y[VEC];
      P::get(mine[r * 32 + lane], x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const bool in = keep.keeps(x[i], v0 + i);
        y[i] = 0.f;
        if (__any_sync(kAll, in)) {
          const u64 w = weigh(x[i]);
          if (in) y[i] = __ull2float_rn(w) * inv;
        }
      }
      if (aligned && v0 >= 0 && v0 + VEC <= V) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
          __stcs(reinterpret_cast<float4*>(out + at * VEC + i), make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (v0 + i >= 0 && v0 + i < V) probs[v0 + i] = y[i];
      }
    }
  }
  settle();   // no peer reads this CTA's memory any more
}

template <typename TT>
cudaError_t launch_typed(const DrawArgs& a, cudaStream_t s, bool pdl) {
  constexpr int kMaxSmem = 200 * 1024;
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!done[dev & 63]) {
    cudaError_t e = cudaFuncSetAttribute(sample_logits_kernel<TT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_logits_kernel<TT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    done[dev & 63] = true;
  }
  constexpr int VEC = Pack<TT>::N;
  const int pieces = (a.V + 2 * VEC - 2) / VEC;          // whatever the row's alignment
  auto rows_of = [&](int parts) { return (pieces + parts * kThreads - 1) / (parts * kThreads); };
  // CTAs a row: as many as leave two of them room in an SM's shared memory (ten rows of
  // 16-byte pieces a warp, 80 KB), and more while they leave SMs idle and have two rows each.
  int parts = 1;
  while (parts < kMaxParts && rows_of(parts) > 10) parts *= 2;
  while (parts < kMaxParts && 2LL * parts * a.N <= 2LL * num_sms_of_current_device() && rows_of(parts) > 2) parts *= 2;
  const int rows = rows_of(parts);
  const size_t smem = static_cast<size_t>(rows) * kWarps * 32 * 16 + kHistInts * sizeof(unsigned);
  if (smem > kMaxSmem) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.N) * parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_logits_kernel<TT>, a, parts, rows);
}

}  // namespace

cudaError_t launch_sample_logits(const DrawArgs& a, cudaStream_t s, bool pdl) {
  return a.bf16 ? launch_typed<__nv_bfloat16>(a, s, pdl) : launch_typed<float>(a, s, pdl);
}

}  // namespace dfl
