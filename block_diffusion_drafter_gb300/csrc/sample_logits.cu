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
// summation: weights are integers W = floor(w 2^43), computed to 2^-30 of
// themselves (2^-27.6 at most) by a function of (x, max, T) alone, and every sum of
// them is exact. At V entries of random weights the drawn token differs from that of
// exact weights with a probability of about sqrt(V) 2^-30 (the errors add at random
// along the prefix), 4e-7 for 151936 entries; fp32 weights would give 1e-3 from the
// exponent's rounding alone.
//
// A row belongs to a cluster of one to 16 CTAs, each warp takes a contiguous part. The
// first pass reads it from HBM; what follows reads it again from shared memory, where
// that holds it (few rows), or from L2. What a row asks for decides how much follows,
// always the same for all CTAs of a cluster:
//   the largest entry (temperature 0, top-k 1): one exchange of the CTAs' maxima;
//   top-k up to kMostListed, and top-p: a lower bound of the border from the maxima of
//     the threads' entries, which leaves some k, or some tens or hundreds, of candidates.
//     The first CTA orders these and finds border and token by itself. What top-p takes a
//     part of, the weight of all, is summed in fp32 with a bound of the error;
//   neither: the weights' sums a warp, and the warp that holds the threshold;
//   where the candidates do not fit the list or do not hold the border (flat rows, many
//     equal entries, a large k): histograms over the values, counts for top-k, weights for
//     top-p, added over the cluster through distributed shared memory, the border's bin
//     put in order, or taken apart further until it holds one entry or one value.
// Rows of 151936 entries, the bytes at a copy's rate and the time in us: 1 row bf16, top-k 20 and
// top-p 0.95, 0.05 / 12.9 (latency: four exchanges of 1.5 us between CTAs and the order of
// 40 candidates); 64 rows f32 5.8 / 20.9; 272 rows f32 24.7 / 63.9; 1024 rows bf16 46.6 / 126,
// the largest entry alone 64; top-p 0.95 alone, temperature 0.7, 293, one row in twenty
// flat and weighed twice; neither 223 (the weights: 16 cycles per 32 entries and SM quarter
// where nothing else runs).
#include <cuda_bf16.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace dfl {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxParts = 16;
constexpr int kCountBins = 2048, kMassBins = 1024;
constexpr int kHistInts = 3 * kMassBins;   // of weights: counts, lower and upper words
constexpr int kList = 2048;          // candidates of a CTA, and of a row: 32 KB
// top-k borders that the list is made for; larger ones by histograms. (Temperature 1, list
// against histograms, us, without / with top-p 0.95. k = 900: 1 row bf16 34.2 / 31.3 against
// 33.2 / 56.5, 64 rows f32 59 / 57 and 61 / 102, 272 f32 140 / 134 and 186 / 323, 1024 bf16
// 273 / 260 and 555 / 1366. k = 1270: 39.6 / 32.1 and 33.4 / 56.5, 68 / 60 and 63 / 108,
// 159 / 140 and 195 / 346, 315 / 328 and 581 / 1427. k = 1500, where the list begins to
// overflow: 40 / 43 and 34 / 57, 72 / 120 and 61 / 111, 187 / 230 and 201 / 359, 399 / 455
// and 593 / 1432.)
constexpr int kMostListed = 1280;
// Candidates among which top-p's border is looked for, and then. (1280 instead of 640: 16
// / 64 rows bf16 at temperature 0.7 46 / 60 instead of 35 / 52 us, 1024 rows 315 instead of
// 293; 272 rows f32, where one row's border decides, 143 instead of 161.)
constexpr int kHoped = 64, kHopedMost = 640;
// Candidates whose ranks are counted, all with all; more are sorted. (Up to 512: 300 rows
// with top-k 400 89 instead of 58 us.)
constexpr int kCounted = 192;
constexpr int kScratchBytes = 2 * kList * 8;   // the lists, or the histograms
constexpr int kInFlight = 5;         // 16-byte loads a thread, first pass
constexpr int kAgain = 2;            // and later ones (4: 1024 rows weighed whole 281 instead of 265 us, registers)
constexpr int kOne = 43;             // the largest weight is 2^43
typedef unsigned long long u64;
constexpr unsigned kAll = 0xffffffffu;

// 2^(j/32), j = 0 .. 31 (from the exponential's definition): the largest float not
// above it, and the relative rest.
__device__ const float kPow2[32][2] = {
    {1.0f, 0.0f}, {1.0218970775604248f, 6.957030507237505e-08f}, {1.0442737340927124f, 4.6285471455576044e-08f}, {1.0671403408050537f, 5.610487008311793e-08f},
    {1.0905076265335083f, 9.732325167988165e-08f}, {1.1143866777420044f, 5.819693527087111e-08f}, {1.1387885808944702f, 4.7297824323777604e-08f}, {1.1637247800827026f, 6.762326876241787e-08f},
    {1.1892070770263672f, 3.1934181521364735e-08f}, {1.2152472734451294f, 7.120800660231907e-08f}, {1.2418577671051025f, 3.621057231839586e-08f}, {1.2690509557724f, 1.1184210224612912e-09f},
    {1.2968394756317139f, 6.093220861203008e-08f}, {1.3252365589141846f, 6.357020509994982e-08f}, {1.3542554378509521f, 8.055049249833246e-08f}, {1.383909821510315f, 4.368313355485043e-08f},
    {1.4142135381698608f, 1.7114270889351246e-08f}, {1.4451807737350464f, 2.300196655369291e-08f}, {1.4768260717391968f, 5.024308791234944e-08f}, {1.5091643333435059f, 6.245172556873513e-08f},
    {1.5422108173370361f, 5.233334210430485e-09f}, {1.57598078250885f, 3.9720685407473866e-08f}, {1.610490322113037f, 6.10759176566944e-09f}, {1.645755410194397f, 4.129384478801512e-08f},
    {1.6817927360534668f, 5.616266562924466e-08f}, {1.7186192274093628f, 4.114530582910447e-08f}, {1.7562520503997803f, 6.261829810227937e-08f}, {1.7947089672088623f, 6.006224140264749e-08f},
    {1.834007978439331f, 5.887106979685086e-08f}, {1.874167561531067f, 3.872611742394838e-08f}, {1.9152065515518188f, 5.140609271592211e-09f}, {1.957144021987915f, 5.221255250376089e-08f}};

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
__device__ __forceinline__ void st_peer_u64(const void* p, int rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void st_peer_u32(const void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "r"(v) : "memory");
}

__device__ __forceinline__ float largest4(const float* x) { return fmaxf(fmaxf(fmaxf(x[0], x[1]), x[2]), x[3]); }

// The least whole number of which at least p of `all` lies before: ceil(p * all), 1 or more.
__device__ __forceinline__ u64 draw_ceil(float p, u64 all) {
  bool whole;
  const u64 t = draw_threshold(fmaxf(p, 0.f), all, whole);
  return t + (whole && t > 0ull ? 0ull : 1ull);
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

__device__ __forceinline__ u64 pair2(float lo, float hi) {
  u64 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float lo_of(u64 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(u64 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
#define DFL_F32X2(name, op)                                                   \
  __device__ __forceinline__ u64 name(u64 a, u64 b) {                         \
    u64 d;                                                                    \
    asm(op ".f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));                  \
    return d;                                                                 \
  }
#define DFL_F32X2_FMA(name, op)                                               \
  __device__ __forceinline__ u64 name(u64 a, u64 b, u64 c) {                  \
    u64 d;                                                                    \
    asm(op ".f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));      \
    return d;                                                                 \
  }
DFL_F32X2(add2, "add.rn")
DFL_F32X2(add2_cut, "add.rz")
DFL_F32X2(mul2, "mul.rn")
DFL_F32X2_FMA(fma2, "fma.rn")
DFL_F32X2_FMA(fma2_down, "fma.rm")
DFL_F32X2_FMA(fma2_cut, "fma.rz")
__device__ __forceinline__ u64 both(float x) { return pair2(x, x); }

// The weight's function: 2^43 exp((x - m) / T), up to a factor near 1 that a row's
// weights share and that changes no ratio: m log2(e) / T is rounded down to 32nds
// (so that no weight is below its value), and r below is raised by 2^-8.
// c = log2(e) / T in two floats; z = x c - M with M that rounded maximum; 32 z's
// floor i comes from one multiply-add rounded down onto 1.5 2^23 (without c's low
// part: 1.23 2^-24 of x c, 0.0024 at most, which 2^-8 covers, so that r stays
// positive); r = z - i / 32 + 2^-8 < 0.038 is one exact sum rounded once, and the low
// part added: off by 2^-29 at most.
// 2^z = 2^(i >> 5) 2^((i & 31) / 32) 2^r: the second factor from a table whose entries
// the lanes hold (a shuffle looks it up: no bank conflicts, where shared memory has
// three lanes a bank), as a float and a relative rest; the third 1 + q by the
// exponential's series to r^4 (r^5: 2^-33). So w = h + l, h the table's float times a
// power of two (exact), l = h (q + rest), rounded. As an integer: adding 2 to h and l
// under rounding towards zero leaves their multiples of 2^-22 in the sums' bits; what
// is cut off of both, added, likewise gives the multiple of 2^-43.
// Entries below `low` have no weight and are raised to it; where |m c| is 32768 or more,
// every entry with a weight lies within a factor of two of m: x - m is then exact and
// takes x's place (base). (Below that |x c| < 32768 + 47, so that multiples of 2^-8 like
// M - i / 32 are floats; from 65536 on they are not.) Two entries at once, nearly all of it
// on the multiply-add pipe (16 cycles an entry and SM quarter, bound by that pipe and
// the shuffles; integer shifts, selects and conversions take 2 to 8 cycles each, and a
// sum of 64-bit shifted integers took 1024 rows of bf16 from 265 to 315 us).
struct Weigh {
  u64 ch32, ch, cl, neg_base, neg_max, start;
  float low;
  float hi, lo;              // this lane's table entry
  static constexpr float kMagic = 12582912.f;         // 1.5 2^23, bits 0x4B400000
  static constexpr unsigned kTwo = 0x40000000u;       // 2.0
  // Temperatures outside 2^-100 .. 2^100 count as these (c's low part would lose bits); an
  // infinite one is its own.
  static __device__ __forceinline__ float inside(float T) { return isinf(T) ? T : fminf(fmaxf(T, 0x1p-100f), 0x1p100f); }
  // c in two floats, T inside. T infinite: 0, so that all weights are equal (then `low` is
  // -inf and -inf times c NaN: entries of -inf have to be left out by the caller).
  static __device__ __forceinline__ float2 factor(float T) {
    if (isinf(T)) return make_float2(0.f, 0.f);
    constexpr float kLh = 1.44269502162933349609375f, kLl = 1.92596303350e-8f;   // log2(e)
    const float c = __fdiv_rn(kLh, T);
    return make_float2(c, __fdiv_rn(__fmaf_rn(-c, T, kLh) + kLl, T));
  }
  __device__ __forceinline__ void set(float m, float2 f, int lane) {
    float c = f.x, d = f.y;
    // so small a temperature that the float below m has no weight: no smaller one is needed
    const float most = 46.f * 0x1p24f / fabsf(m);   // 46 and more for the float below m
    if (c > most) {
      c = most;
      d = 0.f;
    }
    low = __fsub_rd(m, 46.f / c);
    const float base = fabsf(m) * c < 32768.f ? 0.f : m;
    const float top = floorf((m - base) * c * 32.f) * 0.03125f;
    ch32 = both(32.f * c);
    ch = both(c);
    cl = both(d);
    neg_base = both(-base);
    neg_max = both(0x1p-8f - top);
    start = both(kMagic - 32.f * top);
    hi = kPow2[lane][0];
    lo = kPow2[lane][1];
  }
  // The bits of 2 + h, 2 + l and 2 + 2^21 (what they cut off), cut, of two entries,
  // neither above m. Called by a whole warp.
  struct Bits {
    u64 h, l, r;
  };
  __device__ __forceinline__ Bits bits(float x0, float x1) const {
    const u64 x = add2(pair2(fmaxf(x0, low), fmaxf(x1, low)), neg_base);
    const u64 t = fma2_down(x, ch32, start);
    const u64 f = add2(t, both(-kMagic));
    const u64 e = fma2(f, both(-0.03125f), neg_max);                      // exact
    const u64 r = fma2(x, cl, fma2(x, ch, e));
    u64 q = fma2(r, both(9.61812911e-3f), both(5.55041087e-2f));
    q = fma2(r, q, both(0.240226507f));
    q = fma2(r, q, both(0.693147181f));
    const uint32_t i0 = __float_as_uint(lo_of(t)), i1 = __float_as_uint(hi_of(t));   // 0x4B400000 + floor(32 z)
    // the lane is taken modulo 32; the exponent's field grows by i >> 5
    const u64 rest = pair2(__shfl_sync(kAll, lo, i0), __shfl_sync(kAll, lo, i1));
    const float a = __shfl_sync(kAll, hi, i0), b = __shfl_sync(kAll, hi, i1);
    const u64 h = pair2(__uint_as_float(((i0 - 0x4B400000u) >> 5) * 0x800000u + __float_as_uint(a)),
                        __uint_as_float(((i1 - 0x4B400000u) >> 5) * 0x800000u + __float_as_uint(b)));
    const u64 l = mul2(h, fma2(r, q, rest));
    Bits v;
    v.h = add2_cut(h, both(2.f));
    v.l = add2_cut(l, both(2.f));
    // h - (v.h - 2) and l - (v.l - 2), both exact
    const u64 left = add2(add2(h, fma2(v.h, both(-1.f), both(2.f))), add2(l, fma2(v.l, both(-1.f), both(2.f))));
    v.r = fma2_cut(left, both(0x1p21f), both(2.f));
    return v;
  }
  // One entry's weight.
  static __device__ __forceinline__ u64 whole(uint32_t h, uint32_t l, uint32_t r) {
    return (static_cast<u64>(h + l - 2u * kTwo) << 21) + (r - kTwo);
  }
  __device__ __forceinline__ void two(float x0, float x1, u64& w0, u64& w1) const {
    const Bits v = bits(x0, x1);
    w0 = whole(static_cast<uint32_t>(v.h), static_cast<uint32_t>(v.l), static_cast<uint32_t>(v.r));
    w1 = whole(static_cast<uint32_t>(v.h >> 32), static_cast<uint32_t>(v.l >> 32), static_cast<uint32_t>(v.r >> 32));
  }
  // The weights' sum of four entries.
  __device__ __forceinline__ void add4(const float* x, u64& high, u64& rest) const {
    const Bits a = bits(x[0], x[1]), b = bits(x[2], x[3]);
    auto sum = [](u64 p) { return static_cast<uint32_t>(p) + static_cast<uint32_t>(p >> 32); };
    high += sum(a.h) + sum(b.h) + sum(a.l) + sum(b.l);      // 8 kTwo = 0 in 32 bits
    rest += sum(a.r) + sum(b.r);                            // 4 kTwo = 0
  }
  // The sum of four weights in fp32, for rows with |m c| below kNear. Each is off by the
  // rounding of an exponent below 32 (2^-20; what lies beyond weighs V 2^-32 at most) and
  // by c's low part, 1.2235 (|m c| + 32) 2^-24 (half a step of a float just above a power of
  // two, and log2(e)'s own rounding), both times ln 2, by 2^-22 (the exponential) and two
  // roundings of the sum: (0.8481 |m c| + 44.3) 2^-24 of itself. (With the row's own low
  // part instead of 1.2235 fewer rows are weighed twice, yet by its registers top-k 20
  // with top-p is 3 % slower and top-p alone no faster.)
  static constexpr float kNear = 1024.f;
  __device__ __forceinline__ float near4(const float* x) const {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const u64 z = fma2(pair2(x[i], x[i + 1]), ch, neg_max);
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(lo_of(z)));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i + 1]) : "f"(hi_of(z)));
    }
    return (e[0] + e[1]) + (e[2] + e[3]);
  }
  __device__ __forceinline__ float scale() const { return lo_of(ch); }   // log2(e) / T
  __device__ __forceinline__ u64 operator()(float x) const {
    u64 a, b;
    two(x, x, a, b);
    return a;
  }
};

// Whether p of a row's weight lies in more than kHopedMost entries, as a power law
// through the weights of the 1st, the kHoped-th and the kHopedMost-th has it (such rows
// go to the histograms at once). A guess: either way gives the same result.
__device__ __forceinline__ bool looks_flat(float m, float upo, float flo, float c, float p, int V) {
  constexpr float kLogHoped = 6.f, kLogMost = 3.321928f;     // log2 of kHoped, of kHopedMost / kHoped
  static_assert(kHoped == 64 && kHopedMost == 640, "their logarithms");
  const float y1 = fminf((m - upo) * c, 60.f), y2 = fminf((upo - flo) * c, 60.f);
  // the sum of r^-s from r = 1 to 2^l, as an integral
  auto area = [](float s, float l) {
    const float d = (1.f - s) * l;
    return fabsf(d) < 0.01f ? 0.693147f * l : (exp2f(d) - 1.f) / (1.f - s);
  };
  const float s1 = y1 / kLogHoped, s2 = y2 / kLogMost;
  const float w1 = exp2f(-y1) * kHoped, w2 = w1 * exp2f(-y2) * (static_cast<float>(kHopedMost) / kHoped);
  const float top = 1.f + area(s1, kLogHoped) + w1 * area(s2, kLogMost);
  const float tail = V > kHopedMost ? w2 * area(s2, log2f(static_cast<float>(V) / kHopedMost)) : 0.f;
  return top < p * (top + tail);
}

// What stays: entries above `thr`, and of those equal to it the ones up to index `cut`.
struct __align__(8) Border {
  float thr;
  int cut;                   // 8 bytes: sent as one word
  __device__ __forceinline__ bool keeps(float x, int v) const { return x > thr || (x == thr && v <= cut); }
};

// What a CTA tells its peers: its largest entry (its key and the complement of its
// index) and two starts of keys that so many of its threads' maxima reach; then the
// weight of its entries and of those that it lists, and their number.
struct Told {
  u64 top;
  u64 floors;
  u64 sum, listed, count;
};

struct Shared {
  Told told;
  u64 warp[2][kWarps];             // warps' sums, and the CTA's: two joins in turn
  u64 part[2];
  u64 scan[kWarps];
  u64 above;
  float warp_f[kWarps];
  unsigned bin, count;
  int tie, at, len;
  unsigned certain, sure;          // whether the border is, in the first CTA, and told to all
  Border border;                   // what the first CTA found
  u64 total;
  float2 min_log;                  // T ln(min_p), in two floats
};

// Two CTAs an SM leave 64 registers a thread, and all ways share them: the stack frame is 40
// bytes for f32 (112 bytes of spill stores, 140 of loads over the whole kernel), 56 for bf16
// (310, 424). What keeps more values alive pays here first.
template <typename TT>
__global__ void __launch_bounds__(kThreads, 2) sample_logits_kernel(const DrawArgs p, const int parts, const int rows) {
  using P = Pack<TT>;
  constexpr int VEC = P::N;
  extern __shared__ __align__(16) uint4 s_data[];          // [kWarps][rows][32]
  __shared__ Shared sh;
  unsigned* hist = reinterpret_cast<unsigned*>(s_data + kWarps * rows * 32);   // or: own list, all lists
  u64* own = reinterpret_cast<u64*>(hist);
  u64* list = own + kList;
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
  // this warp's rows of 32 pieces, an even share of all, and its first piece
  const int all_rows = (pieces + 31) / 32, id = part * kWarps + warp, warps = parts * kWarps;
  const int row0 = static_cast<int>(static_cast<unsigned>(all_rows) * id / warps);
  const int my_rows = static_cast<int>(static_cast<unsigned>(all_rows) * (id + 1) / warps) - row0, first = row0 * 32;
  // Held in shared memory (rows > 0), or read again from L2.
  const bool held = rows > 0;
  uint4* mine = s_data + warp * rows * 32;
  // Piece `at` of the row: what is not the row's and NaN become -inf, +inf the largest number.
  bool odd_row = false;   // whether any of this thread's entries was NaN or +inf
  auto clean = [&](uint4 q, int at, bool look) -> uint4 {
    float x[VEC];
    P::get(q, x);
    bool odd = at * VEC < shift || (at + 1) * VEC > shift + V;   // also pieces behind the row
    if (look) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < VEC; ++i) bad = bad || !(x[i] <= FLT_MAX);   // NaN or +inf
      odd_row = odd_row || bad;
      odd = odd || bad;
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int v = at * VEC + i - shift;
        if (v < 0 || v >= V || x[i] != x[i]) x[i] = -INFINITY;
        x[i] = fminf(x[i], P::largest());
      }
      q = P::put(x);
    }
    return q;
  };
  float thread_top = -INFINITY;
  int top_at = 0;      // the piece that holds it
  for (int r0 = 0; r0 < my_rows; r0 += kInFlight) {
    uint4 q[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int at = first + (r0 + k) * 32 + lane;
      q[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + k < my_rows && at < pieces) q[k] = held ? __ldcs(base + at) : __ldg(base + at);
    }
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (r0 + k >= my_rows) break;
      const int at = first + (r0 + k) * 32 + lane;
      q[k] = clean(q[k], at, true);
      float x[VEC], top;
      P::get(q[k], x);
      top = x[0];
#pragma unroll
      for (int i = 1; i < VEC; ++i) top = fmaxf(top, x[i]);
      if (top > thread_top) {
        thread_top = top;
        top_at = at;
      }
      if (held) mine[(r0 + k) * 32 + lane] = q[k];
    }
  }
  // Row r of this warp's pieces, this lane's, as values.
  auto piece = [&](int r, float* x) {
    const int at = first + r * 32 + lane;
    if (held) {
      P::get(mine[r * 32 + lane], x);
    } else {
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (at < pieces) q = __ldg(base + at);
      P::get(clean(q, at, odd_row), x);
    }
  };
  const float T_in = p.temperature != nullptr ? p.temperature[n] : 1.f;
  const int k_in = p.top_k != nullptr ? p.top_k[n] : 0;
  const float p_in = p.top_p != nullptr ? p.top_p[n] : 1.f;
  const float min_p = p.min_p != nullptr ? p.min_p[n] : 0.f;
  const bool has_min = min_p > 0.f, has_k = k_in > 0 && k_in < V, has_p = p_in < 1.f;
  const bool greedy = T_in == 0.f || k_in == 1;
  const float T = Weigh::inside(greedy ? 1.f : T_in);
  const float2 c_log2e = Weigh::factor(T);
  // entries that are listed, at least: k, or as many as top-p's border is hoped among
  const int want = greedy ? 0 : has_k ? (k_in <= kMostListed ? k_in : 0) : has_p ? kHopedMost : 0;
  if (has_min && threadIdx.x == 0) {
    const double d = static_cast<double>(T) * log(static_cast<double>(fminf(min_p, 1.f)));
    const float a = static_cast<float>(d);
    sh.min_log = make_float2(a, static_cast<float>(d - static_cast<double>(a)));
  }

  // f(values, index of the first) of this warp's entries, four neighbours a lane, all
  // lanes together. From L2 the last row first: it was read last.
  auto each = [&](auto f) {
    if (held) {
#pragma unroll 1
      for (int r = 0; r < my_rows; ++r) {
        float x[VEC];
        P::get(mine[r * 32 + lane], x);
#pragma unroll
        for (int i = 0; i < VEC; i += 4) f(x + i, (first + r * 32 + lane) * VEC - shift + i);
      }
      return;
    }
    auto ask = [&](int r) {
      const int at = first + r * 32 + lane;
      return r >= 0 && at < pieces ? __ldg(base + at) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 q[kAgain];
#pragma unroll
    for (int k = 0; k < kAgain; ++k) q[k] = ask(my_rows - 1 - k);
#pragma unroll 1
    for (int r0 = my_rows - 1; r0 >= 0; r0 -= kAgain) {
#pragma unroll
      for (int k = 0; k < kAgain; ++k) {
        const int r = r0 - k;
        if (r < 0) break;
        float x[VEC];
        P::get(clean(q[k], first + r * 32 + lane, odd_row), x);
        q[k] = ask(r - kAgain);
#pragma unroll
        for (int i = 0; i < VEC; i += 4) f(x + i, (first + r * 32 + lane) * VEC - shift + i);
      }
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
    if (parts == 1) return;
    cluster_arrive();
    pending = true;
  };
  auto meet = [&]() {
    settle();
    if (parts == 1) __syncthreads(); else cluster_sync();
  };

  // ---------------------------------------------------------------- maximum
  {
    float top = thread_top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    if (lane == 0) sh.warp_f[warp] = top;
    if (threadIdx.x == 0) {
      sh.at = INT32_MAX;
      sh.told.count = 0ull;
    }
    __syncthreads();
    top = sh.warp_f[lane % kWarps];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    // the first entry that equals it, in the first piece of one of few threads
    if (thread_top == top && top > -INFINITY) {
      float x[VEC];
      piece((top_at - first) / 32, x);
      int at = INT32_MAX;
#pragma unroll
      for (int i = VEC - 1; i >= 0; --i) at = x[i] == top ? top_at * VEC - shift + i : at;
      atomicMin(&sh.at, at);
    }
    // The largest 16-bit start of a key that `share` threads' maxima reach: every CTA
    // has so many entries from its own on, so together they have `want` from the least
    // of them on, and few more. Where that takes more than a quarter of the threads,
    // several of the wanted entries share a thread: of T threads T (1 - exp(-w / T)) hold
    // one or more of w entries in no order. That many maxima, for a few entries more
    // than are wanted; what the list then holds is looked at.
    const uint32_t key = key_of(thread_top) >> 16;
    auto start = [&](int of) -> uint32_t {
      int share = (of + parts - 1) / parts;
      if (4 * share > kThreads) {
        const float w = 1.1f * static_cast<float>(share) + 4.f * sqrtf(static_cast<float>(share));
        share = static_cast<int>(kThreads * (1.f - expf(w * (-1.f / kThreads))));
      }
      uint32_t floor = 0u;
#pragma unroll 1
      for (uint32_t bit = 1u << 15; bit > 0u; bit >>= 1)
        if (__syncthreads_count(key >= (floor | bit)) >= share) floor |= bit;
      return floor;
    };
    uint32_t floor = 0u, upper = 0u;
    if (want > 0) {
      floor = start(want);
      upper = has_k ? floor : start(kHoped);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      sh.told.top = static_cast<u64>(key_of(top)) << 32 | (kAll - static_cast<uint32_t>(sh.at));
      sh.told.floors = static_cast<u64>(floor) << 32 | upper;
    }
  }
  meet();
  float m, flo, upo;       // the maximum, and the two starts
  int first_top;
  {
    u64 a = ld_peer_u64(&sh.told.top, lane % parts), b = ld_peer_u64(&sh.told.floors, lane % parts);   // parts divides 32
    uint32_t lower = static_cast<uint32_t>(b >> 32), upper = static_cast<uint32_t>(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 c = __shfl_xor_sync(kAll, a, o);
      a = c > a ? c : a;
    }
    lower = __reduce_min_sync(kAll, lower);
    upper = __reduce_min_sync(kAll, upper);
    m = value_of(static_cast<uint32_t>(a >> 32));
    first_top = static_cast<int>(kAll - static_cast<uint32_t>(a));
    flo = value_of(max(lower << 16, key_of(-FLT_MAX)));
    upo = value_of(max(upper << 16, key_of(-FLT_MAX)));
  }
  const bool bad = m == -INFINITY || !(T_in >= 0.f);
  float* probs = p.probs != nullptr ? p.probs + static_cast<size_t>(n) * V : nullptr;
  Border keep{-FLT_MAX, INT32_MAX};
  Weigh weigh;
  weigh.set(m, c_log2e, lane);
  u64 total = 0ull;
  // min-p: the least float that is not below m + T ln(min_p). That is finite or, where T
  // is infinite (all weights are 1) or the sum passes the lowest number, keeps all.
  float least = -FLT_MAX;
  if (has_min && !isinf(T)) {
    const float a = sh.min_log.x, t = __fadd_rn(m, a), b = __fsub_rn(t, m);   // t + e = m + a
    const float e = __fadd_rn(__fsub_rn(m, __fsub_rn(t, b)), __fsub_rn(a, b));
    if (t >= -FLT_MAX) least = fminf(__fadd_ru(t, __fadd_rn(e, sh.min_log.y)), m);
  }

  // A sum over the cluster of one value a warp: what lies before this warp, and all.
  int turn = 0;
  auto join = [&](u64 v, u64& before, u64& all) {
    turn ^= 1;
    if (lane == 0) sh.warp[turn][warp] = v;
    __syncthreads();
    const u64 w = lane < kWarps ? sh.warp[turn][lane] : 0ull;
    const u64 sum = warp_sum(w);
    if (threadIdx.x == 0) sh.part[turn] = sum;
    meet();
    const u64 t = lane < parts ? ld_peer_u64(&sh.part[turn], lane) : 0ull;
    all = warp_sum(t);
    before = warp_sum((lane < part ? t : 0ull) + (lane < warp ? w : 0ull));
    left();
  };
  // Inclusive sum over the CTA's threads.
  auto block_scan = [&](u64 v, u64& all) -> u64 {
    const u64 incl = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    const u64 w = lane < kWarps ? sh.scan[lane] : 0ull;
    all = warp_sum(w);
    return incl + warp_sum(lane < warp ? w : 0ull);
  };

  // Sum over the CTA's threads.
  auto block_sum = [&](u64 v, u64& all) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.scan[warp] = v;
    __syncthreads();
    all = warp_sum(lane < kWarps ? sh.scan[lane] : 0ull);
  };

  // The first CTA's joint list of all CTAs' lists; c: entries of this lane's CTA.
  auto pull = [&](unsigned c) {
    const unsigned incl = static_cast<unsigned>(warp_scan(c, lane)), len = __shfl_sync(kAll, incl, 31);
    for (unsigned i0 = warp * 32; i0 < len; i0 += kThreads) {
      const unsigned i = i0 + lane;
      unsigned of = 0u, before = 0u;
      for (int r = 0; r < parts; ++r) {
        const unsigned e = __shfl_sync(kAll, incl, r);
        if (i >= e) {
          of = r + 1;
          before = e;
        }
      }
      if (i < len) list[i] = ld_peer_u64(own + (i - before), of);
    }
    if (threadIdx.x == 0) sh.len = len;
  };
  // The border among the joint list's entries: of the first `most` in order those with
  // less than `need` before them (of_most: need is top-p's part of their weight) and not
  // below `lowest`, the first one always: sh.border, their weight sh.total, and the token
  // drawn from them, if no entry has between `need` and `need_most` before it (sh.certain).
  // The first CTA alone.
  auto order = [&](int most, bool of_most, u64 need, u64 need_most, float lowest, bool draw) {
    const int len = sh.len;
    u64 all;
    int stay = 0;
    if (len <= kCounted) {
      // Ranks and the weight before an entry by comparing all with all: a group of
      // threads an entry, no order is made.
      int group = 1;
      while (2 * group * len <= kThreads && group < 32) group *= 2;
      const int i = threadIdx.x / group, s0 = threadIdx.x % group;
      const bool mine_is = i < len;
      const u64 key = mine_is ? list[i] : ~0ull;
      const float x = mine_is ? value_of(~static_cast<uint32_t>(key >> 32)) : -INFINITY;
      const u64 w = weigh(x);
      if (mine_is && s0 == 0) own[i] = w;
      __syncthreads();
      int rank = 0;
      u64 before = 0ull;
#pragma unroll 4
      for (int j = s0; j < len; j += group) {
        const bool less = list[j] < key;
        rank += less;
        before += less ? own[j] : 0ull;
      }
      for (int o = group / 2; o > 0; o /= 2) {
        rank += __shfl_xor_sync(kAll, rank, o);
        before += __shfl_xor_sync(kAll, before, o);
      }
      const bool first_of = mine_is && s0 == 0;
      if (of_most) {
        block_sum(first_of && rank < most ? w : 0ull, all);
        need = need_most = draw_ceil(p_in, all);
      }
      const bool kept = first_of && rank < most && (rank == 0 || (before < need && x >= lowest));
      const bool open = first_of && rank > 0 && rank < most && before >= need && before < need_most && x >= lowest;
      const bool sure = __syncthreads_count(open) == 0;
      if (threadIdx.x == 0) sh.certain = sure;
      block_sum(kept ? w : 0ull, total);
      stay = __syncthreads_count(kept);
      if (first_of) own[i] = kept ? w : 0ull;
      if (kept && rank == stay - 1) {
        sh.border = Border{x, static_cast<int>(static_cast<uint32_t>(key))};
        sh.total = total;
      }
      if (threadIdx.x == 0) sh.at = INT32_MAX;
      __syncthreads();
      if (draw && sure) {
        bool whole;
        const u64 thr = draw_threshold(p.u[n], total, whole);
        const uint32_t index = static_cast<uint32_t>(key);
        u64 upto = 0ull;
#pragma unroll 4
        for (int j = s0; j < len; j += group) upto += static_cast<uint32_t>(list[j]) <= index ? own[j] : 0ull;
        for (int o = group / 2; o > 0; o /= 2) upto += __shfl_xor_sync(kAll, upto, o);
        if (kept && upto > thr) atomicMin(&sh.at, static_cast<int>(index));
        __syncthreads();
        if (threadIdx.x == 0) p.tokens[n] = sh.at;
      }
    } else {
      auto sort = [&](auto* v, int len) {   // ascending; what is behind len is larger than all
        int size = 32;
        while (size < len) size *= 2;
        __syncthreads();
        for (int k = 2; k <= size; k *= 2)
          for (int j = k / 2; j > 0; j /= 2) {
            for (int i = threadIdx.x; i < size / 2; i += kThreads) {
              const int a = 2 * i - (i & (j - 1)), b = a + j;
              const auto x = v[a], y = v[b];
              if ((x > y) == ((a & k) == 0)) {
                v[a] = y;
                v[b] = x;
              }
            }
            // up to a distance of 32 a warp stays within its 64 entries
            if (j > 32 || (j == 1 && k > 32)) __syncthreads(); else __syncwarp();
          }
        __syncthreads();
      };
      for (int i = len + threadIdx.x; i < kList; i += kThreads) list[i] = ~0ull;
      sort(list, len);
      // a thread's entries: PER neighbouring ones
      constexpr int PER = kList / kThreads;
      static_assert(PER == 4, "the draw picks one of four");
      const int kept = min(most, len), at0 = PER * threadIdx.x;
      u64 w[PER], mass = 0ull;
      float x[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] = at0 + i < kept ? value_of(~static_cast<uint32_t>(list[at0 + i] >> 32)) : -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; i += 2) weigh.two(x[i], x[i + 1], w[i], w[i + 1]);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        w[i] = at0 + i < kept ? w[i] : 0ull;
        mass += w[i];
      }
      u64 incl = block_scan(mass, all);
      if (of_most) need = need_most = draw_ceil(p_in, all);
      // the sorted entries that stay: the first ones
      u64 before = incl - mass;
      bool open = false;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        stay += at0 + i < kept && (at0 + i == 0 || (before < need && x[i] >= lowest));
        open = open || (at0 + i < kept && before >= need && before < need_most && x[i] >= lowest);
        before += w[i];
      }
      const bool sure = __syncthreads_count(open) == 0;
      if (threadIdx.x == 0) sh.certain = sure;
      block_sum(static_cast<u64>(stay), all);
      stay = static_cast<int>(all);
      // their weight, and the entry at the border
      const int last = stay - 1;
      if (static_cast<int>(threadIdx.x) == last / PER) {
        before = incl - mass;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i <= last % PER) before += w[i];
        sh.total = before;
        const u64 e = list[last];
        sh.border = Border{value_of(~static_cast<uint32_t>(e >> 32)), static_cast<int>(static_cast<uint32_t>(e))};
      }
      unsigned places[PER];   // index << 11 | place: kept ones are sorted by their index
      static_assert(kList <= 2048 && kDrawMaxVocab <= 1 << 20, "bits of an index and a place");
#pragma unroll
      for (int i = 0; i < PER; ++i) places[i] = static_cast<uint32_t>(list[at0 + i]) << 11 | (at0 + i);
      __syncthreads();
      total = sh.total;
      if (draw && sure) {
        bool whole;
        const u64 thr = draw_threshold(p.u[n], total, whole);
        unsigned* order = reinterpret_cast<unsigned*>(own);   // 2048 words
        u64* weight = list;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          weight[at0 + i] = w[i];
          order[at0 + i] = at0 + i < stay ? places[i] : kAll;
        }
        sort(order, stay);
        mass = 0ull;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          places[i] = order[at0 + i];
          w[i] = at0 + i < stay ? weight[places[i] & 2047u] : 0ull;
          mass += w[i];
        }
        incl = block_scan(mass, all);
        if (incl > thr && incl - mass <= thr) {   // one thread
          u64 c2 = incl - mass;
          int k = 0;
#pragma unroll
          for (int i = 0; i < PER - 1; ++i) {
            c2 += w[i];
            k += c2 <= thr;
          }
          p.tokens[n] = static_cast<int>((k == 0 ? places[0] : k == 1 ? places[1] : k == 2 ? places[2] : places[3]) >> 11);
        }
      }
    }
  };

  // The border and the weight above it, from the first CTA to all.
  auto send = [&]() {
    if (threadIdx.x < parts) {
      const u64 b = static_cast<u64>(static_cast<uint32_t>(sh.border.cut)) << 32 | __float_as_uint(sh.border.thr);
      st_peer_u64(&sh.border, threadIdx.x, b);
      st_peer_u64(&sh.total, threadIdx.x, sh.total);
    }
  };

  unsigned* own_count = reinterpret_cast<unsigned*>(&sh.told.count);   // of this CTA's list
  if (bad || greedy) {
    if (part == 0 && threadIdx.x == 0) {
      if (bad) report(p.dev_status, DFLASH_ERR_INVALID_ARG);
      if (p.tokens != nullptr) p.tokens[n] = bad ? 0 : first_top;
    }
    left();
    keep = bad ? Border{FLT_MAX, -1} : Border{m, first_top};   // nothing, or the one
    total = weigh(m);
  } else {
    bool found = false;                // the border, through the list
    u64 Z = 1ull << kOne;              // the weight that top-p takes a part of, or less
    // where no float below m is without a weight (the lowest number, an infinite
    // temperature), what has no weight cannot be raised to one
    const bool sums = weigh.low > -INFINITY, listed = want > 0 && sums && !(has_p && !has_k && looks_flat(m, upo, flo, weigh.scale(), p_in, V));
    if (listed) {
      // -------------------------------------------------------------- few candidates
      // Entries from a start on go to the CTA's list, all CTAs' lists to the first one, which
      // orders them and knows everything but the weight of the rest. top-p tries the upper
      // start first: a row's list of kHoped is short to make and to order (all in one list
      // of kHopedMost: 1024 rows bf16 of a power law of exponent 2.1 207 instead of 182 us).
      const bool all_weigh = !has_k;
      const float mc = fabsf(m) * weigh.scale();
      const bool near_by = mc < Weigh::kNear;
      u64 need = ~0ull, need_most = ~0ull, near = 0ull;
      unsigned listed_here = 0u;
#pragma unroll 1
      for (bool upper = all_weigh; ; upper = false) {
        const float from = upper ? upo : flo;
        auto append = [&](const float* x, int v0) {
          if (largest4(x) >= from) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (x[i] >= from) {
                const unsigned at = atomicAdd(own_count, 1u);
                if (at < kList) own[at] = static_cast<u64>(~key_of(x[i])) << 32 | static_cast<uint32_t>(v0 + i);
              }
            }
          }
        };
        if (upper) {
          // The weight of all decides how much of it has to lie before the border. The sum
          // in fp32 and a bound of its error tell the border unless it falls between two
          // entries that so little parts; then all is weighed exactly.
          float sum = 0.f;
          u64 all, high = 0ull, rest = 0ull;
          if (near_by) {
            each([&](const float* x, int v0) {
              sum += weigh.near4(x);
              append(x, v0);
            });
          } else {
            each([&](const float* x, int v0) {
              weigh.add4(x, high, rest);
              append(x, v0);
            });
          }
          block_sum(near_by ? __float2ull_rn(sum * 0x1p43f) : (high << 21) + rest, all);
          if (threadIdx.x == 0) sh.told.sum = all;
        } else {
          each(append);
        }
        __syncthreads();
        if (all_weigh) {
          const int len = min(static_cast<int>(*own_count), kList);
          u64 above = 0ull, all;
#pragma unroll 1
          for (int i0 = warp * 32; i0 < len; i0 += kThreads) {
            const bool in = i0 + lane < len;
            const u64 w = weigh(in ? value_of(~static_cast<uint32_t>(own[i0 + lane] >> 32)) : m);
            above += in ? w : 0ull;
          }
          block_sum(above, all);
          if (threadIdx.x == 0) sh.told.listed = all;
        }
        meet();
        u64 has = 0ull;
        listed_here = 0u;
        if (lane < parts) {   // asked for together
          listed_here = static_cast<unsigned>(ld_peer_u64(&sh.told.count, lane));
          if (all_weigh) {
            near = ld_peer_u64(&sh.told.sum, lane);
            has = ld_peer_u64(&sh.told.listed, lane);
          }
        }
        const unsigned len = __reduce_add_sync(kAll, listed_here);
        found = len <= kList && (!has_k || len >= static_cast<unsigned>(k_in));
        if (all_weigh) {
          near = warp_sum(lane < parts ? near : 0ull);
          // rounded once a group of four, and what the integers cut off
          const float adds = static_cast<float>((all_rows / warps + 1) * (VEC / 4));
          const u64 slack = __float2ull_ru(__ull2float_ru(near) * ((0.86f * mc + adds + 50.f) * 0x1p-24f)) + 2ull * V;
          Z = near_by ? near - min(slack, near) : near;          // at least
          need = draw_ceil(p_in, Z);
          need_most = near_by ? draw_ceil(p_in, near + slack) : need;
          const bool enough = warp_sum(has) >= need_most;
          if (upper && !enough && len <= kList) {   // once more, for more entries
            left();
            settle();
            if (threadIdx.x == 0) sh.told.count = 0ull;
            __syncthreads();
            continue;
          }
          found = found && enough;
        }
        break;
      }
      if (found && part == 0) pull(listed_here);
      left();
      if (found && part == 0) {
        __syncthreads();
        order(has_k ? k_in : kList, has_k && has_p, need, need_most, least, p.tokens != nullptr);
        if (all_weigh && threadIdx.x < parts) st_peer_u32(&sh.sure, threadIdx.x, sh.certain);   // the ordering warp itself
      }
      if (found && all_weigh) {
        meet();   // nobody leaves before the border is sure
        if (sh.sure == 0u) {
          u64 sum = 0ull, low_sum = 0ull, before;
          each([&](const float* x, int) { weigh.add4(x, sum, low_sum); });
          join(warp_sum((sum << 21) + low_sum), before, Z);
          if (part == 0) {
            need = draw_ceil(p_in, Z);
            order(kList, false, need, need, least, p.tokens != nullptr);
          }
        }
      }
      if (found && part == 0 && probs != nullptr) {
        __syncthreads();
        send();
      }
      if (found && probs != nullptr) {
        meet();
        keep = sh.border;
        total = sh.total;
      }
    } else {
      left();
    }
    if (!found) {
      // -------------------------------------------------------------- many candidates
      // The index of the r-th entry (from 1) equal to x, in every CTA.
      auto find_tie = [&](float x, unsigned r) -> int {
        unsigned c = 0;
        each([&](const float* y, int) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c += y[i] == x;
        });
        const u64 all = __reduce_add_sync(kAll, c);
        u64 before, sum;
        join(all, before, sum);
        if (before < r && r <= before + all) {
          unsigned cum = static_cast<unsigned>(before);
          int at = -1;
#pragma unroll 1
          for (int i = 0; i < my_rows && at < 0; ++i) {
            float y[VEC];
            piece(i, y);
            unsigned k = 0;
#pragma unroll
            for (int j = 0; j < VEC; ++j) k += y[j] == x;
            const unsigned incl = static_cast<unsigned>(warp_scan(k, lane));
            const unsigned hit = __ballot_sync(kAll, cum + incl >= r);
            if (hit != 0u) {
              unsigned e = cum + incl - k;
              int is = -1;
#pragma unroll
              for (int j = 0; j < VEC; ++j) {
                e += y[j] == x;
                if (is < 0 && e >= r) is = (first + i * 32 + lane) * VEC - shift + j;
              }
              at = __shfl_sync(kAll, is, __ffs(static_cast<int>(hit)) - 1);
            }
            cum += __shfl_sync(kAll, incl, 31);
          }
          if (lane < parts) st_peer_u32(&sh.tie, lane, static_cast<uint32_t>(at));
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
        for (int r0 = 0; r0 < parts; r0 += 4) {   // four CTAs' bins in flight
          if (!mass) {
            uint4 c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = r0 + k < parts ? ld_peer_v4(hist + b0, r0 + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[0] += c[k].x; v[1] += c[k].y; v[2] += c[k].z; v[3] += c[k].w;
            }
          } else {
            u64 c[4], a0[4], a1[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool in = r0 + k < parts;
              c[k] = in && counted ? ld_peer_u64(hist + b0, r0 + k) : 0ull;
              a0[k] = in ? ld_peer_u64(hist + kMassBins + b0, r0 + k) : 0ull;
              a1[k] = in ? ld_peer_u64(hist + 2 * kMassBins + b0, r0 + k) : 0ull;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              cnt[0] += static_cast<unsigned>(c[k]);
              cnt[1] += static_cast<unsigned>(c[k] >> 32);
              v[0] += (a0[k] & kAll) + (a1[k] << 32);
              v[1] += (a0[k] >> 32) + (a1[k] & 0xffffffff00000000ull);
            }
          }
        }
        left();
        const u64 own_sum = v[0] + v[1] + v[2] + v[3];
        u64 all;
        const u64 incl = block_scan(own_sum, all);
        if (all >= need && incl - own_sum < need && need <= incl) {
          u64 cum = incl - own_sum;
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
        return all >= need;
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
      // The keys of a bin, inside lo .. hi.
      auto narrow = [&](bool linear, float scale, int step, uint32_t& lo, uint32_t& hi) {
        const unsigned bin = sh.bin;
        if (linear) {
          hi = min(hi, key_of(linear_edge(static_cast<int>(bin), scale)));
          lo = max(lo, key_of(linear_edge(static_cast<int>(bin) + 1, scale)) + 1u);
        } else {
          hi -= bin << step;
          lo = max(lo, hi - ((1u << step) - 1u));
        }
      };
      // top-k: levels of counts
      if (has_k) {
        u64 need = static_cast<u64>(k_in);
        uint32_t lo = key_of(-FLT_MAX), hi = key_of(m);
        while (true) {
          const float a = value_of(lo), b = value_of(hi);
          int step = max(0, 32 - __clz(hi - lo) - 11);
          if (step <= P::kFinal) step = P::kFinal;
          clear(kCountBins);
          each([&](const float* x, int) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const unsigned bin = (hi - key_of(x[i])) >> step;
              if (x[i] >= a && x[i] <= b && bin < kCountBins) atomicAdd(&hist[bin], 1u);
            }
          });
          if (!find_bin(false, true, need)) break;        // fewer finite entries than k: all stay
          need -= sh.above;
          const unsigned count = sh.count;
          narrow(false, 0.f, step, lo, hi);
          if (need == count) {
            keep.thr = value_of(lo);
            break;
          }
          if (step == P::kFinal) {                        // one value
            keep.thr = value_of(P::at_or_below(hi));
            keep.cut = find_tie(keep.thr, static_cast<unsigned>(need));
            break;
          }
        }
      }
      // top-p: levels of weights
      if (has_p) {
        const Border from = keep;
        if (has_k) {
          u64 sum = 0ull, before;
          each([&](const float* x, int v0) {
            if (__any_sync(kAll, largest4(x) >= from.thr)) {
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                u64 a, b;
                weigh.two(x[i], x[i + 1], a, b);
                sum += (from.keeps(x[i], v0 + i) ? a : 0ull) + (from.keeps(x[i + 1], v0 + i + 1) ? b : 0ull);
              }
            }
          });
          join(warp_sum(sum), before, Z);
        }
        u64 need = draw_ceil(p_in, Z);        // without top-k known after the first level
        // entries below this one weigh less than 1 - p of all together
        const float y0 = log2f(static_cast<float>(V) / ((1.f - fmaxf(p_in, 0.f)) * __ull2float_rn(Z))) + kOne + 0.25f;
        const float cut = fmaxf(fmaxf(__fsub_rd(m, y0 / weigh.scale() * 1.0001f), -FLT_MAX), from.thr);
        uint32_t lo = key_of(cut), hi = key_of(m);
        const float scale = linear_scale(cut, kMassBins);
        u64 under = 0ull;   // the weight above the range
        bool linear = true;
        while (true) {
          const float a = value_of(lo), b = value_of(hi);
          int step = max(0, 32 - __clz(hi - lo) - 10);
          if (step <= P::kFinal) step = P::kFinal;
          clear(kHistInts);
          const bool all_of = linear && !has_k;
          u64 sum = 0ull;
          each([&](const float* x, int v0) {
            if (__any_sync(kAll, all_of || largest4(x) >= a)) {
              u64 w[4];
#pragma unroll
              for (int i = 0; i < 4; i += 2) weigh.two(x[i], x[i + 1], w[i], w[i + 1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (all_of && x[i] > -INFINITY) sum += w[i];
                const unsigned bin = linear ? linear_bin(x[i], scale) : (hi - key_of(x[i])) >> step;
                if (x[i] >= a && x[i] <= b && from.keeps(x[i], v0 + i) && bin < kMassBins) {
                  if (!linear) atomicAdd(&hist[bin], 1u);
                  // 64 bits in two words: the lower one's old value tells the carry (3 cycles an
                  // SM each, where a 64-bit addition in shared memory takes 20 and more)
                  const unsigned low = static_cast<unsigned>(w[i]), old = atomicAdd(&hist[kMassBins + bin], low);
                  atomicAdd(&hist[2 * kMassBins + bin], static_cast<unsigned>(w[i] >> 32) + (old + low < old));
                }
              }
            }
          });
          if (all_of) {
            u64 before;
            join(warp_sum(sum), before, Z);
            need = draw_ceil(p_in, Z);
          }
          if (!find_bin(true, !linear, need - under)) break;   // cannot be: everything below the cut would be needed
          under += sh.above;
          const unsigned count = sh.count;
          narrow(linear, scale, step, lo, hi);
          if (!linear && count == 1u) {
            const float x = value_of(lo);
            keep = x <= from.thr ? from : Border{x, INT32_MAX};
            break;
          }
          if (!linear && step == P::kFinal) {                  // one value
            const float x = value_of(P::at_or_below(hi));
            const u64 w = weigh(x);                            // above 0: the sum grows in this bin
            const u64 r = (need - under + w - 1ull) / w;
            if (r < count) keep = Border{x, find_tie(x, static_cast<unsigned>(r))};
            else keep = x == from.thr ? from : Border{x, INT32_MAX};
            break;
          }
          if (linear) {
            // the bin's entries, if they fit the list: their order tells the border
            linear = false;
            settle();
            if (threadIdx.x == 0) sh.told.count = 0ull;
            __syncthreads();
            const float first_in = value_of(lo), last_in = value_of(hi);
            each([&](const float* x, int v0) {
              if (largest4(x) < first_in) return;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (x[i] >= first_in && x[i] <= last_in && from.keeps(x[i], v0 + i)) {
                  const unsigned at = atomicAdd(own_count, 1u);
                  if (at < kList) own[at] = static_cast<u64>(~key_of(x[i])) << 32 | static_cast<uint32_t>(v0 + i);
                }
              }
            });
            meet();
            const unsigned c = lane < parts ? static_cast<unsigned>(ld_peer_u64(&sh.told.count, lane)) : 0u;
            const unsigned all_len = __reduce_add_sync(kAll, c);
            const bool fits = all_len <= kList;
            if (fits && part == 0) pull(c);
            left();
            if (fits) {
              if (part == 0) {
                __syncthreads();
                order(kList, false, need - under, need - under, -FLT_MAX, false);
                __syncthreads();
                send();
              }
              meet();
              keep = sh.border;
              break;
            }
          }
        }
      }
      if (least > keep.thr) keep = Border{least, INT32_MAX};
      // the draw: every warp's kept weight, then the warp whose range holds the threshold
      u64 sum = 0ull, low_sum = 0ull, cum;
      const bool all_stay = keep.thr == -FLT_MAX && keep.cut == INT32_MAX && sums;
      each([&](const float* x, int v0) {
        if (all_stay) {
          weigh.add4(x, sum, low_sum);
          return;
        }
        if (__any_sync(kAll, largest4(x) >= keep.thr)) {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            u64 a, b;
            weigh.two(x[i], x[i + 1], a, b);
            sum += (keep.keeps(x[i], v0 + i) ? a : 0ull) + (keep.keeps(x[i + 1], v0 + i + 1) ? b : 0ull);
          }
        }
      });
      sum = warp_sum(all_stay ? (sum << 21) + low_sum : sum);
      join(sum, cum, total);
      if (p.tokens != nullptr) {
        bool whole;
        const u64 thr = draw_threshold(p.u[n], total, whole);
        // The warp whose range holds the threshold, in one CTA; that range's rows divided
        // over all its warps, then the one of these (a warp alone, its 74 rows one after
        // another: 1024 rows of 151936 bf16 entries 265 instead of 223 us).
        const bool here = cum <= thr && thr - cum < sum;
        if (threadIdx.x == 0) sh.at = -1;
        __syncthreads();
        if (here && lane == 0) {
          sh.at = warp;
          sh.above = cum;
        }
        __syncthreads();
        const int of = sh.at;
        if (of >= 0) {
          const int of_id = part * kWarps + of, of_row0 = static_cast<int>(static_cast<unsigned>(all_rows) * of_id / warps);
          const int of_rows = static_cast<int>(static_cast<unsigned>(all_rows) * (of_id + 1) / warps) - of_row0;
          const int r0 = of_rows * warp / kWarps, r1 = of_rows * (warp + 1) / kWarps;
          u64 w[VEC];
          auto weigh_row = [&](int r, int& v0) -> u64 {   // this lane's piece: its weights, their sum
            const int at = (of_row0 + r) * 32 + lane;
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            if (held) q = s_data[(of * rows + r) * 32 + lane];
            else if (at < pieces) q = clean(__ldg(base + at), at, true);
            else q = clean(q, at, true);
            float x[VEC];
            P::get(q, x);
            v0 = at * VEC - shift;
            u64 own_sum = 0ull;
#pragma unroll
            for (int i = 0; i < VEC; i += 2) weigh.two(x[i], x[i + 1], w[i], w[i + 1]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              if (!keep.keeps(x[i], v0 + i)) w[i] = 0ull;
              own_sum += w[i];
            }
            return own_sum;
          };
          u64 part_sum = 0ull;
          int v0;
#pragma unroll 1
          for (int r = r0; r < r1; ++r) part_sum += weigh_row(r, v0);
          part_sum = warp_sum(part_sum);
          if (lane == 0) sh.warp[0][warp] = part_sum;
          __syncthreads();
          u64 c0 = sh.above + warp_sum(lane < warp ? sh.warp[0][lane % kWarps] : 0ull);
          if (c0 <= thr && thr - c0 < part_sum) {
#pragma unroll 1
            for (int r = r0; r < r1; ++r) {
              const u64 own_sum = weigh_row(r, v0);
              const u64 incl = warp_scan(own_sum, lane);
              const unsigned hit = __ballot_sync(kAll, c0 + incl > thr);
              if (hit != 0u) {
                u64 c = c0 + incl - own_sum;
                int k = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                  c += w[i];
                  k += c <= thr;
                }
                const int token = __shfl_sync(kAll, v0 + k, __ffs(static_cast<int>(hit)) - 1);
                if (lane == 0) p.tokens[n] = token;
                break;
              }
              c0 += __shfl_sync(kAll, incl, 31);
            }
          }
        }
      }
    }
  }
  // ---------------------------------------------------------------- distribution
  if (probs != nullptr) {
    // 1 / total in two floats, so that a probability is rounded twice: as a weight, and here
    const float t = __ull2float_rn(total), inv = total > 0ull ? __fdiv_rn(1.f, t) : 0.f;
    const float rest = static_cast<float>(static_cast<long long>(total - static_cast<u64>(t)));
    const float low = inv * __fmaf_rn(-inv, rest, __fmaf_rn(-inv, t, 1.f));
    auto share = [&](u64 w) {
      const float x = __ull2float_rn(w);
      return __fmaf_rn(x, inv, x * low);
    };
    float* out = probs - shift;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    each([&](const float* x, int v0) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = 0.f;
      if (__any_sync(kAll, largest4(x) >= keep.thr)) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          u64 a, b;
          weigh.two(x[i], x[i + 1], a, b);
          if (keep.keeps(x[i], v0 + i)) y[i] = share(a);
          if (keep.keeps(x[i + 1], v0 + i + 1)) y[i + 1] = share(b);
        }
      }
      if (aligned && v0 >= 0 && v0 + 4 <= V) {
#pragma unroll
        for (int i = 0; i < 4; i += 4) __stcs(reinterpret_cast<float4*>(probs + v0 + i), make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (v0 + i >= 0 && v0 + i < V) probs[v0 + i] = y[i];
      }
    });
  }
  settle();   // no peer reads this CTA's memory any more
}

template <typename TT>
cudaError_t launch_typed(const DrawArgs& a, cudaStream_t s, bool pdl) {
  constexpr int kMaxSmem = 10 * kWarps * 32 * 16 + kScratchBytes;
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
  const int all_rows = (pieces + 31) / 32;
  auto rows_of = [&](int parts) { return (all_rows + parts * kWarps - 1) / (parts * kWarps); };
  // CTAs a row: as many as find room at once, two an SM, while each warp has two rows of
  // 16-byte pieces; at least as many as keep what is read again within L2 (96 MB for
  // the rows under way). Clusters of 16 find no room beside one another: only for few rows.
  // (Twice as many, in two rounds: 64 rows bf16 with top-k 20 27.6 instead of 17.6 us, 272
  // rows f32 75 instead of 64; rows of all kinds, where the flat ones decide, 54.7 / 54.9
  // and 155 / 200.)
  const long long slots = 2LL * num_sms_of_current_device();
  const long long row_bytes = 16LL * pieces;
  int parts = 1;
  while (parts < 8 && slots / parts * row_bytes > 96LL << 20 && a.N * row_bytes > 96LL << 20) parts *= 2;
  while (parts < (a.N <= 4 ? kMaxParts : 8) && 2LL * parts * a.N <= slots && rows_of(parts) > 2) parts *= 2;
  // held in shared memory where two CTAs find room (ten rows a warp: 80 KB)
  const int rows = rows_of(parts) <= 10 ? rows_of(parts) : 0;
  const size_t smem = static_cast<size_t>(rows) * kWarps * 32 * 16 + kScratchBytes;
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
