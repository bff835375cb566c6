// Chunk attention over a paged KV cache on the 5th-generation tensor cores.
//
//   S = Q K^T (fp32 in TMEM);  P = 2^(scale S - m) (bf16);  O += P V (fp32)
//
// Units of work. The G query heads of a KV head are packed into the rows of
// one tile (row = token * G + head), so a page's K and V are read once for all
// of them. A unit is up to two 128-row tiles of one (sequence, KV head):
// 2 * floor(128 / G) tokens. Its work is its 128-key pages, up to the last key its last
// token sees, and a share of its own. All units, laid end to end, are cut into
// ranges of equal cost, one a CTA and one CTA an SM, whatever mix of long prompts
// and single tokens the batch holds: a CTA walks through its range, and only
// the first and the last unit of a range can be incomplete. Incomplete units
// write unnormalised rows to the workspace; chunk_merge_kernel joins them in
// key order. Over few pages (whole_units) a unit goes to the CTA in whose range it
// starts, and no merge follows.
//
// Two streams keep the tensor core busy: each has its own S / P and O columns in
// TMEM and its own four softmax warps, one thread a row.
//   pair mode  (a unit of more than one tile): stream s takes rows of tile s,
//              both the same keys; a K or V page in shared memory serves both;
//   split mode (one tile of rows: decoding, a drafted block, a chunk's rest):
//              both streams take the same rows, alternate pages, and their
//              (O, max, sum) are joined at the end of the piece.
// So while one stream's scores are in the softmax, the other's products run.
// P goes back to TMEM over the columns of its own S (bf16, half the columns)
// and is the A operand of the second product. P is rounded to bf16 because both
// operands of a product have one type and V is bf16 (fp32 weights would need a
// tf32 product at half the rate and a copy of V): half a step, 2^-8 of a weight,
// of either sign. The row's sum adds the weights before that rounding, scores,
// maximum, sum and O stay fp32, and the exponentials' own error (2^-22) lies far
// below it. Against 64 bits 1.9 to 2.3e-3 relative, where an output that is only
// rounded once to bf16 has 1.7e-3. A warp of its own issues each
// stream's MMAs, S of the next page after P V of the last one on the same
// columns; the tensor core executes them in that order.
//
// K, V pages come by TMA through a ring of 32 KB stages that runs on across
// units, Q tiles through two buffers, so the next unit's loads are in flight
// while the current one ends.
#include "chunk.cuh"

namespace dfl {
namespace {

constexpr int kKeys = kPageKeys;             // keys of a tile: one page
constexpr uint32_t kSubTile = 128 * 128;     // 128 rows x 128 bytes, swizzled
constexpr int kStages = 5;                   // K / V ring
constexpr int kTcThreads = 384;              // K and V, 2 x MMAs, Q; 2 x 4 softmax warps
constexpr int kLoadRegs = 72, kSoftmaxRegs = 216;   // 128 * 72 + 256 * 216 = 384 * 168
constexpr float kLog2eTc = 1.4426950408889634f;
constexpr float kLag = 8.0f;                 // log2 units that the running maximum may lag behind

struct ChunkSmem {
  uint64_t kv_full[kStages], kv_empty[kStages], q_full[2], q_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], turn[2], drained[2];
  uint32_t tmem_base;
  int abort_flag;
  int start[7];                // where this CTA begins: sequence, unit, KV head, position in the unit; the sequence's rows and lengths
  long long warp_sum[kTcThreads / 32];
  float row_max[2][128], row_sum[2][128];   // split mode: the streams' statistics
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// Tensor-core instructions of a converged warp: one elected lane (the same one
// every time) issues a product's MMAs. The election and the MMAs are one block:
// issued so, eight MMAs cost 170 cycles; with an election each 340; one by one
// from a branch that one lane takes 570 to 830, more than the 512 that the
// tensor core needs for them.
#define DFL_ELECT "elect.sync _|e, 0xffffffff;\n\t"
#define DFL_MMA_SS(off, acc)                                 \
  "add.s64 a, %1, " #off ";\n\tadd.s64 b, %2, " #off ";\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " #acc ";\n\t"
// D[tmem] = A[smem] * B[smem]^T over a depth of DH: 16 columns are 32 bytes (2 in
// a descriptor's address), a 64-column half is kSubTile on (1024).
template <int DH>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  static_assert(kSubTile == 1024 * 16, "offset of the second half");
  if (DH == 128) {
    asm volatile(
        "{\n\t.reg .pred n, y, e;\n\t.reg .b64 a, b;\n\t" DFL_ELECT "setp.ne.b32 n, 0, 0;\n\tsetp.eq.b32 y, 0, 0;\n\t"
        DFL_MMA_SS(0, n) DFL_MMA_SS(2, y) DFL_MMA_SS(4, y) DFL_MMA_SS(6, y)
        DFL_MMA_SS(1024, y) DFL_MMA_SS(1026, y) DFL_MMA_SS(1028, y) DFL_MMA_SS(1030, y) "}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred n, y, e;\n\t.reg .b64 a, b;\n\t" DFL_ELECT "setp.ne.b32 n, 0, 0;\n\tsetp.eq.b32 y, 0, 0;\n\t"
        DFL_MMA_SS(0, n) DFL_MMA_SS(2, y) DFL_MMA_SS(4, y) DFL_MMA_SS(6, y) "}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc)
        : "memory");
  }
}
#define DFL_MMA_TS(col, off, acc)                            \
  "add.s32 a, %1, " #col ";\n\tadd.s64 b, %2, " #off ";\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, " #acc ";\n\t"
// D[tmem] (+)= A[tmem] * B[smem] over 64 keys from 16 KS0 on: row r of A in TMEM lane
// r, two consecutive keys a column; 16 keys of B are 2048 bytes (128).
template <int KS0>
__device__ __forceinline__ void mma_values(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  if (KS0 == 0) {
    asm volatile(
        "{\n\t.reg .pred p, y, e;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t" DFL_ELECT
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 y, 0, 0;\n\t"
        DFL_MMA_TS(0, 0, p) DFL_MMA_TS(8, 128, y) DFL_MMA_TS(16, 256, y) DFL_MMA_TS(24, 384, y) "}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred y, e;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t" DFL_ELECT "setp.eq.b32 y, 0, 0;\n\t"
        DFL_MMA_TS(32, 512, y) DFL_MMA_TS(40, 640, y) DFL_MMA_TS(48, 768, y) DFL_MMA_TS(56, 896, y) "}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc)
        : "memory");
  }
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t" DFL_ELECT
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t l2_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// Matrix descriptors in two words (the fields of sw128_desc and sw128_desc_mn):
// the low one holds the address / 16 and, for values, the byte offset / 16
// between 64-column halves; the high one is the same for all.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr) { return (smem_addr & 0x3FFFFu) >> 4; }
// A value that all lanes hold alike, told to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// Bounded wait that also ends (false) once any role of the CTA gave up. The
// polling loop is a call, as is all code that is run rarely: inlined wherever
// it is used, it made a kernel of 110 KB, whose roles drove each other's code
// out of the instruction cache (thousands of cycles at every unit's end).
__device__ __forceinline__ bool poll_bar(uint32_t bar, uint32_t parity, int* abort_flag, int* status) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(abort_flag)) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      report(status, DFLASH_ERR_TIMEOUT);
      atomicExch(abort_flag, 1);
      return false;
    }
  }
  return true;
}
__device__ __noinline__ bool poll_bar_call(uint32_t bar, uint32_t parity, int* abort_flag, int* status) {
  return poll_bar(bar, parity, abort_flag, status);
}
// Waits of a converged warp: a call in the warps that load and issue, inline in the
// softmax, whose registers are full.
__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, ChunkSmem* h, int* status) {
  const uint32_t b = smem_u32(bar);
  const bool ok = mbar_try_wait(b, parity) || poll_bar_call(b, parity, &h->abort_flag, status);
  return __all_sync(0xffffffffu, ok) != 0;
}
__device__ __forceinline__ bool softmax_wait_bar(uint64_t* bar, uint32_t parity, ChunkSmem* h, int* status) {
  const uint32_t b = smem_u32(bar);
  const bool ok = mbar_try_wait(b, parity) || poll_bar(b, parity, &h->abort_flag, status);
  return __all_sync(0xffffffffu, ok) != 0;
}
// a * b / c; a 64-bit division takes some 300 cycles, at the start of every CTA
__device__ __noinline__ long long mul_div64(long long a, long long b, long long c) { return a * b / c; }
__device__ __forceinline__ long long mul_div(long long a, int b, long long c) {
  if (a < (1 << 22) && c < (1 << 22)) return static_cast<uint32_t>(a) * static_cast<uint32_t>(b) / static_cast<uint32_t>(c);   // b <= 1024
  return mul_div64(a, b, c);
}
// A warp's arrival, behind its lanes' TMEM accesses.
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(bar));
}

// O row *= f, in TMEM.
template <int DH>
__device__ __forceinline__ void rescale(uint32_t t_o, float f) {
#pragma unroll 1
  for (int c = 0; c < DH; c += 16) {
    float o[16];
    tmem_ld16(t_o + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= f;
    tmem_st16(t_o + c, o);
  }
}

// 32 columns of a warp's 32 output rows as bf16, a row a lane, to rows that lie
// apart: four lanes exchange 16-byte pieces so that each then stores one piece
// of each of their four rows, 64 contiguous bytes a row (stored straight from
// the row's own lane, every 16 bytes are a line of their own; a unit of one
// page took 7.7 us, most of it here). rows: the four lanes' rows, -1 for none.
__device__ __forceinline__ void store_rows32(__nv_bfloat16* out, const long long* rows, const float* o, float f, int lane) {
  uint32_t c[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = pack_bf16(o[8 * i + 2 * j] * f, o[8 * i + 2 * j + 1] * f);
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t t = __shfl_xor_sync(0xffffffffu, up ? c[i][j] : c[i | bit][j], bit);
        if (up) c[i][j] = t; else c[i | bit][j] = t;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (rows[i] >= 0) *reinterpret_cast<uint4*>(out + rows[i] + (lane & 3) * 8) = make_uint4(c[i][0], c[i][1], c[i][2], c[i][3]);
  }
}

// Pages of unit j of a sequence of n rows behind ctx keys; a unit without keys
// still takes one (masked) page, so that its rows are written.
__device__ __forceinline__ int unit_pages(const ChunkArgs& p, int n, int ctx, int j, int unit_tok) {
  ChunkUnit u{0, 0, n, ctx, 0};
  const int keys = row_keys(p, u, min((j + 1) * unit_tok, n) - 1);
  return max(1, (keys + kKeys - 1) / kKeys);
}

// Stage and phase of the i-th load of the ring.
struct RingPos {
  int st;
  uint32_t phase;
  __device__ __forceinline__ explicit RingPos(int i) : st(i % kStages), phase((i / kStages) & 1) {}
  __device__ __forceinline__ RingPos plus(int n) const {   // n <= kStages
    RingPos r = *this;
    r.st += n;
    if (r.st >= kStages) { r.st -= kStages; r.phase ^= 1u; }
    return r;
  }
};

// Cost of a unit in thirds of a microsecond: its own share (Q, the first page's
// latency, the rows' way out), then its pages. From 1520 units of one and of eight
// pages: two tiles of rows 5 us and 1.7 us a page; one tile 3 to 4 us, by its
// rows, and 1.4 us a page. Cut by pages alone, the first CTA of an 8192-token
// prompt got 60 short units and ran 1.6 times as long as the others (614 us
// instead of 380). Measured with 32 heads over 8 of 128 and used for every layout:
// heads of 64 have half the bytes and products a page but the same softmax. Only
// how evenly the CTAs end depends on it.
__device__ __forceinline__ bool is_pair(int n_tok, int unit_tok) { return n_tok * 2 > unit_tok; }
__device__ __forceinline__ int unit_share(int n_tok, int unit_tok) {
  return is_pair(n_tok, unit_tok) ? 15 : n_tok * 8 > unit_tok ? 12 : 9;   // more than 32 rows of 256
}
__device__ __forceinline__ int page_share(bool pair) { return pair ? 5 : 4; }
constexpr int kMinRange = 8;   // a CTA's least range: at least one page of any kind

__device__ __forceinline__ int unit_cost(const ChunkArgs& p, int n, int ctx, int j, int unit_tok) {
  const int n_tok = min(unit_tok, n - j * unit_tok);
  return unit_share(n_tok, unit_tok) + unit_pages(p, n, ctx, j, unit_tok) * page_share(is_pair(n_tok, unit_tok));
}

// A CTA's walk over its range: the current piece.
struct Walk {
  int b, j, kvh;        // unit
  int row0, n, ctx;     // its sequence
  int pages;            // the unit's pages
  int kt0, nt;          // the piece: pages kt0 .. kt0 + nt - 1
  int begin, end;       // the range's ends, relative to the unit's first position
  int tok0, n_tok;      // the unit's tokens
  int share;            // its own share of the cost
  bool pair, more;

  __device__ __forceinline__ void load_unit(const ChunkArgs& p, int unit_tok) {
    tok0 = j * unit_tok;
    n_tok = min(unit_tok, n - tok0);
    pages = unit_pages(p, n, ctx, j, unit_tok);
    pair = is_pair(n_tok, unit_tok);
    share = unit_share(n_tok, unit_tok);
  }
  __device__ __forceinline__ int span() const { return share + pages * page_share(pair); }
  // Pages whose position (the unit's share, then page by page) lies before x.
  __device__ __forceinline__ int pages_before(int x) const {
    const int d = x - share;
    const unsigned up = static_cast<unsigned>(max(d, 0) + page_share(pair) - 1);
    return min(pages, static_cast<int>(pair ? up / 5u : up / 4u));
  }
  __device__ __forceinline__ void place(const ChunkArgs& p) {
    if (p.whole_units) {   // a unit belongs to the range it starts in
      kt0 = 0;
      nt = begin <= 0 && end > 0 ? pages : 0;
    } else {
      kt0 = pages_before(begin);
      nt = pages_before(end) - kt0;
    }
  }
  __device__ __forceinline__ void start(const ChunkArgs& p, const ChunkSmem* h, int count, int unit_tok) {
    more = count > 0;
    if (!more) return;
    b = h->start[0]; j = h->start[1]; kvh = h->start[2];
    begin = h->start[3];
    end = begin + count;
    row0 = h->start[4]; n = h->start[5]; ctx = h->start[6];
    load_unit(p, unit_tok);
    place(p);
    if (nt == 0) next(p, unit_tok);   // behind the last page's position, or before the first one's
  }
  __device__ __forceinline__ void next(const ChunkArgs& p, int unit_tok) {
    const int used = span();
    begin -= used;
    end -= used;
    more = end > 0;
    if (!more) return;
    if (++kvh == p.n_kv_heads) {
      kvh = 0;
      if (tok0 + n_tok >= n) {
        j = 0;
        do {
          ++b;
          chunk_rows(p, b, row0, n);
        } while (n == 0 && b + 1 < p.B);
        ctx = p.ctx_len[b];
      } else {
        ++j;
      }
      load_unit(p, unit_tok);
    }
    place(p);
    more = nt > 0;   // a range that ends in a unit's own share has none of its pages
  }
  __device__ __forceinline__ bool whole() const { return nt == pages; }
  // tiles of stream s, and the page (relative to kt0) of its k-th
  __device__ __forceinline__ int count(int s) const { return pair ? nt : (nt + 1 - s) >> 1; }
  __device__ __forceinline__ int tile(int s, int k) const { return pair ? k : 2 * k + s; }
};

template <int DH>
__global__ void __launch_bounds__(kTcThreads, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const ChunkArgs p) {
  constexpr int NSUB = DH / 64;
  constexpr uint32_t kTileBytes = NSUB * kSubTile;
  constexpr uint32_t kOCol = 256;
  extern __shared__ __align__(1024) uint8_t smem_raw[];   // tiles, then the header
  ChunkSmem* hdr = reinterpret_cast<ChunkSmem*>(smem_raw + (2 + kStages) * kTileBytes);
  const uint32_t q_s = smem_u32(smem_raw), kv_s = q_s + 2 * kTileBytes;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.n_q_heads / p.n_kv_heads;
  const int tile_tok = 128 / G, unit_tok = 2 * tile_tok;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&hdr->kv_full[i]), 1);
      mbar_init(smem_u32(&hdr->kv_empty[i]), 2);   // a stream each
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&hdr->q_full[i]), 1);
      mbar_init(smem_u32(&hdr->q_empty[i]), 2);
      mbar_init(smem_u32(&hdr->s_full[i]), 1);
      mbar_init(smem_u32(&hdr->p_half[i]), 4);   // a softmax warp each
      mbar_init(smem_u32(&hdr->p_full[i]), 4);
      mbar_init(smem_u32(&hdr->o_full[i]), 1);
      mbar_init(smem_u32(&hdr->turn[i]), 1);
      mbar_init(smem_u32(&hdr->drained[i]), 1);
    }
    hdr->abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async();
    tma_prefetch_map(&q_map);
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&hdr->tmem_base), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();   // after the wait: the merge may read what this kernel may read
  if (threadIdx.x == 96) p.desc[blockIdx.x * kChunkDescInts] = 0;   // no incomplete unit starts here yet

  // ---------------------------------------------------------------- ranges
  // The units' cost for one KV head, summed by threads over contiguous runs of
  // units (parts of a sequence, or whole sequences where there are more of them
  // than threads); a scan gives the total and finds where this CTA begins.
  long long mine = 0;
  const int per = (p.B + kTcThreads - 1) / kTcThreads, parts = max(1, kTcThreads / p.B);
  const int part = threadIdx.x % parts;
  const int b_first = threadIdx.x / parts * per, b_last = min(p.B, b_first + per);
#pragma unroll 1
  for (int b = b_first; b < b_last; ++b) {
    int row0, n;
    chunk_rows(p, b, row0, n);
    const int ctx = p.ctx_len[b], units = (n + unit_tok - 1) / unit_tok;
    const int j1 = units * (part + 1) / parts;
#pragma unroll 1
    for (int j = units * part / parts; j < j1; ++j) mine += unit_cost(p, n, ctx, j, unit_tok);
    if (blockIdx.x == 0 && part == 0 && n > 0) check_capacity(p, ChunkUnit{b, row0, n, ctx, 0});
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) hdr->warp_sum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = hdr->tmem_base;
  long long before = incl - mine, total = 0;
  for (int w = 0; w < kTcThreads / 32; ++w) {
    if (w < warp) before += hdr->warp_sum[w];
    total += hdr->warp_sum[w];
  }
  total *= p.n_kv_heads;
  before *= p.n_kv_heads;
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), max(total / kMinRange, 1LL)));
  const int cta = blockIdx.x;
  const long long first = cta < ctas ? mul_div(total, cta, ctas) : total;
  const int count = cta < ctas ? static_cast<int>(mul_div(total, cta + 1, ctas) - first) : 0;
  if (count > 0 && first >= before && first < before + mine * p.n_kv_heads) {
    long long rem = first - before;
#pragma unroll 1
    for (int b = b_first; b < b_last; ++b) {
      int row0, n;
      chunk_rows(p, b, row0, n);
      const int ctx = p.ctx_len[b], units = (n + unit_tok - 1) / unit_tok;
      const int j1 = units * (part + 1) / parts;
      bool found = false;
#pragma unroll 1
      for (int j = units * part / parts; j < j1 && !found; ++j) {
        const int cost = unit_cost(p, n, ctx, j, unit_tok);
        if (rem < static_cast<long long>(cost) * p.n_kv_heads) {
          hdr->start[0] = b; hdr->start[1] = j;
          hdr->start[2] = static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(cost));   // rem < cost * Hkv
          hdr->start[3] = static_cast<int>(static_cast<uint32_t>(rem) % static_cast<uint32_t>(cost));
          hdr->start[4] = row0; hdr->start[5] = n; hdr->start[6] = ctx;
          found = true;
        } else {
          rem -= static_cast<long long>(cost) * p.n_kv_heads;
        }
      }
      if (found) break;
    }
  }
  __syncthreads();
  int* status = p.dev_status;
  // The walk begins in each branch: alive across it, it spilled in both (56 bytes of
  // stack, and 3 to 10 % of the time: 2048 rows behind 6000 keys 166 instead of 161 us).
  if (warp < 4) {
    regs_dec<kLoadRegs>();
    Walk w;
    w.start(p, hdr, count, unit_tok);
    if (warp == 0) {
      // -------------------------------------------------------------- K and V
      const uint64_t once = l2_evict_first(), again = l2_evict_normal();
      int g = 0, issued = 0;   // loads so far, of which issued (a failed wait skips one)
      bool ok = true;
      for (; w.more && ok; w.next(p, unit_tok)) {
        // a sequence of several units reads its pages again from L2
        const uint64_t pol = w.n > unit_tok ? again : once;
        const int32_t* table = p.pages.table + static_cast<size_t>(w.b) * p.pages.pages_per_seq;
        const bool keyless = w.ctx + w.n <= 0;
        int ids = 0;
        for (int t = 0; t < w.nt && ok; ++t) {
          if ((t & 31) == 0) {
            const int at = w.kt0 + t + lane;
            ids = 0;
            if (t + lane < w.nt && !keyless) {
              ids = table[at];
              if (ids < 0 || ids >= p.pages.n_pages) {   // not a page: page 0 is read instead
                report(status, DFLASH_ERR_CAPACITY);
                ids = 0;
              }
            }
          }
          const int page = __shfl_sync(0xffffffffu, ids, t & 31);
          const int z = (p.layer * p.pages.n_pages + page) * p.n_kv_heads + w.kvh;
          for (int v = 0; v < 2 && ok; ++v, ++g) {
            const int st = g % kStages;
            if (g >= kStages) ok = warp_wait_bar(&hdr->kv_empty[st], (g / kStages - 1) & 1, hdr, status);
            if (ok && lane == 0) {
              const uint32_t bar = smem_u32(&hdr->kv_full[st]);
              mbar_expect_tx(bar, kTileBytes);
#pragma unroll
              for (int s = 0; s < NSUB; ++s)
                tma_load_3d(kv_s + st * kTileBytes + s * kSubTile, v ? &v_map : &k_map, bar, 64 * s, 0, z, pol);
            }
            if (ok) issued = g + 1;
          }
        }
      }
      // after a timeout no load of this CTA may still be landing when it exits
      if (lane == 0 && *reinterpret_cast<volatile int*>(&hdr->abort_flag)) {
        for (int i = max(0, issued - kStages); i < issued; ++i) mbar_wait(smem_u32(&hdr->kv_full[i % kStages]), (i / kStages) & 1);
      }
      __syncwarp();
    } else if (warp == 3) {
      // -------------------------------------------------------------- Q
      // A warp of its own: waiting for a Q buffer holds up no K or V.
      const uint32_t q_bytes = static_cast<uint32_t>(NSUB) * 128u * (tile_tok * G);
      const uint64_t once = l2_evict_first();
      int qi = 0, issued = 0;
      bool ok = true;
      for (; w.more && ok; w.next(p, unit_tok)) {
        // the unit that starts here and goes on in the next CTAs: what to join
        if (lane == 0 && w.kt0 == 0 && !w.whole()) {
          // its last page lies in the last CTA whose range starts at or before that page
          const long long x = first - w.begin + w.share + (w.pages - 1) * page_share(w.pair);
          const int last = static_cast<int>(mul_div64((x + 1) * ctas + total - 1, 1, total)) - 1;
          int* d = p.desc + cta * kChunkDescInts;
          d[0] = last - cta + 1;
          d[1] = w.row0 + w.tok0;
          d[2] = w.n_tok;
          d[3] = w.kvh;
          d[4] = 2 * cta + 1;
          d[5] = 2 * (cta + 1);
          d[6] = 2;
        }
        const int nq = w.pair ? 2 : 1;
        for (int i = 0; i < nq && ok; ++i, ++qi) {
          const int buf = qi & 1;
          if (qi >= 2) ok = warp_wait_bar(&hdr->q_empty[buf], ((qi >> 1) - 1) & 1, hdr, status);
          if (ok && lane == 0) {
            const uint32_t bar = smem_u32(&hdr->q_full[buf]);
            mbar_expect_tx(bar, q_bytes);
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
              tma_load_3d(q_s + buf * kTileBytes + s * kSubTile, &q_map, bar, 64 * s, w.kvh * G,
                          w.row0 + w.tok0 + i * tile_tok, once);
          }
          if (ok) issued = qi + 1;
        }
      }
      if (lane == 0 && *reinterpret_cast<volatile int*>(&hdr->abort_flag)) {
        for (int i = max(0, issued - 2); i < issued; ++i) mbar_wait(smem_u32(&hdr->q_full[i & 1]), (i >> 1) & 1);
      }
      __syncwarp();
    } else if (warp < 3) {
      // -------------------------------------------------------------- MMAs
      // A warp a stream. Waits (100 cycles each even where nothing is to be
      // waited for) and issuing are kept off the path from a page's weights to
      // the next page's scores: everything else is awaited before the weights,
      // and both products then issue in one go.
      const int s = warp - 1;
      const uint32_t idesc_s = make_idesc(128, kKeys, kFmtBF16);
      const uint32_t idesc_o = make_idesc(128, DH, kFmtBF16, 1);
      const uint32_t t_s = uniform(tmem + s * 128), t_o = uniform(tmem + kOCol + s * DH);
      int g0 = 0, qi = 0, tiles = 0, turns = 0;   // loads, Q tiles, stream tiles and turns before this piece
      bool ok = true;
      for (; w.more && ok; w.next(p, unit_tok)) {
        // Both streams take every load in order, also those that only the other
        // one reads: a barrier's phases are seen one by one, and none passes
        // before both saw it.
        const bool pair = w.pair;
        const int n = w.count(s), qt = qi + (pair ? s : 0);   // this stream's Q tile
        const int qo = pair ? qi + 1 - s : n == 0 ? qt : -1;  // a Q tile it only passes
        RingPos at(g0), v = at;
        auto wait_load = [&](const RingPos& r) { ok = ok && warp_wait_bar(&hdr->kv_full[r.st], r.phase, hdr, status); };
        if (n > 0) ok = warp_wait_bar(&hdr->q_full[qt & 1], (qt >> 1) & 1, hdr, status);
        const uint64_t qd = desc_of(uniform(desc_lo(q_s + (qt & 1) * kTileBytes)), kDescHi);
#pragma unroll 1
        for (int k = 0; k <= n && ok; ++k) {
          if (k > 0) {   // P V of page k - 1
            const uint32_t phase = (tiles + k - 1) & 1;
            v = at.plus(1);
            at = at.plus(2);
            wait_load(v);
            if (pair && k < n) wait_load(at);
            // 64-column halves of V lie kSubTile apart
            const uint64_t vd = desc_of(uniform(desc_lo(kv_s + v.st * kTileBytes) + ((kSubTile >> 4) << 16)), kDescHi);
            // the weights come in two halves of 64 keys, the first while the softmax still works on the second
            ok = ok && warp_wait_bar(&hdr->p_half[s], phase, hdr, status);
            // pair mode: in turn, so that one stream's softmax runs beside the other's products
            if (pair && turns + k - 1 + s > 0) ok = ok && warp_wait_bar(&hdr->turn[s], (turns + k - 2 + s) & 1, hdr, status);
            if (!ok) break;
            tc_fence_after();
            mma_values<0>(t_o, t_s, vd, idesc_o, k > 1 ? 1u : 0u);
            ok = warp_wait_bar(&hdr->p_full[s], phase, hdr, status);
            if (!ok) break;
            tc_fence_after();
            mma_values<4>(t_o, t_s, vd, idesc_o, 1u);
            if (k == n) mma_commit(&hdr->o_full[s]);
            if (!pair) mma_commit(&hdr->kv_empty[v.st]);
          }
          // split mode: the other stream's page before this stream's k-th
          if (!pair && 2 * k + s >= 1 && 2 * k + s - 1 < w.nt) {
#pragma unroll 1
            for (int i = 0; i < 2 && ok; ++i) {
              wait_load(at);
              if (ok && lane == 0) mbar_arrive(smem_u32(&hdr->kv_empty[at.st]));
              at = at.plus(1);
            }
          }
          if (k < n) {   // S of page k
            if (!pair || k == 0) wait_load(at);
            if (!ok) break;
            tc_fence_after();
            mma_scores<DH>(t_s, qd, desc_of(uniform(desc_lo(kv_s + at.st * kTileBytes)), kDescHi), idesc_s);
            mma_commit(&hdr->s_full[s]);
            mma_commit(&hdr->kv_empty[at.st]);
            if (k == n - 1) mma_commit(&hdr->q_empty[qt & 1]);
          }
          if (pair && k > 0) {
            if (lane == 0) mbar_arrive(smem_u32(&hdr->turn[1 - s]));
            mma_commit(&hdr->kv_empty[v.st]);
          }
          if (k == 0 && qo >= 0) {   // early: the tile is free once the other stream is done with it
            ok = warp_wait_bar(&hdr->q_full[qo & 1], (qo >> 1) & 1, hdr, status);
            if (ok && lane == 0) mbar_arrive(smem_u32(&hdr->q_empty[qo & 1]));
          }
        }
        g0 += 2 * w.nt;
        qi += pair ? 2 : 1;
        tiles += n;
        if (pair) turns += n;
      }
      // every MMA issued is done before the block frees its TMEM
      mma_commit(&hdr->drained[s]);
      mbar_wait(smem_u32(&hdr->drained[s]), 0);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    regs_inc<kSoftmaxRegs>();
    Walk w;
    w.start(p, hdr, count, unit_tok);
    const int s = (warp - 4) >> 2;                       // stream
    const int r = (warp & 3) * 32 + lane;                // row of the stream's tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + s * 128;
    const float scale = p.scale * kLog2eTc;
    const int r_tok = r / G, r_head = r - r_tok * G;
    int g0 = 0, tiles = 0, pieces[2] = {0, 0};
    bool ok = true;
    for (; w.more; w.next(p, unit_tok)) {
      const bool pair = w.pair;
      const int ns = w.count(s);
      const int tok = (pair ? s * tile_tok : 0) + r_tok;   // token of the unit
      const bool valid = r_tok < tile_tok && tok < w.n_tok;
      const ChunkUnit u{w.b, w.row0, w.n, w.ctx, w.tok0};
      const int lim = valid ? row_keys(p, u, w.tok0 + tok) : 0;
      const bool live = __any_sync(0xffffffffu, valid) != 0;   // warp-uniform
      const int keys = max(0, min(w.ctx + w.n, p.pages.pages_per_seq * kPageKeys));   // rows of the cache that hold keys
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < ns && ok; ++k) {
        const int t = w.tile(s, k);
        const int kb = (w.kt0 + t) * kKeys;
        ok = softmax_wait_bar(&hdr->s_full[s], (tiles + k) & 1, hdr, status);
        if (!ok) break;
        tc_fence_after();
        if (keys - kb < kKeys) {
          // rows of the last page behind the last key: zero their values (0 * NaN
          // would poison O). In pair mode both streams do, each before its own product.
          const int g = g0 + 2 * t + 1, st = g % kStages;
          ok = softmax_wait_bar(&hdr->kv_full[st], (g / kStages) & 1, hdr, status);
          if (!ok) break;
          if (r >= keys - kb) {
            const uint32_t vt = kv_s + st * kTileBytes + r * 128;
#pragma unroll
            for (int i = 0; i < NSUB; ++i)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + i * kSubTile + c * 16), "r"(0u) : "memory");
          }
          fence_proxy_async();
        }
        if (live) {
          // Scores that the row does not see are overwritten where they lie. (A
          // page that is cut anywhere is a unit's last one or two.)
          const int seen = lim - kb;      // keys of this page that the row sees
          if (__any_sync(0xffffffffu, seen < kKeys)) {
            // From the first column that a row of the warp's does not see; behind the last
            // one that any sees unread. (All columns read and written: six prompts of 500
            // to 2000 tokens 137 instead of 114 us.)
            const int all = __reduce_min_sync(0xffffffffu, valid ? max(seen, 0) : kKeys);
            const int some = __reduce_max_sync(0xffffffffu, seen);
#pragma unroll 1
            for (int c = all & ~15; c < kKeys; c += 16) {
              float v[16];
              if (c < some) {
                tmem_ld16(t_s + c, v);
                tmem_ld_wait();
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = c + i < seen ? v[i] : -INFINITY;
              tmem_st16(t_s + c, v);
            }
            tmem_st_wait();
          }
          // The row's scores are read in halves: the second once for the maximum
          // and again for its exponentials, so that at most 96 of them are live
          // (all 128 kept: 2048 rows behind 6000 keys 169 instead of 161 us; the
          // maximum of the first half under the second one's load: 164). P of keys
          // 2c, 2c + 1 goes to column c: columns that hold scores not yet turned into
          // weights are never hit.
          float x[64], y[32];
          float top;
          {
            float z[64];
            tmem_ld32(t_s + 64, z);
            tmem_ld32(t_s + 96, z + 32);
            tmem_ld32(t_s, x);
            tmem_ld32(t_s + 32, x + 32);
            tmem_ld_wait();
            float m0 = max3(x[0], x[1], z[0]), m1 = max3(x[2], x[3], z[1]), m2 = max3(x[4], x[5], z[2]),
                  m3 = max3(x[6], x[7], z[3]);
#pragma unroll
            for (int i = 8; i < 64; i += 8) {
              m0 = max3(m0, x[i], x[i + 1]); m1 = max3(m1, x[i + 2], x[i + 3]);
              m2 = max3(m2, x[i + 4], x[i + 5]); m3 = max3(m3, x[i + 6], x[i + 7]);
            }
#pragma unroll
            for (int i = 4; i < 60; i += 8) {
              m0 = max3(m0, z[i], z[i + 1]); m1 = max3(m1, z[i + 2], z[i + 3]);
              m2 = max3(m2, z[i + 4], z[i + 5]); m3 = max3(m3, z[i + 6], z[i + 7]);
            }
            m0 = max3(m0, z[60], z[61]); m1 = max3(m1, z[62], z[63]);
            top = fmaxf(max3(m0, m1, m2), m3) * scale;
          }
          // the maximum is raised only when it grew by more than 2^kLag: P and
          // the sums stay far inside fp32 and bf16 range, and O is rarely touched
          const bool raise = top > m + kLag;
          if (k > 0 && __any_sync(0xffffffffu, raise)) {
            // S of this page was issued after P V of the last one: O is at rest
            const float f = raise ? ex2(m - top) : 1.f;
            l *= f;
            rescale<DH>(tmem + lanes + kOCol + s * DH, f);
          }
          if (raise) m = top;
          const float ref = m == -INFINITY ? 0.f : m;   // nothing seen yet: every term is 2^-inf = 0
          const uint64_t scale2 = pair2(scale, scale), ref2 = pair2(-ref, -ref);
          uint64_t sum2[2] = {0ull, 0ull};
          auto weights = [&](const float* v, int col) {   // 32 scores to P's 16 columns from col on
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const uint64_t e = fma2(pair2(v[i], v[i + 1]), scale2, ref2);
              const float a = ex2(lo_of(e)), b = ex2(hi_of(e));
              sum2[(i >> 1) & 1] = add2(sum2[(i >> 1) & 1], pair2(a, b));
              pk[i >> 1] = pack_bf16(a, b);
            }
            tmem_st16u(t_s + col, pk);
          };
          tmem_ld32(t_s + 64, y);
          weights(x, 0);
          weights(x + 32, 16);
          tmem_ld_wait();
          tmem_st_wait();
          arrive_warp(&hdr->p_half[s], lane);
          tmem_ld32(t_s + 96, x);
          weights(y, 32);
          tmem_ld_wait();
          weights(x, 48);
          l += (lo_of(sum2[0]) + hi_of(sum2[0])) + (lo_of(sum2[1]) + hi_of(sum2[1]));
          tmem_st_wait();
        } else {
          arrive_warp(&hdr->p_half[s], lane);
        }
        arrive_warp(&hdr->p_full[s], lane);
      }

      // ------------------------------------------------------------ the piece's rows
      float* slot = nullptr;
      if (!w.whole()) slot = p.partials + static_cast<size_t>(2 * cta + (w.kt0 > 0 ? 0 : 1)) * chunk_slot_floats(DH);
      const int row = (pair ? s * tile_tok : 0) * G + r;     // packed row of the unit
      const long long out_at = valid ? (static_cast<long long>(w.row0) + w.tok0 + tok) * p.ldo + (w.kvh * G + r_head) * DH : -1;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
      // pair mode: all columns of the stream's own rows. Split mode: the streams hold
      // the same rows over alternate pages; each joins half of the columns.
      const bool both = !pair && w.count(1) > 0;
      float f0 = 1.f, f1 = 0.f;
      if (!pair) {
        // The first barrier also tells that the other stream is in this piece,
        // so that its o_full is waited for in the right phase.
        hdr->row_max[s][r] = m;
        hdr->row_sum[s][r] = l;
        named_bar(1, 256);
        const float m0 = hdr->row_max[0][r], m1 = hdr->row_max[1][r];
        m = fmaxf(m0, m1);
        const float ref = m == -INFINITY ? 0.f : m;
        f0 = ex2(m0 - ref);
        f1 = ex2(m1 - ref);
        l = hdr->row_sum[0][r] * f0 + hdr->row_sum[1][r] * f1;
        ok = ok && softmax_wait_bar(&hdr->o_full[0], pieces[0] & 1, hdr, status);
      }
      if (pair ? ns > 0 : both) ok = ok && softmax_wait_bar(&hdr->o_full[pair ? s : 1], pieces[pair ? s : 1] & 1, hdr, status);
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int c0 = pair ? 0 : s * (DH / 2), c1 = pair ? DH : c0 + DH / 2;
      const uint32_t t_o = tmem + lanes + kOCol + (pair ? s * DH : 0);
      if (slot != nullptr && valid && c0 == 0)
        reinterpret_cast<float2*>(slot + static_cast<size_t>(kChunkRows) * DH)[row] = make_float2(m, l);
      long long rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xffffffffu, out_at, (lane & 28) | i);
#pragma unroll 1
      for (int c = c0; c < c1 && ok && live; c += 32) {
        float o[32];
        tmem_ld32(t_o + c, o);
        tmem_ld_wait();
        if (!pair) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f0;
        }
        if (both) {
          float e[32];
          tmem_ld32(t_o + DH + c, e);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(e[i], f1, o[i]);
        }
        if (slot == nullptr) {
          store_rows32(out + c, rows, o, inv, lane);
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(slot + partial_at<DH>(row, c / 4 + i)) =
                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      tc_fence_before();
      if (!pair) named_bar(1, 256);   // both streams' O and statistics are read: the next piece may overwrite them
      g0 += 2 * w.nt;
      tiles += ns;
      pieces[0] += w.count(0) > 0 ? 1 : 0;
      pieces[1] += w.count(1) > 0 ? 1 : 0;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DH>
cudaError_t launch_tc(const ChunkArgs& a, const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, int ctas,
                      cudaStream_t s, bool pdl) {
  constexpr int smem = static_cast<int>((2 + kStages) * static_cast<size_t>(DH / 64) * kSubTile + sizeof(ChunkSmem));
  static_assert(smem <= 232448, "shared memory of a CTA");
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!done[dev & 63]) {
    const cudaError_t e = cudaFuncSetAttribute(chunk_tc_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    done[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, chunk_tc_kernel<DH>, qm, km, vm, a);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkArgs& a, int* ctas, cudaStream_t s, bool pdl) {
  const int G = a.n_q_heads / a.n_kv_heads;
  const uint64_t slabs = static_cast<uint64_t>(a.n_layers) * a.pages.n_pages * a.n_kv_heads;
  CUtensorMap qm, km, vm;
  if (!make_rows_map(&qm, a.q, a.head_dim, a.n_q_heads, a.T, a.ldq, G, 128 / G) ||
      !make_operand_map(&km, a.k_pool, 2, a.head_dim, kPageKeys, slabs, kKeys) ||
      !make_operand_map(&vm, a.v_pool, 2, a.head_dim, kPageKeys, slabs, kKeys))
    return cudaErrorInvalidValue;
  const int sms = num_sms_of_current_device();
  *ctas = sms < kChunkMaxCtas ? sms : kChunkMaxCtas;
  return a.head_dim == 128 ? launch_tc<128>(a, qm, km, vm, *ctas, s, pdl) : launch_tc<64>(a, qm, km, vm, *ctas, s, pdl);
}

}  // namespace dfl
