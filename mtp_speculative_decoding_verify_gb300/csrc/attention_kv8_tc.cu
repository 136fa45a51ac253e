// Verify attention of bf16 rows over the 8-bit cache on the 5th-generation
// tensor cores.
//
// out = softmax(scale Q K^T) V over the slots each row sees; work is shared
// out and joined as in attention_window_mma.cu: every CTA takes an equal
// number of pages of one KV head's line, crossing from request to request.
//
// Both products run on the bytes as TMA brought them (kind::f8f6f4, fp32
// sums). The other operand is split into e4m3 terms, 4 bits each:
//   S = Q K^T   a row of Q is scaled by a power of two (largest value in
//               [2^7, 2^8)) and q = hi + lo holds bf16's 8 bits. What lo
//               cannot hold (up to 2^-17 of the row's largest value) goes
//               into a third e5m2 term, used only for requests with a row
//               where these rests pass 2^-19 of the row's sum.
//   O += P V    p = hi + lo / 16: 8 bits, as bf16 would keep (the rounding of
//               the other bf16 kernels; rms error of an output 1.7e-3, of which
//               its own rounding to bf16 makes 1.66e-3).
// No operand is converted in shared memory, whose bandwidth is what two
// products with f16 values of V run out of (32 requests x 48 rows, 4096
// tokens: 112 us with V converted to f16, 68 us with the first form of this).
//
// M = 128 TMEM lanes. Lanes 32 w .. 32 w + 15, of warp w, hold a block of 16
// query rows as hi, lanes 32 w + 16 .. the same rows as lo: one MMA gives
// both terms, added after they are read. With fewer than 64 rows several
// warps hold the same block (row block w % NRB, key group w / NRB) and each
// takes its own keys of the tile: P is zero outside a warp's own keys, so every
// row of every warp is an online softmax of its own, and warps exchange
// nothing until the request ends. The 16x32bx2 form of the TMEM loads and
// stores gives the threads t and t + 16 of a warp two column ranges of one
// lane: they share a row and halve its keys and output dims, with a shuffle
// for the common maximum.
//
// A row's probabilities are 2^(score + log2(v scale) - ref): the block's
// scale of V rides along, and the sum, which is kept relative to a maximum of
// scores alone, divides it out again. e4m3 holds 2^-9 (lo: 2^-13) to 2^8, so
// ref follows the tiles up and down: when a tile's largest probability would
// pass 2^8, or those of three of the row's tiles in turn were below 2^-4, O is
// rescaled in TMEM. (Down, so that a few large scores do not cost the rest of
// the context its bits; O in fp32 has room for the 60 octaves that are
// allowed.)
//
// Two groups of four softmax warps share the work, each with an O of its own
// (joined with the rest when the request ends); P lies in the columns of the S
// it came from. Up to 32 rows they take alternate tiles, each with its own S
// buffer, so that one computes while the other waits for its products. With
// more rows the softmax is the longer part: there each takes a page of every
// tile, and both S buffers serve the two of them, so that the next S is there
// before this softmax ends (64 requests x 48 rows, 4096 tokens: 161 us with
// alternate tiles, 137 us with pages; 16 rows, 1k-32k: 3 % more with pages).
//
// Hidden slots: only tiles with a slot that not every row sees are masked.
// There V's bytes that are NaN become 0 in shared memory (0 x NaN), and a
// bitmap of (verify token, dim) puts NaN back into the rows that do see them.
//
// Bound: the read of the cache (it holds at 16 rows: 343 us for 64 requests of
// 1k-32k tokens, 95 % of the copy rate). At 48 rows the chain of a tile is
// longer than its read (P V, then S of the tile that takes its buffer, and a
// softmax of some 1500 cycles): 137 us for 64 requests of 4096 tokens, 59 %.
// More than 64 rows read all pages again for each 64 (120 rows, 32 requests of
// 4096 tokens: 145 us, 64 rows 84 us).
//
// Warps: 0 and 1 P V, 2 TMA (block ids and scales of 32 pages at a time, one a
// lane), 3 S, 4-11 softmax and output, 12-15 masked V and the next request's
// Q. (One polling warp for all products was the slowest part of a tile.)
#include <cuda.h>
#include <cudaTypedefs.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "attention_window.h"
#include "kv8.cuh"
#include "sm100.cuh"

namespace mtp {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 512;
constexpr int kKeys = 128;
constexpr int kInfo = 8;               // tiles whose scales and pages are held: the TMA warp is at most 6 stages and 2 S buffers ahead
constexpr int kSegs = 4;               // requests whose row factors are held; the Q warps are at most 3 ahead
constexpr int kNanSegs = 8;            // requests whose NaN bitmaps are held; their writers are at most 6 stages ahead
constexpr int kSegRing = 16;           // requests announced; the TMA warp is at most 6 stages, 2 S and 1 ahead
// log2 of a tile's largest probability: the bounds that ref keeps, where the first tile puts it, and where a rescale
// up and one down do. Twelve octaves apart, and the landings leave room for what comes: tiles whose maxima alternate
// over up to nine octaves (blocks of different scales) settle after a move or two.
constexpr float kMostP = 8.0f, kLeastP = -4.0f, kFirstP = 1.0f, kUpP = 5.0f, kDownP = -1.0f;
constexpr int kLowTiles = 3;
constexpr float kDown = 60.0f;         // ref is never further below the largest there was
// A probability is never held further below what it adds to the row's sum (2^(score - the sum's maximum, at most 2^20))
// than this: fp32 has 126 octaves below 1, so weights down to 2^-66 of the largest count, and one so far below rounds
// to 0 in e4m3 as it did before.
constexpr float kFarBack = 60.0f;
constexpr float kLoScale = 16.0f;      // P's second term is held times this
constexpr uint32_t kColO = 256;        // S (and P) buffers at columns 0 and 128, O at 256 and 384

template <int D>
struct Smem {
  static constexpr int kTile = kKeys * D;                 // bytes of K or V of a tile
  // V is held longer (to P V, two tiles behind S). Its stages are even: where the groups take alternate tiles, a stage
  // then serves one of them only, whose P V warp meets its phases one after the other (a wait's parity tells only two
  // apart).
  static constexpr int kKStages = D == 128 ? 4 : 6, kVStages = 6;
  static constexpr int kK = 0, kV = kK + kKStages * kTile;
  static constexpr int kQ = kV + kVStages * kTile;         // hi and lo, rest
  static constexpr int kX = kQ + 2 * kTile;               // join of a row's partial results: [8 warps][16][36] floats
  static constexpr int kRed = kX + 128 * 36 * 4;          // [8 warps][16] (maximum, sum)
  static constexpr int kInfoOff = kRed + 128 * 8;         // [kInfo] TileInfo
  static constexpr int kRing = kInfoOff + kInfo * 32;     // [kSegRing] Seg
  static constexpr int kFac = kRing + kSegRing * 32;      // [kSegs][64] factors of the rows' scores
  static constexpr int kNan = kFac + kSegs * 64 * 4;      // [kNanSegs][16][4] words
  static constexpr int kBar = kNan + kNanSegs * 16 * 4 * 4;
  static constexpr int kBars = 2 * kKStages + 3 * kVStages + 2 + 2 + 4 + 4 + kInfo + kSegs + kSegRing;
  static constexpr int kMisc = kBar + kBars * 8;          // rest flags [kSegs], join flag, abort, TMEM base
  static constexpr int kBytes = kMisc + kSegs * 4 + 16 + 1024;
  // byte offset of 16-byte chunk c of row r of a K-major operand tile, as TMA swizzles it
  __device__ __forceinline__ static uint32_t at(int r, int c) {
    if constexpr (D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * 128 + ((c ^ (r & 7)) << 4);
  }
};
static_assert(Smem<128>::kBytes <= 232448 && Smem<64>::kBytes <= 232448, "227 KB of shared memory");

struct alignas(16) PageInfo {
  float sk, lsv;             // scale of K, log2 of the scale of V
  int mark;                  // the page's index in the request; -2 - index: some row does not see all of it; -1: not loaded
};
struct TileInfo {
  PageInfo page[2];
};

// ------------------------------------------------------------- instructions
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// (a, b) += (c, d) and (a, b) = (a, b) f + g as one instruction each.
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n  .reg .b64 p, q;\n  mov.b64 p, {%0, %1};\n  mov.b64 q, {%2, %3};\n  add.rn.f32x2 p, p, q;\n  mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void fma2(float& a, float& b, float f, float g) {
  asm("{\n  .reg .b64 p, q, r;\n  mov.b64 p, {%0, %1};\n  mov.b64 q, {%2, %2};\n  mov.b64 r, {%3, %3};\n"
      "  fma.rn.f32x2 p, p, q, r;\n  mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(f), "f"(g));
}

// Four probabilities (at most 2^8) as e4m3 terms: hi, and lo = 16 (p - hi).
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo) {
  asm("{\n"
      "  .reg .b16 h0, h1, l0, l1;\n"
      "  .reg .b32 p0, p1, q0, q1, m, s;\n"
      "  mov.b32 m, 0xcc00cc00;\n"                        // f16 -16, -16
      "  mov.b32 s, 0x4c004c00;\n"                        // f16 16, 16
      "  cvt.rn.f16x2.f32 p0, %3, %2;\n"
      "  cvt.rn.f16x2.f32 p1, %5, %4;\n"
      "  cvt.rn.satfinite.e4m3x2.f16x2 h0, p0;\n"
      "  cvt.rn.satfinite.e4m3x2.f16x2 h1, p1;\n"
      "  cvt.rn.f16x2.e4m3x2 q0, h0;\n"
      "  cvt.rn.f16x2.e4m3x2 q1, h1;\n"
      "  mul.rn.f16x2 p0, p0, s;\n"
      "  mul.rn.f16x2 p1, p1, s;\n"
      "  fma.rn.f16x2 p0, q0, m, p0;\n"
      "  fma.rn.f16x2 p1, q1, m, p1;\n"
      "  cvt.rn.satfinite.e4m3x2.f16x2 l0, p0;\n"
      "  cvt.rn.satfinite.e4m3x2.f16x2 l1, p1;\n"
      "  mov.b32 %0, {h0, h1};\n"
      "  mov.b32 %1, {l0, l1};\n"
      "}\n"
      : "=r"(hi), "=r"(lo)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}

// Named barrier over `count` threads; true if all of them passed true. What
// decides whether a group of warps that meet at barriers goes on.
template <int kId, int kCount>
__device__ __forceinline__ bool barrier_all(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbar.red.and.pred po, %2, %3, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kId), "n"(kCount)
      : "memory");
  return r != 0;
}

// D[tmem] (+)= A[smem] x B[smem]^T of 8-bit operands, K = 32.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A from TMEM, four bytes a column.
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// TMEM lanes 0-15 of the warp's quarter: threads t < 16 get lane t's columns
// col.., threads t >= 16 lane t - 16's columns col + HALF...
template <int N, int HALF>
__device__ __forceinline__ void ld_halves(uint32_t addr, float* v) {
  uint32_t r[32];
  static_assert(N == 8 || N == 16 || N == 32, "columns");
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], %9;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr), "n"(HALF));
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16], %17;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr), "n"(HALF));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32], %33;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr), "n"(HALF));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N, int HALF>
__device__ __forceinline__ void st_halves(uint32_t addr, const uint32_t* r) {
  static_assert(N == 2 || N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 2) {
    asm volatile("tcgen05.st.sync.aligned.16x32bx2.x2.b32 [%0], %1, {%2, %3};" ::"r"(addr), "n"(HALF), "r"(r[0]), "r"(r[1])
                 : "memory");
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.st.sync.aligned.16x32bx2.x4.b32 [%0], %1, {%2, %3, %4, %5};" ::"r"(addr), "n"(HALF), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], %1, {%2, %3, %4, %5, %6, %7, %8, %9};" ::"r"(addr), "n"(HALF),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, "
        "{%2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17};" ::"r"(addr),
        "n"(HALF), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  }
}

// K-major operand tile of D-byte rows as TMA swizzles it (128 or 64 bytes).
template <int D>
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(8 * D >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)(D == 128 ? 2 : 4) << 61;
}

// The V tile as MN-major operand: D dims of a key are one swizzle row, eight
// keys a group.
template <int D>
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t addr) {
  return desc_kmajor<D>(addr);
}

// --------------------------------------------------------------- work shares
// The part of a request that this CTA does: pages i0 .. i1-1 of its n, the
// first of which is page p0 of the line; n = 0 ends the work.
struct Seg {
  int b, i0, i1, n, ctx;
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == n; }
  __device__ __forceinline__ int tiles() const { return (i1 - i0 + 1) / 2; }
};

// Walks the segments of pages [pos, end) in order, from a place in request b
// (pages p0 .. p1 - 1, context ctx) on.
struct Walk {
  const WindowParams& p;
  int pos, end, p0, p1, b, ctx;
  __device__ __forceinline__ bool next(Seg& s) {
    if (pos >= end) return false;
    while (p1 <= pos) {
      ++b;
      ctx = __ldg(p.ctx_lens + b);
      p0 = p1;
      p1 = __ldcg(p.prefix + b + 1);
    }
    s.b = b;
    s.ctx = ctx;
    s.i0 = pos - p0;
    s.i1 = min(end, p1) - p0;
    s.n = p1 - p0;
    pos = p0 + s.i1;
    return true;
  }
};

// Every row sees the whole page.
__device__ __forceinline__ bool page_whole(const WindowParams& p, int page, int ctx) {
  const int first = page * kBlock, last = first + kBlock - 1;
  return last <= ctx && (p.window == 0 || first > ctx + p.R - 1 - p.window || last < p.sinks);
}

// Four bytes of V of a tile with hidden slots: a NaN becomes 0, and its dim's
// bit is set in the row of every verify token that sees the slot (rare).
__device__ __forceinline__ uint32_t hide_nan(const WindowParams& p, uint32_t w, int slot, int ctx, uint32_t* row_bits, int bit) {
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // 0x80 where a byte is 0x7f or 0xff
  if (nan != 0) {
    for (int e = 0; e < 4; ++e) {
      if (!((nan >> (8 * e + 7)) & 1)) continue;
      w &= ~(0xffu << (8 * e));
      for (int j = 0; j < p.R; ++j)
        if (slot_visible(slot, ctx + j, p.window, p.sinks)) atomicOr(row_bits + j * 4, 1u << (bit + e));
    }
  }
  return w;
}

// Where CTA gg of a KV head leaves its part of a request: slot 0 for one it
// did not begin, slot 1 for one it began. [rows][D] values, divided by their
// sum (so that V's largest values stay finite), then (maximum, sum) of each
// row.
template <int D, int NRB>
__device__ __forceinline__ float* part_slot(const WindowParams& p, int gg, int which, int kvh, int row_tile) {
  return p.part_o + ((((size_t)gg * 2 + which) * p.Hkv + kvh) * p.row_tiles + row_tile) * ((size_t)NRB * 16 * (D + 2));
}

// Join the parts of a request, in the order of the CTAs. Thread t of n.
template <int D, int NRB>
__device__ void join_parts(const WindowParams& p, const Seg& seg, int2 in, int kvh, int row_tile, int t, int n) {
  const int g0 = in.x, g1 = in.y;
  const int first_row = row_tile * 64, n_rows = min(NRB * 16, p.rows - first_row);
  const int64_t out0 = (int64_t)seg.b * p.R * p.Hq + kvh * p.group;
  for (int u = t; u < n_rows * (D / 4); u += n) {
    const int local = u / (D / 4), dim = u % (D / 4) * 4;
    float m = -INFINITY, l = 0.0f;                             // maximum, sum and mean of the parts so far
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int gg = g0; gg <= g1; ++gg) {
      const float* from = part_slot<D, NRB>(p, gg, gg == g0, kvh, row_tile);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(from + NRB * 16 * D) + local);
      const float4 o4 = __ldcg(reinterpret_cast<const float4*>(from + (size_t)local * D + dim));
      const float top = fmaxf(m, ml.x);                        // (-inf: nothing seen, and sums of 0 or NaN)
      const float a = m == top ? l : l * ex2(m - top), b = ml.x == top ? ml.y : ml.y * ex2(ml.x - top);
      m = top;
      l = a + b;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l, ca = a * inv, cb = b * inv;
      v.x = v.x * ca + o4.x * cb, v.y = v.y * ca + o4.y * cb, v.z = v.z * ca + o4.z * cb, v.w = v.w * ca + o4.w * cb;
    }
    const int row = first_row + local;
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + (out0 + (int64_t)(row / p.group) * p.Hq + row % p.group) * D + dim;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

// NRB: blocks of 16 query rows (1, 2, 4).
template <int D, int NRB>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const WindowParams p) {
  using S = Smem<D>;
  constexpr int kKStages = S::kKStages, kVStages = S::kVStages;
  constexpr int KG = 4 / NRB;            // key groups: warps that share a row block
  constexpr bool kPages = NRB == 4;      // the groups take pages instead of tiles
  constexpr int NK = kPages ? 32 : 16 * NRB;        // keys of a tile that a thread takes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* xbuf = reinterpret_cast<float*>(smem + S::kX);
  float2* red = reinterpret_cast<float2*>(smem + S::kRed);
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + S::kInfoOff);
  float* fac = reinterpret_cast<float*>(smem + S::kFac);
  uint32_t* nanmap = reinterpret_cast<uint32_t*>(smem + S::kNan);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint64_t* k_empty = k_full + kKStages;
  uint64_t* v_full = k_empty + kKStages;
  uint64_t* v_ready = v_full + kVStages;  // masked bytes have been dealt with
  uint64_t* v_empty = v_ready + kVStages;
  uint64_t* q_full = v_empty + kVStages;  // Q of the next request is in place
  uint64_t* q_empty = q_full + 1;        // the last S of a request is done
  // Of tile g, in buffer g % 2 (pages: of each group, at 2 group + g % 2):
  uint64_t* s_full = q_full + 2;         // S is there, and so O of tile g - 2
  uint64_t* p_full = s_full + 2;         // P has replaced S
  uint64_t* pv_done = p_full + 4;        // O holds the tile
  uint64_t* info_full = pv_done + 4;     // [kInfo]
  uint64_t* fac_full = info_full + kInfo;   // [kSegs]
  uint64_t* seg_full = fac_full + kSegs;    // [kSegRing]
  Seg* ring = reinterpret_cast<Seg*>(smem + S::kRing);
  volatile int* rest = reinterpret_cast<volatile int*>(smem + S::kMisc);   // [kSegs] the third term of Q is needed
  volatile int* last_flag = rest + kSegs;
  volatile int* abort = last_flag + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc + kSegs * 4 + 8);

  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int heads = p.Hkv * p.row_tiles;
  const int kvh = blockIdx.x % heads / p.row_tiles, row_tile = blockIdx.x % heads % p.row_tiles;
  const int g_cta = blockIdx.x / heads;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKStages; ++s) {
      sm100::mbar_init(&k_full[s], 1);
      sm100::mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      sm100::mbar_init(&v_full[s], 1);
      sm100::mbar_init(&v_ready[s], 4);
      sm100::mbar_init(&v_empty[s], kPages ? 2 : 1);
    }
    sm100::mbar_init(q_full, 128);
    sm100::mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) sm100::mbar_init(&s_full[i], 1);
    for (int i = 0; i < 4; ++i) {
      sm100::mbar_init(&p_full[i], 4);
      sm100::mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kSegRing; ++i) sm100::mbar_init(&seg_full[i], 1);
    for (int i = 0; i < kInfo; ++i) sm100::mbar_init(&info_full[i], 1);
    for (int i = 0; i < kSegs; ++i) sm100::mbar_init(&fac_full[i], 128);
    *abort = 0;
    sm100::fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    sm100::tma_prefetch_desc(&tm_k);
    sm100::tma_prefetch_desc(&tm_v);
  }
  for (int i = threadIdx.x; i < kNanSegs * 16 * 4; i += kThreads) nanmap[i] = 0;
  for (int i = threadIdx.x; i < S::kTile / 16; i += kThreads)   // the rest term has no second one
    *reinterpret_cast<uint4*>(smem + S::kQ + S::kTile + i * 16) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  if (warp == 0) {
    sm100::tmem_alloc(tmem_slot, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Everything up to here may run while the append still does; what follows
  // reads what it writes (which the read-only path may not: __ldcg).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Share share = load_share(p.shares, g_cta);
  const int t_end = share_end(p.shares, g_cta);
  if (g_cta >= share_count(p.shares)) {
    __syncthreads();
    if (warp == 0) sm100::tmem_dealloc(tmem, 512);
    return;
  }
  const uint32_t sbase = sm100::smem_u32(smem);

  // Registers: 128 a thread at launch; the softmax warps take what the others
  // leave (104 + 2 x 152 + 104 = 4 x 128).
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {   // the whole warp
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort) ? 1 : 0) != 0;
  };
  // Segment sn, as the TMA warp announced it.
  auto take = [&](int sn, Seg& seg) -> bool {
    if (!wait(&seg_full[sn % kSegRing], (uint32_t)((sn / kSegRing) & 1))) return false;
    seg = ring[sn % kSegRing];
    return true;
  };
  bool ok = true;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    constexpr uint32_t kShape = (1u << 4) | ((uint32_t)(128 >> 4) << 24);   // fp32 D, M = 128
    // (In the warps that issue MMAs the whole warp walks the tiles, so that
    // the descriptors stay uniform; one elected lane issues.)
    if (warp < 2) {
      // --------------------------------------------------------------- P V
      // Of softmax group `warp`: its tiles, or its page of each.
      constexpr uint32_t idesc_pv = kShape | ((uint32_t)(D >> 3) << 17) | (1u << 16);   // V MN-major
      constexpr int kCount = kPages ? kBlock : kKeys;      // keys of a product
      const int wg = warp;
      const uint64_t vd0 = desc_mnmajor<D>(sbase + S::kV + (kPages ? wg * (S::kTile / 2) : 0));
      int g = 0, last_g = -1;
      Seg seg;
      for (int sn = 0; (ok = ok && take(sn, seg)) && seg.n != 0; ++sn) {
        const int tiles = seg.tiles();
        for (int i = 0; i < tiles; ++i, ++g) {
          const int buf = g & 1, stage = g % kVStages, bar = kPages ? wg * 2 + buf : wg;
          if (!kPages && buf != wg) continue;
          ok = wait(&p_full[bar], (uint32_t)((g >> 1) & 1)) && wait(&v_ready[stage], (uint32_t)((g / kVStages) & 1));
          if (!ok) break;
          last_g = g;
          sm100::tc_fence_after();
          if (sm100::elect_one()) {
            const uint64_t vd = vd0 + (uint64_t)(stage * (S::kTile >> 4));
            const uint32_t first = i < (kPages ? 1 : 2) ? 1u : 0u;   // it begins the group's O
#pragma unroll
            for (int kk = 0; kk < kCount / 32; ++kk)
              mma_f8_ts(tmem + kColO + wg * 128, tmem + buf * 128 + (kPages ? wg * 64 : 0) + kk * 8,
                        vd + (uint64_t)(kk * (32 * D >> 4)), idesc_pv, kk > 0 ? 1u : 1u - first);
            sm100::tc_commit(&pv_done[bar]);
            sm100::tc_commit(&v_empty[stage]);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        *abort = 1;
        if (lane == 0) raise_error(p.err, MTP_ERR_TIMEOUT);
        // MMAs in flight end before the shared memory and TMEM go (else the softmax warps have waited for every one)
        if (last_g >= 0)
          sm100::mbar_wait_timeout(&pv_done[kPages ? wg * 2 + (last_g & 1) : wg], (uint32_t)((last_g >> 1) & 1), sm100::kWaitTimeoutNs);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ----------------------------------------------------------------- S
      // Of each tile, as soon as its keys are there and P V of tile g - 2 (of
      // both groups' pages) has read P from the buffer.
      constexpr uint32_t idesc_qk = kShape | ((uint32_t)(kKeys >> 3) << 17);            // e4m3 x e4m3
      constexpr uint32_t idesc_rest = idesc_qk | (1u << 7);                             // e5m2 x e4m3
      const uint64_t qd = desc_kmajor<D>(sbase + S::kQ), kd0 = desc_kmajor<D>(sbase + S::kK);
      int g = 0;
      Seg seg;
      for (int sn = 0; (ok = ok && take(sn, seg)) && seg.n != 0; ++sn) {
        const int tiles = seg.tiles();
        if (!(ok = wait(q_full, (uint32_t)(sn & 1)))) break;
        const bool third = rest[sn % kSegs] != 0;
        for (int i = 0; i < tiles; ++i, ++g) {
          const int buf = g & 1, stage = g % kKStages;
          const uint32_t two_back = (uint32_t)(((g - 2) >> 1) & 1);
          ok = wait(&k_full[stage], (uint32_t)((g / kKStages) & 1)) &&
               (g < 2 || (wait(&pv_done[buf], two_back) && (!kPages || wait(&pv_done[2 + buf], two_back))));
          if (!ok) break;
          sm100::tc_fence_after();
          if (sm100::elect_one()) {
            const uint32_t d = tmem + buf * 128;
            const uint64_t kd = kd0 + (uint64_t)(stage * (S::kTile >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) mma_f8(d, qd + 2 * kk, kd + 2 * kk, idesc_qk, kk ? 1u : 0u);
            if (third) {
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) mma_f8(d, qd + (uint64_t)((S::kTile >> 4) + 2 * kk), kd + 2 * kk, idesc_rest, 1u);
            }
            sm100::tc_commit(&s_full[buf]);
            sm100::tc_commit(&k_empty[stage]);
            if (i + 1 == tiles) sm100::tc_commit(q_empty);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        *abort = 1;
        if (lane == 0) raise_error(p.err, MTP_ERR_TIMEOUT);
        if (g > 0) sm100::mbar_wait_timeout(&s_full[(g - 1) & 1], (uint32_t)(((g - 1) >> 1) & 1), sm100::kWaitTimeoutNs);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------------- TMA
      const uint64_t pol = sm100::l2_policy_evict_first();
      Walk walk{p, share.begin, t_end, share.p0, share.p0 + share.n, share.b, share.ctx};
      int g = 0;
      Seg seg;
      for (int sn = 0; ok; ++sn) {
        if (!walk.next(seg)) seg.n = 0;
        if (lane == 0) {
          ring[sn % kSegRing] = seg;
          sm100::mbar_arrive(&seg_full[sn % kSegRing]);
        }
        if (seg.n == 0) break;
        const PageSpan span = page_span(seg.ctx, p.R, p.window, p.sinks);
        for (int i = seg.i0; i < seg.i1 && ok; i += kWarp) {
          int blk = -1, page = -1;
          float sk = 1.0f, lsv = 0.0f;
          if (i + lane < seg.i1) {
            page = span.page(i + lane);
            blk = p.block_table[(int64_t)seg.b * p.max_blocks + page];
            if (blk < 0 || blk >= p.num_blocks) {
              raise_error(p.err, MTP_ERR_BLOCK_ID);
              page = -1;
            } else {
              sk = __ldcg(p.k_scale + (int64_t)blk * p.Hkv + kvh);
              const float sv = __ldcg(p.v_scale + (int64_t)blk * p.Hkv + kvh);
              if (!scale_ok(sk) || !scale_ok(sv)) {
                raise_error(p.err, MTP_ERR_SCALE);
                page = -1;
                sk = 1.0f;
              } else {
                lsv = log2f(sv);
                if (!page_whole(p, page, seg.ctx)) page = -2 - page;
              }
            }
          }
          const int n = min(kWarp, seg.i1 - i);
          for (int x = 0; x < n; x += 2, ++g) {
            TileInfo in;
            int id[2];
  #pragma unroll
            for (int y = 0; y < 2; ++y) {        // (lane 31 of an odd rest has page -1)
              id[y] = __shfl_sync(0xffffffffu, blk, x + y);
              in.page[y].mark = __shfl_sync(0xffffffffu, page, x + y);
              in.page[y].sk = __shfl_sync(0xffffffffu, sk, x + y);
              in.page[y].lsv = __shfl_sync(0xffffffffu, lsv, x + y);
            }
            int go = 1;
            if (lane == 0) {
              const int s = g % kKStages, vs = g % kVStages;
              const uint32_t bytes = ((in.page[0].mark != -1) + (in.page[1].mark != -1)) * (uint32_t)(S::kTile / 2);
              go = sm100::mbar_wait(&k_empty[s], (uint32_t)((g / kKStages) & 1) ^ 1u, abort);
              if (go) {
                info[g % kInfo] = in;
                sm100::mbar_arrive(&info_full[g % kInfo]);
                if (bytes) sm100::mbar_arrive_expect_tx(&k_full[s], bytes);
                else sm100::mbar_arrive(&k_full[s]);
  #pragma unroll
                for (int y = 0; y < 2; ++y)
                  if (in.page[y].mark != -1)
                    sm100::tma_load_4d(smem + S::kK + s * S::kTile + y * (S::kTile / 2), &tm_k, &k_full[s], 0, kvh, 0, id[y], pol);
                go = sm100::mbar_wait(&v_empty[vs], (uint32_t)((g / kVStages) & 1) ^ 1u, abort);
              }
              if (go) {
                if (bytes) sm100::mbar_arrive_expect_tx(&v_full[vs], bytes);
                else sm100::mbar_arrive(&v_full[vs]);
  #pragma unroll
                for (int y = 0; y < 2; ++y)
                  if (in.page[y].mark != -1)
                    sm100::tma_load_4d(smem + S::kV + vs * S::kTile + y * (S::kTile / 2), &tm_v, &v_full[vs], 0, kvh, 0, id[y], pol);
              } else {
                *abort = 1;
                raise_error(p.err, MTP_ERR_TIMEOUT);
              }
            }
            ok = __shfl_sync(0xffffffffu, go, 0) != 0;
            if (!ok) break;
          }
        }
      }
      // Every copy issued lands before the CTA may exit: the last fill of each
      // stage (after a timeout the K copy of tile g may be on its way too; each
      // wait is bounded).
      if (lane == 0) {
        const int nk = ok ? g : g + 1;
        for (int x = max(0, nk - kKStages); x < nk; ++x)
          sm100::mbar_wait_timeout(&k_full[x % kKStages], (uint32_t)((x / kKStages) & 1), ok ? sm100::kWaitTimeoutNs : 1000000);
        for (int x = max(0, g - kVStages); x < g; ++x)
          sm100::mbar_wait_timeout(&v_full[x % kVStages], (uint32_t)((x / kVStages) & 1), ok ? sm100::kWaitTimeoutNs : 1000000);
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    // -------------------------------------------------- softmax and output
    const int w = warp & 3, wg = (warp >> 2) - 1, st = threadIdx.x - 128;
    const int rb = w % NRB, kg = w / NRB, half = lane >> 4, r16 = lane & 15;
    const int page_half = kPages ? wg : (kg * 2 + half) * NK / kBlock, in_page = (kg * 2 + half) * NK % kBlock;   // its keys
    const int row = row_tile * 64 + rb * 16 + r16;
    const int j = min(row, p.rows - 1) / p.group;
    const uint32_t quarter = tmem + ((uint32_t)(32 * w) << 16);
    const uint32_t o_hi = quarter + kColO + wg * 128, o_lo = o_hi + (16u << 16);
    auto soft_sync = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    int g = 0;
    Seg seg;
    for (int sn = 0; (ok = barrier_all<1, 256>(ok && take(sn, seg))) && seg.n != 0; ++sn) {
      const int tiles = seg.tiles(), pos = seg.ctx + j;
      const int low = p.window == 0 ? 0 : pos - p.window + 1;
      ok = ok && __all_sync(0xffffffffu, sm100::mbar_wait(&fac_full[sn % kSegs], (uint32_t)((sn / kSegs) & 1), abort) ? 1 : 0);
      const float row_fac = fac[(sn % kSegs) * 64 + rb * 16 + r16];
      float ref = -INFINITY, top_ref = -INFINITY;          // of the probabilities; the largest it was
      float lref = -INFINITY, sum = 0.0f;                  // maximum of the scores (lazy), sum relative to it
      int low_tiles = 0;                                   // in a row, with a small largest probability
      bool begun = false;                                  // O holds something
      const int g_end = g + tiles;
      for (g += kPages ? 0 : (g ^ wg) & 1; g < g_end; g += kPages ? 1 : 2) {   // this group's tiles
        const int buf = g & 1;                             // (its own buffer where it takes tiles)
        const uint32_t s_hi = quarter + buf * 128 + (kPages ? wg * 64 : 0), s_lo = s_hi + (16u << 16);
        ok = ok && wait(&info_full[g % kInfo], (uint32_t)((g / kInfo) & 1)) && wait(&s_full[buf], (uint32_t)((g >> 1) & 1));
        if (!ok) break;                                    // the segment's end still meets the others
        sm100::tc_fence_after();
        const PageInfo in = info[g % kInfo].page[page_half];
        float x[NK];
        {
          float y[NK];
          ld_halves<NK, NK>(s_hi + kg * 2 * NK, x);
          ld_halves<NK, NK>(s_lo + kg * 2 * NK, y);
          sm100::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < NK; k += 2) add2(x[k], x[k + 1], y[k], y[k + 1]);
        }
        const int mark = in.mark;
        if (mark < 0) {
          const int slot = (-2 - mark) * kBlock + in_page, top = mark == -1 ? INT_MIN : pos;
#pragma unroll
          for (int k = 0; k < NK; ++k)
            if (!(slot + k <= top && (slot + k >= low || slot + k < p.sinks))) x[k] = -INFINITY;
        }
        // (a factor of 0 would turn a hidden -inf into NaN; scores that small are 0 all the same)
        const float f = fmaxf(row_fac * in.sk, 1e-36f);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < NK; ++k) mx[k & 3] = fmaxf(mx[k & 3], x[k]);
        const float score = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
        float most = score + in.lsv, highest = score;
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));   // with the row's other half
        highest = fmaxf(highest, __shfl_xor_sync(0xffffffffu, highest, 16));
        if (highest > lref + 20.0f) {
          sum *= lref == -INFINITY ? 0.0f : ex2(lref - highest);
          lref = highest;
        }
        // (a row with nothing visible in the tile stays as it is)
        const float to = fmaxf(most - (ref == -INFINITY ? kFirstP : most > ref ? kUpP : kDownP), top_ref - kDown);
        low_tiles = most < ref + kLeastP && most != -INFINITY ? low_tiles + 1 : 0;
        const bool move = most > ref + kMostP || (low_tiles >= kLowTiles && to < ref - 1.0f);
        if (__any_sync(0xffffffffu, move)) {
          const float c = !move ? 1.0f : ref == -INFINITY ? 0.0f : ex2(ref - to);
          if (move) ref = to;
          top_ref = fmaxf(top_ref, ref);
          if (begun) {
            if (kPages) {                                  // (else S of tile g came after the group's last P V)
              ok = wait(&pv_done[wg * 2 + (buf ^ 1)], (uint32_t)(((g - 1) >> 1) & 1));
              if (!ok) break;
              sm100::tc_fence_after();
            }
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {               // this thread's half of the row's dims, 16 at a time
              float o[16], o2[16];
              ld_halves<16, D / 2>(o_hi + q * 16, o);
              ld_halves<16, D / 2>(o_lo + q * 16, o2);
              sm100::tmem_ld_wait();
              uint32_t r[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(o[k] * c);
              st_halves<16, D / 2>(o_hi + q * 16, r);
#pragma unroll
              for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(o2[k] * c);
              st_halves<16, D / 2>(o_lo + q * 16, r);
            }
          }
        }
        // The sum is of 2^(score - lref): 2^back times the probabilities, without V's scale. Where this page's scale
        // is far below what ref follows (zeros of V have 2^-100) both would leave fp32's range, hence the bound.
        const float lr = lref == -INFINITY ? 0.0f : lref;    // (nothing visible yet: a sum of 0, or NaN from K)
        const float shift = fmaxf(in.lsv - (ref == -INFINITY ? 0.0f : ref), -kFarBack - lr), back = -shift - lr;
        float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t hi[NK / 4], lo[NK / 4];
#pragma unroll
        for (int k = 0; k < NK; k += 4) {
          fma2(x[k], x[k + 1], f, shift);
          fma2(x[k + 2], x[k + 3], f, shift);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[k + e] = ex2(x[k + e]);
          add2(add[0], add[1], x[k], x[k + 1]);
          add2(add[2], add[3], x[k + 2], x[k + 3]);
          split4(x[k], x[k + 1], x[k + 2], x[k + 3], hi[k / 4], lo[k / 4]);
        }
        sum += ((add[0] + add[1]) + (add[2] + add[3])) * ex2(back);
        if constexpr (KG > 1) {                            // columns of the other warps' keys
          const uint32_t z[NK / 4] = {};
#pragma unroll
          for (int y = 1; y < KG; ++y) {
            const int other = (kg + y) % KG * (NK / 2);
            st_halves<NK / 4, NK / 4>(s_hi + other, z);
            st_halves<NK / 4, NK / 4>(s_lo + other, z);
          }
        }
        st_halves<NK / 4, NK / 4>(s_hi + kg * (NK / 2), hi);
        st_halves<NK / 4, NK / 4>(s_lo + kg * (NK / 2), lo);
        tmem_st_wait();
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&p_full[kPages ? wg * 2 + buf : wg]);
        begun = true;
      }
      // ---- the request's part is done: join the lanes of each row
      g = g_end;
      const int last_g = kPages ? g - 1 : g - 1 - ((g - 1 - wg) & 1);   // this group's last tile so far
      ok = ok && (!begun || wait(&pv_done[kPages ? wg * 2 + (last_g & 1) : wg], (uint32_t)((last_g >> 1) & 1)));
      sm100::tc_fence_after();
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (half == 0) red[(wg * 4 + w) * 16 + r16] = make_float2(lref, sum);
      soft_sync();
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int y = 0; y < 2 * KG; ++y) M = fmaxf(M, red[((y / KG) * 4 + rb + NRB * (y % KG)) * 16 + r16].x);
#pragma unroll
      for (int y = 0; y < 2 * KG; ++y) {
        const float2 v = red[((y / KG) * 4 + rb + NRB * (y % KG)) * 16 + r16];
        L += v.y * (v.x == -INFINITY ? 1.0f : ex2(v.x - M));   // (nothing seen: 0, or NaN from K)
      }
      const bool whole = seg.whole();
      const int2 in = whole ? make_int2(0, 0) : __ldcg(p.sharers + seg.b);
      // (two factors: V's scale is in the second, and their product may leave fp32's range where a result does not)
      const float inv = L == 0.0f ? 0.0f : 1.0f / L, own = ex2(ref - M);
      const float poison = sum != sum ? sum : 0.0f;            // NaN in K: every dim of the row
      const int first_row = row_tile * 64, n_rows = min(NRB * 16, p.rows - first_row);
      const int64_t out0 = (int64_t)seg.b * p.R * p.Hq + kvh * p.group;
      float* part = whole ? nullptr : part_slot<D, NRB>(p, g_cta, seg.i0 > 0 ? 0 : 1, kvh, row_tile);
      if (!whole && wg == 0 && kg == 0 && half == 0) reinterpret_cast<float2*>(part + (size_t)NRB * 16 * D)[rb * 16 + r16] = make_float2(M, L);
      auto out_row = [&](int local) {
        const int rr = first_row + local;
        return static_cast<__nv_bfloat16*>(p.out) + (out0 + (int64_t)(rr / p.group) * p.Hq + rr % p.group) * D;
      };
      // 16 of the thread's output dims, from dim0 on, with its weight
      auto get = [&](int c, float (&y)[16]) {
        float y2[16];
        if (ok) {
          ld_halves<16, D / 2>(o_hi + c * 16, y);
          ld_halves<16, D / 2>(o_lo + c * 16, y2);
          sm100::tmem_ld_wait();
        }
        const int dim0 = half * (D / 2) + c * 16;
        const uint32_t bits = nanmap[((sn % kNanSegs) * 16 + j) * 4 + (dim0 >> 5)] >> (dim0 & 31) & 0xffffu;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          // (nothing seen: the lane's O may be anything, so it takes no part)
          y[k] = ref == -INFINITY || !ok ? 0.0f : fmaf(y2[k], 1.0f / kLoScale, y[k]) * inv * own;
        }
        if (__any_sync(0xffffffffu, bits != 0 || poison != 0.0f)) {
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] += ((bits >> k) & 1) ? NAN : poison;
        }
      };
      // four dims of a row whose output starts at `to`
      auto put = [&](int local, __nv_bfloat16* to, int dim, const float4& v) {
        if (local >= n_rows) return;
        if (whole) *reinterpret_cast<uint2*>(to + dim) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else *reinterpret_cast<float4*>(part + (size_t)local * D + dim) = v;
      };
      if constexpr (KG == 1) {
        // A row is in two warps, one of each group: they swap halves of its
        // dims, 16 a thread and step, each thread for its counterpart's.
        const int local = rb * 16 + r16;
        __nv_bfloat16* to = out_row(min(local, n_rows - 1));
        float4* mine = reinterpret_cast<float4*>(xbuf) + (st & 127) + wg * 512;
        const float4* theirs = reinterpret_cast<const float4*>(xbuf) + (st & 127) + (wg ^ 1) * 512;
#pragma unroll 1
        for (int u = 0; u < D / 32; ++u) {
          const bool give = (u & 1) == 0;
          const int c = (give ? wg ^ 1 : wg) * (D / 64) + (u >> 1);
          float y[16];
          get(c, y);
          if (!give || u > 0) soft_sync();
          if (give) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mine[k * 128] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 v = theirs[k * 128];
              put(local, to, half * (D / 2) + c * 16 + 4 * k,
                  make_float4(y[4 * k] + v.x, y[4 * k + 1] + v.y, y[4 * k + 2] + v.z, y[4 * k + 3] + v.w));
            }
          }
        }
      } else {
        // A row is in 2 KG warps: all of them leave 32 of its dims, and 256
        // threads add four dims each.
        __nv_bfloat16* put_out = out_row(min(st >> 3, n_rows - 1));
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float y[16];
          get(c, y);
          float* to = xbuf + (size_t)((wg * 4 + w) * 16 + r16) * 36 + half * 16;
#pragma unroll
          for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(to + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
          soft_sync();
          const int local = st >> 3, d4 = (st & 7) * 4;
          if (local < NRB * 16) {
            const float* from = xbuf + (size_t)local * 36 + d4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int y2 = 0; y2 < 2 * KG; ++y2) {
              const float4 o4 = *reinterpret_cast<const float4*>(from + ((y2 / KG) * 4 + NRB * (y2 % KG)) * 16 * 36);
              v.x += o4.x, v.y += o4.y, v.z += o4.z, v.w += o4.w;
            }
            put(local, put_out, (d4 >> 4) * (D / 2) + c * 16 + (d4 & 15), v);
          }
          soft_sync();
        }
      }
      sm100::tc_fence_before();
      if (!whole) {
        soft_sync();
        if (st == 0)
          *last_flag = arrive_at(p.arrived + ((int64_t)seg.b * p.Hkv + kvh) * p.row_tiles + row_tile) == in.y - in.x;
        soft_sync();
        if (*last_flag) join_parts<D, NRB>(p, seg, in, kvh, row_tile, st, 256);
      }
      soft_sync();                                             // red, the flag and the bitmap have been read
      if (st < 64) nanmap[(sn % kNanSegs) * 64 + st] = 0;
    }
    if (!ok && lane == 0) {
      *abort = 1;
      raise_error(p.err, MTP_ERR_TIMEOUT);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    // --------------------------------------------------- Q, then masked V
    // Q of a request: eight threads a row, D/8 dims each, read while the last
    // one's tiles are still worked on, and written once its last S is done.
    constexpr int kDims = D / 8, kVec = kDims / 8;         // 16-byte vectors of bf16
    const int cw = warp - 12;            // 32 of a tile's keys
    const int t128 = threadIdx.x - 384, r16 = t128 >> 3, part = t128 & 7;
    int s = 0, g = 0;
    uint32_t phase = 0;
    Seg seg;
    for (int sn = 0;; ++sn) {
      if (threadIdx.x == 384) rest[sn % kSegs] = 0;
      ok = barrier_all<2, 128>(ok && take(sn, seg));
      if (!ok || seg.n == 0) break;
      uint4 w[NRB][kVec];
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb) {
        const int row = min(row_tile * 64 + rb * 16 + r16, p.rows - 1);   // padding repeats the last row
        const int64_t at = ((int64_t)(seg.b * (int64_t)p.R + row / p.group) * p.Hq + kvh * p.group + row % p.group) * D;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at + part * kDims);
#pragma unroll
        for (int v = 0; v < kVec; ++v) w[rb][v] = __ldg(src + v);
      }
      ok = __all_sync(0xffffffffu, sm100::mbar_wait(q_empty, (uint32_t)((sn & 1) ^ 1), abort) ? 1 : 0);
      bool need = false;
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb) {
        float top = 0.0f, sum = 0.0f, left = 0.0f;
        float q[kDims];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const uint32_t word[4] = {w[rb][v].x, w[rb][v].y, w[rb][v].z, w[rb][v].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            q[v * 8 + e] = __uint_as_float((e & 1) ? word[e >> 1] & 0xffff0000u : word[e >> 1] << 16);
            const float a = fabsf(q[v * 8 + e]);
            top = fmaxf(top, a <= FLT_MAX ? a : 0.0f);
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = top > 0.0f ? max(-100, (int)(__float_as_uint(top) >> 23) - 127 - 7) : 0;
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        uint32_t hi[kDims / 4], lo[kDims / 4], re[kDims / 4];
#pragma unroll
        for (int x = 0; x < kDims / 4; ++x) {
          float a[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = fabsf(q[x * 4 + e]) <= FLT_MAX ? q[x * 4 + e] * down : __uint_as_float(0x7fffffffu);
            sum += fabsf(a[e]);
          }
          hi[x] = f_to_e4m3x4(a[0], a[1], a[2], a[3]);
          const float4 h = e4m3x4_to_f(hi[x]);
          a[0] -= h.x, a[1] -= h.y, a[2] -= h.z, a[3] -= h.w;
          lo[x] = f_to_e4m3x4(a[0], a[1], a[2], a[3]);
          const float4 l = e4m3x4_to_f(lo[x]);
          a[0] -= l.x, a[1] -= l.y, a[2] -= l.z, a[3] -= l.w;
          left += fabsf(a[0]) + fabsf(a[1]) + fabsf(a[2]) + fabsf(a[3]);
          const uint32_t r0 = __nv_cvt_float2_to_fp8x2(make_float2(a[0], a[1]), __NV_SATFINITE, __NV_E5M2);
          const uint32_t r1 = __nv_cvt_float2_to_fp8x2(make_float2(a[2], a[3]), __NV_SATFINITE, __NV_E5M2);
          re[x] = r0 | (r1 << 16);
        }
#pragma unroll
        for (int y = 0; y < KG; ++y) {                     // the row's lanes: of warps rb, rb + NRB, ..
          const int l128 = 32 * (rb + NRB * y) + r16;
          auto put = [&](uint8_t* to, const uint32_t* v) {  // 16 or 8 bytes
            if constexpr (kDims == 16) *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
            else *reinterpret_cast<uint2*>(to) = make_uint2(v[0], v[1]);
          };
          const int chunk = part * kDims / 16, in = part * kDims % 16;
          if (ok) {
            put(smem + S::kQ + S::at(l128, chunk) + in, hi);
            put(smem + S::kQ + S::at(l128 + 16, chunk) + in, lo);
            put(smem + S::kQ + S::kTile + S::at(l128, chunk) + in, re);
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
          left += __shfl_xor_sync(0xffffffffu, left, o);
        }
        need |= left > sum * 0x1p-19f;
        if (part == 0) fac[(sn % kSegs) * 64 + rb * 16 + r16] = p.sm_scale * kLog2e * __uint_as_float((uint32_t)(127 + ex) << 23);
      }
      if (need) rest[sn % kSegs] = 1;
      fence_async_smem();
      sm100::mbar_arrive(&fac_full[sn % kSegs]);
      sm100::mbar_arrive(q_full);

      const int tiles = seg.tiles();
      for (int i = 0; i < tiles; ++i, ++g) {
        ok = ok && __all_sync(0xffffffffu, (sm100::mbar_wait(&info_full[g % kInfo], (uint32_t)((g / kInfo) & 1), abort) &&
                                            sm100::mbar_wait(&v_full[s], phase, abort))
                                               ? 1
                                               : 0);
        if (!ok) break;
        const int mark = info[g % kInfo].page[cw >> 1].mark;
        if (mark < 0) {                  // some of its slots are hidden, or nothing was loaded
          uint8_t* v = smem + S::kV + s * S::kTile;
          for (int x = lane; x < 32 * (D / 16); x += kWarp) {
            const int key = cw * 32 + x / (D / 16), c = x % (D / 16);
            uint4* at = reinterpret_cast<uint4*>(v + S::at(key, c));
            uint4 b = *at;
            const int slot = (-2 - mark) * kBlock + (key & 63), bit = c * 16 & 31;
            uint32_t* row_bits = nanmap + (sn % kNanSegs) * 64 + (c >> 1);
            if (mark == -1) {
              b = make_uint4(0, 0, 0, 0);
            } else {
              b.x = hide_nan(p, b.x, slot, seg.ctx, row_bits, bit);
              b.y = hide_nan(p, b.y, slot, seg.ctx, row_bits, bit + 4);
              b.z = hide_nan(p, b.z, slot, seg.ctx, row_bits, bit + 8);
              b.w = hide_nan(p, b.w, slot, seg.ctx, row_bits, bit + 12);
            }
            *at = b;
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&v_ready[s]);
        if (++s == kVStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      raise_error(p.err, MTP_ERR_TIMEOUT);
    }
  }

  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  if (warp == 0) sm100::tmem_dealloc(tmem, 512);
}

template <int D, int NRB>
cudaError_t launch(const mtp_window_attn_args& a, const WindowPlan& pl, const WindowParams& p, cudaStream_t s) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.Hkv, (cuuint64_t)kBlock, (cuuint64_t)a.num_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)a.Hkv * D, (cuuint64_t)kBlock * a.Hkv * D};
  const cuuint32_t box[4] = {(cuuint32_t)D, 1, (cuuint32_t)kBlock, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i) {
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i == 0 ? a.k_cache : a.v_cache, dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kern = kv8_tc_kernel<D, NRB>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_behind_append(kern, (unsigned)(pl.ctas_per_head * a.Hkv * pl.row_tiles), kThreads, Smem<D>::kBytes, s, maps[0],
                              maps[1], p);
}

// Blocks of 16 rows of a CTA: 1, 2 or 4; a KV head of more than 64 rows takes
// several CTAs of 64.
int row_blocks(const mtp_window_attn_args& a) {
  const int rows = a.Hq / a.Hkv * (a.D + 1);
  return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

}  // namespace

WindowPlan plan_kv8_tc(const mtp_window_attn_args& a, int sm_count) {
  WindowPlan pl{};
  const int nrb = row_blocks(a);
  pl.row_tiles = (a.Hq / a.Hkv * (a.D + 1) + 63) / 64;
  pl.row_warps = 1;                                        // arrival counters per (request, KV head, row tile)
  const size_t heads = (size_t)a.Hkv * pl.row_tiles;
  pl.ctas_per_head = head_ctas(a, sm_count, (long long)heads);
  pl.ws_partial_o = plan_schedule(&pl, a.B, a.Hkv);
  pl.ws_bytes = pl.ws_partial_o + (size_t)pl.ctas_per_head * 2 * heads * nrb * 16 * (a.d + 2) * sizeof(float);
  pl.ws_bytes = (pl.ws_bytes + 255) / 256 * 256;
  return pl;
}

cudaError_t launch_kv8_tc(const mtp_window_attn_args& a, const WindowPlan& pl, const WindowParams& p, cudaStream_t s) {
  const int nrb = row_blocks(a);
  if (a.d == 128) return nrb == 1 ? launch<128, 1>(a, pl, p, s) : nrb == 2 ? launch<128, 2>(a, pl, p, s) : launch<128, 4>(a, pl, p, s);
  return nrb == 1 ? launch<64, 1>(a, pl, p, s) : nrb == 2 ? launch<64, 2>(a, pl, p, s) : launch<64, 4>(a, pl, p, s);
}

}  // namespace mtp
