// The 8-bit paged cache: e4m3 bytes and one fp32 scale for each block of 64
// tokens and KV head (value = byte * scale), and the pages that a windowed
// request reads. Shared by the append, attention and release kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>

#include "attention_window.h"
#include "common.cuh"

namespace mtp {

constexpr float kE4m3Max = 448.0f;
constexpr int kMinScaleExp = -100;   // scale of a block of zeros; what is tiny next to it was never written

// ------------------------------------------------------------------ e4m3
// Four bytes (ascending address) to floats; exact.
__device__ __forceinline__ float4 e4m3x4_to_f(uint32_t w) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Round to e4m3, to nearest even, and pack (a in the lowest byte). The
// inputs are at most 448 in magnitude or NaN.
__device__ __forceinline__ uint32_t f_to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Scales that the append makes lie in [2^-100, 2^121): what is outside was not
// written by it, and a block with such a scale takes no part.
__device__ __forceinline__ bool scale_ok(float s) { return s >= 0x1p-100f && s < 0x1p121f; }

// Scale of a block's head after values of largest finite magnitude `a` are
// written to it: the old scale (2^-100 when the block's first slot is among
// the written ones) doubled until a <= 448 scale. Doubling keeps what the
// block holds exact (a byte's value halves) except for e4m3 subnormals, which
// round once per call. *k is the number of doublings.
__device__ __forceinline__ float grown_scale(float old, bool fresh, float a, int* k) {
  float s = fresh ? ldexpf(1.0f, kMinScaleExp) : old;
  int n = 0;
  if (kE4m3Max * s < a) {
    int ea, es;
    frexpf(a, &ea);
    frexpf(s, &es);
    n = max(0, ea - es - 10);   // 448 s 2^n < a still, or n = 0: at most three doublings follow
    s = ldexpf(s, n);
    while (kE4m3Max * s < a) {
      s *= 2.0f;
      ++n;
    }
  }
  *k = n;
  return s;
}

// --------------------------------------------------------- pages of a window
// Row j of a request with ctx cached tokens sits at position p = ctx + j and
// sees slot t iff t <= p and (window == 0, or t > p - window, or t < sinks).
__host__ __device__ __forceinline__ bool slot_visible(int t, int p, int window, int sinks) {
  return t <= p && (window == 0 || t > p - window || t < sinks);
}

// The row sees a slot of the page.
__device__ __forceinline__ bool page_seen(int page, int p, int window, int sinks) {
  const int first = page * kBlock;
  return first <= p && (window == 0 || first + kBlock - 1 > p - window || first < sinks);
}

// The blocks that hold a slot some row of the request sees, in order: the
// sink blocks 0 .. n_sink-1, then w0 .. the block of the last verify token.
struct PageSpan {
  int n_sink, w0, n;
  __host__ __device__ __forceinline__ int page(int i) const { return i < n_sink ? i : w0 + (i - n_sink); }
};

__host__ __device__ __forceinline__ PageSpan page_span(int ctx, int R, int window, int sinks) {
  PageSpan s;
  const int pages = (ctx + R + kBlock - 1) / kBlock;
  const int lo = ctx - window + 1;   // first slot in row 0's window
  s.w0 = (window == 0 || lo <= 0) ? 0 : lo / kBlock;
  const int sink_pages = (sinks + kBlock - 1) / kBlock;
  s.n_sink = window == 0 ? 0 : (sink_pages < s.w0 ? sink_pages : s.w0);
  s.n = s.n_sink + pages - s.w0;
  return s;
}

// ----------------------------------------------------------- shares of work
struct Cuts {
  int total;       // pages of the line
  int G;           // shares: all CTAs that there are, as long as each has eight pages
  int size, more;  // pages of a share; the first `more` have one page more
  int near;        // pages that a cut moves at most: less than half a share, so that none is empty, and no more
                   // than a moved cut saves (none for shares over 64 pages)
  bool whole;      // share g is request g instead
  __device__ __forceinline__ int even(int g) const { return g * size + min(g, more); }
  __device__ __forceinline__ int share_of(int page) const {   // with even cuts
    const int split = more * (size + 1);
    return page < split ? page / (size + 1) : more + (page - split) / size;
  }
};

__device__ __forceinline__ Cuts make_cuts(int total, int ctas, int B, int longest) {
  Cuts c;
  c.total = total;
  c.G = min((int)((total + 7u) / 8u), ctas);
  c.size = c.G == 0 ? 0 : total / c.G;
  c.more = total - c.G * c.size;
  c.near = c.size == 0 || c.size > 64 ? 0 : c.size > 8 ? 4 : (c.size - 1) / 2;
  c.whole = total > 0 && B <= ctas && longest <= max(c.size + 4, 16);
  if (c.whole) c.G = B;
  return c;
}

// Request b, pages p0 .. p1 - 1 of the line: the shares that begin in it, and the first and last that it is in.
__device__ __forceinline__ void write_shares(const WindowSchedule& w, const Cuts& c, int b, int p0, int p1, int ctx) {
  Share s{p0, p0, b, p1 - p0, ctx, c.G};
  if (c.whole) {
    w.shares[b] = s;
    w.sharers[b] = make_int2(b, b);
    return;
  }
  if (p0 == p1) return;
  int a = c.share_of(p0), z = c.share_of(p1 - 1);
  for (int g = c.even(a) == p0 ? a : a + 1; g <= z; ++g) {
    const int cut = c.even(g);
    s.begin = cut - p0 <= c.near ? p0 : p1 - cut <= c.near ? p1 : cut;
    w.shares[g] = s;
  }
  if (a < z && c.even(a + 1) - p0 <= c.near) ++a;   // the cut after p0 moved to p0
  const int cut = c.even(z);
  if (cut - p0 > c.near && p1 - cut <= c.near) --z;   // the last one moved to p1
  w.sharers[b] = make_int2(a, z);
}

// What a CTA behind the append reads of it: not by the read-only path, since
// the append may still have run when this grid began. The three are
// independent, and within the array whatever g is.
__device__ __forceinline__ Share load_share(const Share* shares, int g) {
  const int4 v = __ldcg(reinterpret_cast<const int4*>(shares + g));
  const int2 r = __ldcg(reinterpret_cast<const int2*>(&shares[g].ctx));
  return Share{v.x, v.y, v.z, v.w, r.x, r.y};
}
__device__ __forceinline__ int share_end(const Share* shares, int g) { return __ldcg(&shares[g + 1].begin); }
__device__ __forceinline__ int share_count(const Share* shares) { return __ldcg(&shares[0].count); }

// Count a part as left at *arrived; how many were before. One thread: what
// others wrote before they met it is released with it, and what was left
// before is there for those that meet it later.
__device__ __forceinline__ int arrive_at(int32_t* arrived) {
  int before;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(arrived) : "memory");
  return before;
}

// The work of one CTA of THREADS threads (a multiple of 32): see WindowSchedule.
// It stands between the lengths and the attention, and most of its time is the
// fetch of its own instructions: no division of 64 bits, and no search. (64
// requests x 48 rows of 4096 tokens, 8-bit: 148.5 us with both, 141.3 us so.)
template <int THREADS>
__device__ void window_schedule(const WindowSchedule& w) {
  constexpr int kWarps = THREADS / kWarp;
  __shared__ int s_sum[kWarps], s_most[kWarps];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  int base = 0, most = 0, n = 0, p1 = 0, ctx = 0;
  for (int b0 = 0; b0 < w.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    n = 0;
    if (b < w.B) {
      ctx = w.ctx_lens[b];                // a bad length has no pages: its rows stay as they were
      if (ctx >= 0 && ctx <= w.max_blocks * kBlock - w.R) n = page_span(ctx, w.R, w.window, w.sinks).n;
    }
    most = max(most, n);
    p1 = n;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, p1, o);
      if (lane >= o) p1 += y;
    }
    __syncthreads();                       // the last chunk's totals have been read
    if (lane == kWarp - 1) s_sum[warp] = p1;
    const int warp_most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_most[warp] = warp_most;
    __syncthreads();
    p1 += base;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) p1 += s_sum[i];
      base += s_sum[i];
      most = max(most, s_most[i]);
    }
    if (b < w.B) w.prefix[b + 1] = p1;
  }
  const Cuts cuts = make_cuts(base, w.ctas, w.B, most);
  if (threadIdx.x == 0) {
    w.prefix[0] = 0;
    w.shares[cuts.G] = Share{base, base, 0, 0, 0, cuts.G};
  }
  if (w.B <= THREADS) {
    if (threadIdx.x < w.B) write_shares(w, cuts, threadIdx.x, p1 - n, p1, ctx);
  } else {
    __syncthreads();                       // (writes to global memory too, for this CTA)
    for (int b = threadIdx.x; b < w.B; b += THREADS) write_shares(w, cuts, b, w.prefix[b], w.prefix[b + 1], w.ctx_lens[b]);
  }
  for (int64_t i = threadIdx.x; i < w.n_arrived; i += THREADS) w.arrived[i] = 0;
}

}  // namespace mtp
