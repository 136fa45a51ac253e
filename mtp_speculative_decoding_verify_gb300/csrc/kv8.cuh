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
  int64_t total;   // pages of the line
  int G;           // shares: all CTAs that there are, as long as each has eight pages
  int near;        // pages that a cut moves at most: less than half a share, so that none is empty, and no more
                   // than a moved cut saves (none for shares over 64 pages)
  __device__ __forceinline__ int64_t even(int64_t g) const { return total * g / G; }
};

__device__ __forceinline__ Cuts make_cuts(int64_t total, int ctas) {
  Cuts c;
  c.total = total;
  const int64_t want = (total + 7) / 8;
  c.G = (int)(want < ctas ? want : ctas);
  const int64_t share = c.G == 0 ? 0 : total / c.G;
  c.near = share == 0 || share > 64 ? 0 : (int)(share > 8 ? 4 : (share - 1) / 2);
  return c;
}

// Where share g begins, and (an early bound of) its request.
__device__ __forceinline__ Share share_begin(const Cuts& c, const int64_t* prefix, int B, int g) {
  Share s{};
  s.begin = c.total;
  if (g == 0) s.begin = 0;
  if (g == 0 || g >= c.G) return s;
  const int64_t pos = c.even(g);
  int lo = 0, hi = B;              // prefix[lo] <= pos < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (prefix[mid] <= pos) lo = mid;
    else hi = mid;
  }
  const int64_t p0 = prefix[lo], p1 = prefix[lo + 1];
  s.begin = pos - p0 <= c.near ? p0 : p1 - pos <= c.near ? p1 : pos;
  s.b = lo;
  return s;
}

// The first and last share that a request of pages p0 .. p1 - 1 of the line is in.
__device__ __forceinline__ int2 request_shares(const Cuts& c, int64_t p0, int64_t p1) {
  int a = (int)(((p0 + 1) * c.G - 1) / c.total), z = (int)((p1 * c.G - 1) / c.total);   // of even cuts
  if (a + 1 < c.G && c.even(a + 1) < p1 && c.even(a + 1) - p0 <= c.near) ++a;            // the cut after p0 moved to p0
  const int64_t cut = c.even(z);
  if (z > 0 && cut >= p0 && cut - p0 > c.near && p1 - cut <= c.near) --z;                // the last one moved to p1
  return make_int2(a, z);
}

// The work of one CTA of THREADS threads (a multiple of 32): see WindowSchedule.
template <int THREADS>
__device__ void window_schedule(const WindowSchedule& w) {
  __shared__ int64_t s_warp[THREADS / kWarp];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  int64_t base = 0;
  for (int b0 = 0; b0 < w.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0;
    if (b < w.B) {
      const int ctx = w.ctx_lens[b];      // a bad length has no pages: its rows stay as they were
      if (ctx >= 0 && ctx <= w.max_blocks * kBlock - w.R) n = page_span(ctx, w.R, w.window, w.sinks).n;
    }
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += y;
    }
    __syncthreads();                       // the last chunk's totals have been read
    if (lane == kWarp - 1) s_warp[warp] = n;
    __syncthreads();
    n += base;
    for (int i = 0; i < THREADS / kWarp; ++i) {
      if (i < warp) n += s_warp[i];
      base += s_warp[i];
    }
    if (b < w.B) w.prefix[b + 1] = n;
  }
  if (threadIdx.x == 0) w.prefix[0] = 0;
  __syncthreads();                         // (writes to global memory too, for this CTA)
  const Cuts cuts = make_cuts(base, w.ctas);
  for (int g = threadIdx.x; g <= cuts.G; g += THREADS) {
    Share sh = share_begin(cuts, w.prefix, w.B, g);
    sh.pad = cuts.G;
    w.shares[g] = sh;
  }
  for (int b = threadIdx.x; b < w.B; b += THREADS) {
    const int64_t p0 = w.prefix[b], p1 = w.prefix[b + 1];
    if (p1 > p0) w.sharers[b] = request_shares(cuts, p0, p1);
  }
  for (int64_t i = threadIdx.x; i < w.n_arrived; i += THREADS) w.arrived[i] = 0;
}

}  // namespace mtp
