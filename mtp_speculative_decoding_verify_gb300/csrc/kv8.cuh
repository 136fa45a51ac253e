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

// CTAs of a KV head that get work: all there are, as long as each has four
// pages (a shared request costs a join, about as long as four pages take).
__device__ __forceinline__ int window_ctas(int64_t total, int most) {
  const int64_t want = (total + 3) / 4;
  return (int)(want < most ? want : most);
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
  for (int64_t i = threadIdx.x; i < w.n_arrived; i += THREADS) w.arrived[i] = 0;
}

}  // namespace mtp
