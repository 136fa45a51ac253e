// The join of mtp_verify_attention_prefix: the results over the group's prefix
// and over the request's own slots become the output.
#include <math.h>

#include "attention_prefix.h"
#include "attention_window.h"
#include "mma_sync.cuh"

namespace mtp {
namespace {

constexpr int kJoinThreads = 128;
// 32 dims of a row a warp from 1024 rows on (2496 rows of trees: 21.0 us with 16,
// 19.5 us so; 256 rows with 17 results: 15.0 us with 16, and 17.2 with those in
// batches of 8), 64 from 4096 on (7808 rows: 101.5 us with 32, 105.0 with 128, 99.7
// so; 24576 rows: 50.2 with 128, 48.7 so); calls in a graph. Where they cross goes by
// the number of results, too: D = 3, 32/8 x 128, 2048 shared tokens, up to 200 own, us
// with 16, 32 and 64: 512 rows 15.2, 17.6, 23.0; 1024 16.8, 18.4, 23.6; 1536 21.6, 20.7,
// 25.3; 2048 22.2, 20.1, 24.2; 4096 31.8, 26.0, 26.5; 6144 38.2, 27.8, 27.3; 8192 45.7,
// 33.2, 30.4.
constexpr unsigned kSomeRows = 1024, kManyRows = 4096;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// out = (sum of o 2^(m - top)) / (sum of l 2^(m - top)) over a row's partial
// results, the prefix's and then its own. A warp takes 8 rows of one KV head,
// as they lie in the results, and SLICES x 16 dims, 4 of each a lane: the more
// rows there are to fill the device, the more dims, so that the finding of the
// results is paid less often; with fewer, more warps share the work and more
// results are read as one batch. Bound by what it reads, out of L2 mostly
// (32768 rows, 59 MB: 16 us), and by one round of reads where that is little.
template <typename T>
__device__ __forceinline__ void store4(T* to, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* to, float4 v) {
  *reinterpret_cast<float4*>(to) = v;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* to, float4 v) {
  *reinterpret_cast<uint2*>(to) = make_uint2(mma::pack_bf16(v.x, v.y), mma::pack_bf16(v.z, v.w));
}

template <typename T, int D, int SLICES>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixParams p, unsigned n_rows) {
  constexpr unsigned kUnits = D / 16 / SLICES;   // warps that share a row
  constexpr int kMost = SLICES == 1 ? 20 : SLICES == 2 ? 8 : 4;   // results read as one batch
  const unsigned lane = threadIdx.x % kWarp, unit = blockIdx.x * (kJoinThreads / kWarp) + threadIdx.x / kWarp;
  const unsigned place = unit / kUnits * 8 + lane / 4, idx = min(place, n_rows - 1);
  const int dim4 = unit % kUnits * SLICES * 4 + lane % 4;   // 4 dims from 4 dim4 + 16 x on
  const unsigned rows = p.rows, bh = idx / rows, r = idx - bh * rows, b = bh / (unsigned)p.Hkv, kvh = bh - b * p.Hkv;
  const PrefixView& v = p.view;
  const int first = __ldcg(v.first + b), gi = __ldcg(v.group_of + b);
  const PrefixHead head = load_head(v.head);
  const unsigned j = r / (unsigned)p.group, h = kvh * p.group + (r - j * p.group);
  const int64_t row = ((int64_t)b * p.R + j) * p.Hq + h;
  // The own results: n1 of them, step1 rows from one to the next.
  const unsigned step1 = p.row_warps * 16, tile = r / step1;
  const PrefixHead own = load_head(v.own);
  const int before = __ldcg(v.pages + b), pages = __ldcg(v.pages + b + 1) - before;
  const int heads = p.Hkv * p.row_tiles, hr = kvh * p.row_tiles + tile, u0 = before * heads + hr * pages;
  const int c0 = prefix_cta_of(own, u0), n1 = prefix_cta_of(own, u0 + pages - 1) - c0 + 1;
  const int64_t at1 = ((int64_t)b * heads + hr + c0) * step1 + (r - tile * step1);
  const float* o1 = v.own_parts + at1 * D;
  const float2* m1 = v.own_stats + at1;
  PrefixRow pre{nullptr, nullptr, 0, 0};
  if (gi >= 0) pre = prefix_row(v, head, load_group(v.groups + gi), p.R, p.group, b, kvh, r, D);
  const int n = pre.n + n1, rows0 = v.shape.rows;
  // So far only what the append's launch left has been read, which was complete before the kernel ahead let this one
  // begin (if it did before its own end). What follows reads that kernel's results.
  // A warp without rows waits too: the launch behind this one may only begin once the kernel ahead is done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (place >= n_rows || first < 0) return;  // (a flagged request's rows stay as they were)

  float m = -INFINITY, l = 0.0f;
  float4 o[SLICES];
#pragma unroll
  for (int x = 0; x < SLICES; ++x) o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k0 = 0; k0 < n; k0 += kMost) {
    float2 ml[kMost];
    const float* from[kMost];
    int step[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      ml[k] = make_float2(-INFINITY, 0.0f);
      from[k] = nullptr;
      step[k] = 0;
      const int i = k0 + k;
      if (i < pre.n) {
        const int64_t at = (int64_t)i * pre.step * rows0;
        ml[k] = __ldcg(pre.ml + at);
        from[k] = pre.o + at * D + dim4 * rows0 * 4;
        step[k] = rows0 * 16;                // from 4 dims to those 16 on
      } else if (i < n) {
        const int64_t at = (int64_t)(i - pre.n) * step1;
        ml[k] = __ldcg(m1 + at);
        from[k] = o1 + at * D + dim4 * 4;
        step[k] = 16;
      }
    }
    // (the first slice with the maxima, each next one while one is added up)
    float4 w[2][kMost];
    auto read = [&](int x) {
#pragma unroll
      for (int k = 0; k < kMost; ++k)
        if (from[k] != nullptr) w[x & 1][k] = __ldcg(reinterpret_cast<const float4*>(from[k] + x * step[k]));
    };
    read(0);
    float top = m;
#pragma unroll
    for (int k = 0; k < kMost; ++k) top = fmaxf(top, ml[k].x);
    const float a = m == -INFINITY ? 0.0f : ex2(m - top);
    m = top;
    l *= a;
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      ml[k].x = ml[k].x == -INFINITY ? 0.0f : ex2(ml[k].x - top);
      l += ml[k].y * ml[k].x;
    }
#pragma unroll
    for (int x = 0; x < SLICES; ++x) {
      if (x + 1 < SLICES) read(x + 1);
      o[x].x *= a, o[x].y *= a, o[x].z *= a, o[x].w *= a;
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        if (k0 + k < n) {                    // (0 x NaN of a part that is none)
          const float c = ml[k].x;
          const float4 y = w[x & 1][k];
          o[x].x += y.x * c, o[x].y += y.y * c, o[x].z += y.z * c, o[x].w += y.w * c;
        }
      }
    }
  }
  // no weight: nothing seen (bad blocks only), or -inf only
  const float inv = l != 0.0f ? 1.0f / l : m == -INFINITY ? 0.0f : NAN;
#pragma unroll
  for (int x = 0; x < SLICES; ++x)
    store4<T>(static_cast<T*>(p.out) + row * D + dim4 * 4 + x * 16, make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv));
}

template <typename T, int D>
cudaError_t launch_join(const PrefixParams& p, cudaStream_t s) {
  const unsigned rows = (unsigned)p.B * p.Hkv * p.rows, groups = (rows + 7) / 8, warps = kJoinThreads / kWarp;
  auto launch = [&](auto kernel, unsigned slices) {
    return launch_behind_append(kernel, (groups * (D / 16 / slices) + warps - 1) / warps, kJoinThreads, 0, s, p, rows);
  };
  if (rows >= kManyRows) return launch(prefix_join_kernel<T, D, 4>, 4);
  if (rows >= kSomeRows) return launch(prefix_join_kernel<T, D, 2>, 2);
  return launch(prefix_join_kernel<T, D, 1>, 1);
}

}  // namespace

cudaError_t launch_prefix_join(const mtp_prefix_attn_args& a, const PrefixParams& p, cudaStream_t s) {
  if (a.dtype == MTP_F32) return a.d == 128 ? launch_join<float, 128>(p, s) : launch_join<float, 64>(p, s);
  return a.d == 128 ? launch_join<__nv_bfloat16, 128>(p, s) : launch_join<__nv_bfloat16, 64>(p, s);
}

}  // namespace mtp
