// Launch parameters shared by attention_window.cu, attention_window_mma.cu
// and the appends that run before them.
#pragma once

#include <float.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mtp {

// The running maximum of a row that has seen slots, all with scores of -inf: its softmax is NaN. (-inf: it has seen
// none, and is 0.)
constexpr float kNoWeight = -FLT_MAX;

struct WindowPlan {
  int n_splits;                      // SIMT: ranges a request's pages are cut into
  int row_tiles, row_warps, key_parts, stages, ctas_per_head, smem;   // tensor cores
  size_t ws_partial_o, ws_partial_lse;
  size_t ws_prefix, ws_shares, ws_sharers, ws_arrived;
  size_t ws_bytes;
};

// How the pages that the requests' rows see are shared out. Request after
// request they form one line for each KV head, cut into a share for each of
// its CTAs, of eight pages at least (4 to 16: within 1 us). Cuts are even,
// except that those of small shares move to a border of two requests that is
// near: a request that several CTAs share is joined at the end, which takes
// about as long as four pages, and so does beginning one (5 windowed requests
// of 8 pages: 20.1 us with even cuts, 12.8 us so). For the same reason each
// request is a share where there are CTAs for all and the longest is no more
// than four pages over an even share (16 requests of 17 or 18 pages on 19 CTAs
// a head: 31.8 us with cuts, 24.4 us so), or has no more than 16 pages. One
// request of n pages, 8 KV heads x 128, in one share / in cuts:
//   n = 9 / 12 / 16 / 17 / 20 / 24
//   8-bit, 16 rows   11.5/12.7  12.1/13.1  13.2/13.4  13.9/13.7  14.4/13.8  15.7/14.2 us
//   8-bit, 48 rows   15.4/19.3  16.4/19.5  17.8/20.1  19.1/21.6  19.6/22.2  21.8/22.4
//   bf16, 16 rows    11.6/12.9  12.7/13.6  14.4/14.4  14.6/13.6  15.6/14.0  17.3/14.6
//   bf16, 48 rows    15.6/14.3  17.8/15.8  21.1/17.5  22.2/15.8  24.4/16.3  27.7/18.1
// (1 row, and head dim 64, as 16 rows; one edge for all forms, which 48 rows
// would have at 24 pages in 8 bits and at 8 in bf16).
// The append launch works this out in one more CTA (window_schedule) and
// clears the arrival counters of shared requests.
struct alignas(16) Share {
  int32_t begin, p0;                // its first page of the line; the first one of that page's request,
  int32_t b, n, ctx;                // .. which has n pages and a context of ctx
  int32_t count;                    // of shares
};
struct WindowParams {
  const void* q;
  void* out;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;   // [num_blocks, Hkv], nullptr: the cache holds the rows' type
  const int32_t *block_table, *ctx_lens;
  float *part_o, *part_lse;         // SIMT: [row][split][d], [row][split] (base 2); tensor cores: see the kernel
  const int32_t* prefix;            // see WindowSchedule
  const Share* shares;
  const int2* sharers;
  int32_t* arrived;                 // [B][Hkv][row blocks] CTAs that have left a partial result
  unsigned* err;
  int B, R, Hq, Hkv, group, rows;   // rows = query rows per (request, KV head)
  int max_blocks, num_blocks, window, sinks, n_splits;
  int row_tiles, row_warps, key_parts, stages;
  float sm_scale;
};

struct WindowSchedule {
  int32_t* prefix;                  // [B+1] pages of the requests before each; nullptr: nothing to prepare
  Share* shares;                    // [ctas + 1]; the one after the last begins at the line's end
  int2* sharers;                    // [B] first and last share that a request is in
  int32_t* arrived;
  int64_t n_arrived;
  const int32_t* ctx_lens;
  int B, R, max_blocks, window, sinks, ctas;
};

// CTAs of a head (a KV head's tile of rows): those that fit the device once,
// as far as the widest table gives them a request or eight pages each. A whole
// number for each head, so what 152 SMs leave over is idle (the same work as
// 8 / 32 / 40 / 80 / 160 KV heads, group 1: 8-bit 221 / 243 / 255 / 361 / 385
// us, windowed bf16 218 / 239 / 235 / 312 / 353 us).
inline int head_ctas(const mtp_window_attn_args& a, int sm_count, long long heads) {
  const long long seen = a.window == 0 ? a.max_blocks   // pages that a request's rows see at most
                                       : std::min<long long>(a.max_blocks, ((long long)a.window + a.D + 127) / kBlock +
                                                                               ((long long)a.sinks + kBlock - 1) / kBlock);
  const long long useful = std::max<long long>(a.B, (a.B * seen + 7) / 8);
  return (int)std::max<long long>(1, std::min(sm_count / heads, useful));
}

// Lay the schedule out in the workspace of a plan whose ctas_per_head, row_tiles and row_warps are set.
inline size_t plan_schedule(WindowPlan* pl, int B, int Hkv) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  pl->ws_prefix = 0;
  pl->ws_shares = up((size_t)(B + 1) * sizeof(int32_t));
  pl->ws_sharers = pl->ws_shares + up((size_t)(pl->ctas_per_head + 1) * sizeof(Share));
  pl->ws_arrived = pl->ws_sharers + up((size_t)B * sizeof(int2));
  return pl->ws_arrived + up((size_t)B * Hkv * pl->row_tiles * pl->row_warps * sizeof(int32_t));
}

WindowPlan plan_window_mma(const mtp_window_attn_args& a, int sm_count);
cudaError_t launch_window_mma(const mtp_window_attn_args& a, const WindowPlan& pl, const WindowParams& p, cudaStream_t s);
WindowPlan plan_kv8_tc(const mtp_window_attn_args& a, int sm_count);
cudaError_t launch_kv8_tc(const mtp_window_attn_args& a, const WindowPlan& pl, const WindowParams& p, cudaStream_t s);
cudaError_t launch_kv8_append(const mtp_kv8_append_args& a, int uniform, const WindowSchedule& sch, unsigned* err,
                              cudaStream_t s);

// Launch a kernel that waits (griddepcontrol.wait) for the append before it:
// its CTAs may be set up while the append's still run.
template <typename... Params, typename... Args>
cudaError_t launch_behind_append(void (*kern)(Params...), unsigned grid, unsigned threads, int smem, cudaStream_t s,
                                 Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, Params(args)...);
}

}  // namespace mtp
