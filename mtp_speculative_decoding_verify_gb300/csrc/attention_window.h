// Launch parameters shared by attention_window.cu, attention_window_mma.cu
// and the appends that run before them.
#pragma once

#include "kernels.h"

namespace mtp {

struct WindowPlan {
  int n_splits;                      // SIMT: ranges a request's pages are cut into
  int row_tiles, row_warps, key_parts, stages, ctas_per_head, smem;   // tensor cores
  size_t ws_partial_o, ws_partial_lse;
  size_t ws_prefix, ws_arrived;
  size_t ws_bytes;
};

struct WindowParams {
  const void* q;
  void* out;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;   // [num_blocks, Hkv], nullptr: the cache holds the rows' type
  const int32_t *block_table, *ctx_lens;
  float *part_o, *part_lse;         // SIMT: [row][split][d], [row][split] (base 2); tensor cores: see the kernel
  const int64_t* prefix;            // [B+1] pages of the requests before each (WindowSchedule)
  int32_t* arrived;                 // [B][Hkv][row blocks] CTAs that have left a partial result
  unsigned* err;
  int B, R, Hq, Hkv, group, rows;   // rows = query rows per (request, KV head)
  int max_blocks, num_blocks, window, sinks, n_splits;
  int row_tiles, row_warps, key_parts, stages;
  float sm_scale;
};

// What the append launch prepares for the tensor-core kernel in one more CTA:
// the prefix sums of the requests' pages, and zeros for the arrival counters.
struct WindowSchedule {
  int64_t* prefix;                  // nullptr: nothing to prepare
  int32_t* arrived;
  int64_t n_arrived;
  const int32_t* ctx_lens;
  int B, R, max_blocks, window, sinks;
};

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
