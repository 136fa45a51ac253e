// Launch parameters shared by the kernels of attention_window.cu and
// attention_window_mma.cu.
#pragma once

#include "kernels.h"

namespace mtp {

struct WindowPlan {
  int n_splits;            // SIMT: ranges a request's pages are cut into
  size_t ws_partial_o, ws_partial_lse, ws_bytes;
};

struct WindowParams {
  const void* q;
  void* out;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;   // [num_blocks, Hkv], nullptr: the cache holds the rows' type
  const int32_t *block_table, *ctx_lens;
  float *part_o, *part_lse;         // [row][split][d], [row][split] (base 2)
  unsigned* err;
  int B, R, Hq, Hkv, group, rows;   // rows = query rows per (request, KV head)
  int max_blocks, num_blocks, window, sinks, n_splits;
  float sm_scale;
};

}  // namespace mtp
