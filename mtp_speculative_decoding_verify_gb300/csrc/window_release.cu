// kv_window_release: the blocks that have left every row's window go back to
// the free list, beside kv_rollback, which gives back the blocks behind the
// kept tokens ("MTP in TensorRT-LLM", MTP Vanilla / MTP Eagle and the Fig. 4
// workflow: the cache is trimmed outside the engine forward).
//
// With L tokens kept, the next step's rows sit at positions >= L and see
// slots > L - window and slots < sinks, so block i holds nothing visible iff
// 64 i >= sinks and 64 i + 63 <= L - window: ceil(sinks/64) <= i <
// (L - window + 1) / 64. Blocks are appended request-major, ascending.
//
// Two launches of one CTA per request: the first counts the blocks to free
// (table entries >= 0 in the range), the second sums the counts of the
// earlier requests to find its place and moves its entries with a scan over
// each 1024. Both read the range once; the launches and the chain of
// dependent loads bound it, not bytes: 3.3 us for 16 requests of 129 blocks,
// 10.1 us for 512 of 2048. (One CTA and one launch for small tables: 4.3 us for
// the 16, 14 us for 63 requests of 130 blocks, which take 4.2 us so.)
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mtp {
int device_context(unsigned** err, int* sm_count);
int set_error(int code, const char* msg);
int set_cuda_error(cudaError_t e, const char* what);
void set_launch_count(int n);

namespace {

constexpr int kThreads = 256, kWarps = kThreads / kWarp, kPer = 4;

// The request's range of blocks to look through, empty when its length is bad.
__device__ __forceinline__ bool release_range(int len, int window, int sink_blocks, int max_blocks, int* i0, int* i1) {
  *i0 = *i1 = 0;
  if (len < 0 || len > max_blocks * kBlock) return false;
  *i0 = sink_blocks;
  *i1 = max(sink_blocks, max(0, len - window + 1) / kBlock);
  return true;
}

__global__ void __launch_bounds__(kThreads) window_count_kernel(const int32_t* __restrict__ table,
                                                               const int32_t* __restrict__ seq_lens,
                                                               const int32_t* __restrict__ free_count, int window,
                                                               int sink_blocks, int max_blocks,
                                                               int32_t* __restrict__ counts, unsigned* err) {
  __shared__ int s_warp[kWarps];
  const int b = blockIdx.x;
  int i0, i1, n = 0;
  if (!release_range(seq_lens[b], window, sink_blocks, max_blocks, &i0, &i1) && threadIdx.x == 0)
    raise_error(err, MTP_ERR_LENGTH);
  for (int i = i0 + threadIdx.x; i < i1; i += kThreads) n += table[(int64_t)b * max_blocks + i] >= 0;
  n = __reduce_add_sync(0xffffffffu, n);
  if (threadIdx.x % kWarp == 0) s_warp[threadIdx.x / kWarp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    n = 0;
    for (int w = 0; w < kWarps; ++w) n += s_warp[w];
    counts[b + 1] = n;
    if (b == 0) counts[0] = *free_count;   // the second launch advances it while others still need it
  }
}

__global__ void __launch_bounds__(kThreads) window_move_kernel(int32_t* __restrict__ table,
                                                              const int32_t* __restrict__ seq_lens,
                                                              int32_t* __restrict__ free_list,
                                                              int32_t* __restrict__ free_count, int window,
                                                              int sink_blocks, int max_blocks, int capacity,
                                                              const int32_t* __restrict__ counts, unsigned* err) {
  __shared__ long long s_sum[kWarps];
  __shared__ int s_warp[kWarps];
  const int b = blockIdx.x, lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int n = counts[b + 1];
  if (n == 0) return;
  long long before = 0;                    // the free list's length and the earlier requests' blocks
  for (int i = threadIdx.x; i <= b; i += kThreads) before += counts[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) s_sum[warp] = before;
  __syncthreads();
  before = 0;
  for (int w = 0; w < kWarps; ++w) before += s_sum[w];
  if (counts[0] < 0 || before + n > capacity) {   // whole or not at all, as in kv_rollback
    if (threadIdx.x == 0) raise_error(err, MTP_ERR_FREE_LIST);
    return;
  }
  int i0, i1;
  release_range(seq_lens[b], window, sink_blocks, max_blocks, &i0, &i1);
  int32_t* row = table + (int64_t)b * max_blocks;
  int at = (int)before;
  for (int base = i0; base < i1; base += kThreads * kPer) {
    const int i = base + threadIdx.x * kPer;
    int v[kPer], mine = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      v[e] = i + e < i1 ? row[i + e] : -1;
      mine += v[e] >= 0;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();                       // the last chunk's totals have been read
    if (lane == kWarp - 1) s_warp[warp] = incl;
    __syncthreads();
    int pos = at + incl - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pos += s_warp[w];
      total += s_warp[w];
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (v[e] >= 0) {
        free_list[pos++] = v[e];
        row[i + e] = -1;
      }
    }
    at += total;
  }
  if (threadIdx.x == 0) atomicMax(free_count, (int)before + n);
}

int fail(const char* msg) { return set_error(MTP_INVALID_ARG, msg); }

int check_release(const mtp_window_release_args* a) {
  if (!a) return fail("kv_window_release: args is NULL");
  if (a->B < 0) return fail("kv_window_release: B < 0");
  if (a->block_size != MTP_BLOCK_SIZE) return fail("kv_window_release: block_size must be 64");
  if (a->max_blocks <= 0 || a->max_blocks > (1 << 24) || a->free_capacity < 0)
    return fail("kv_window_release: max_blocks outside [1, 2^24], or free_capacity < 0");
  if (a->window < 1 || a->sinks < 0) return fail("kv_window_release: window must be >= 1 and sinks >= 0");
  if (a->B == 0) return MTP_OK;
  if (!a->block_table || !a->seq_lens || !a->free_list || !a->free_count)
    return fail("kv_window_release: a required pointer is NULL");
  if (!a->workspace || a->workspace_bytes < ((size_t)a->B + 1) * sizeof(int32_t))
    return fail("kv_window_release: workspace too small (mtp_window_release_workspace_size)");
  if ((uintptr_t)a->workspace % 256) return fail("workspace must be 256-byte aligned");
  return MTP_OK;
}

}  // namespace
}  // namespace mtp

extern "C" {

size_t mtp_window_release_workspace_size(int32_t B) {
  return B < 0 ? 0 : (((size_t)B + 1) * sizeof(int32_t) + 255) / 256 * 256;
}

int kv_window_release(const mtp_window_release_args* a, void* stream) {
  int rc = mtp::check_release(a);
  if (rc != MTP_OK) return rc;
  mtp::set_launch_count(0);
  if (a->B == 0) return MTP_OK;
  unsigned* err = nullptr;
  int sm_count = 0;
  if ((rc = mtp::device_context(&err, &sm_count)) != MTP_OK) return rc;
  const int slots = a->max_blocks * mtp::kBlock;
  const int window = std::min(a->window, slots + 1), sink_blocks = (std::min(a->sinks, slots) + mtp::kBlock - 1) / mtp::kBlock;
  int32_t* counts = static_cast<int32_t*>(a->workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  mtp::window_count_kernel<<<a->B, mtp::kThreads, 0, s>>>(a->block_table, a->seq_lens, a->free_count, window, sink_blocks,
                                                         a->max_blocks, counts, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return mtp::set_cuda_error(e, "window release launch");
  mtp::window_move_kernel<<<a->B, mtp::kThreads, 0, s>>>(a->block_table, a->seq_lens, a->free_list, a->free_count, window,
                                                        sink_blocks, a->max_blocks, a->free_capacity, counts, err);
  if ((e = cudaGetLastError()) != cudaSuccess) return mtp::set_cuda_error(e, "window release launch");
  mtp::set_launch_count(2);
  return MTP_OK;
}

}  // extern "C"
