// Verify attention behind a window and over the 8-bit cache: the C entries,
// the plan, the SIMT kernel (fp32) and the merge of split results.
//
// "Multi Token Prediction" note, overall flow for K=3 draft tokens, step 2,
// as in mtp_verify_attention: the R verify rows of a request attend the
// reused cache and each other causally. Two things differ here. A row may be
// held to the last `window` positions and the first `sinks` tokens; only the
// blocks that some row sees (page_span) are read, so the table may hold -1
// for the others. And the cache may hold e4m3 bytes with a scale for each
// block and KV head.
#include <math.h>
#include <stdio.h>

#include <algorithm>

#include "attention_window.h"
#include "kv8.cuh"

namespace mtp {
int device_context(unsigned** err, int* sm_count);
int set_error(int code, const char* msg);
int set_cuda_error(cudaError_t e, const char* what);
void set_launch_count(int n);

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------- append
// One CTA per (request, verify token): its K and V rows go to slot ctx+j of
// the cache, 16 bytes a thread. A chain of three loads bounds it, not bytes
// (about 2 us, as the 8-bit append of such a step).
__global__ void __launch_bounds__(128) window_append_kernel(const uint4* __restrict__ k_new,
                                                            const uint4* __restrict__ v_new, uint4* __restrict__ k_cache,
                                                            uint4* __restrict__ v_cache,
                                                            const int32_t* __restrict__ block_table,
                                                            const int32_t* __restrict__ ctx_lens, int R, int vecs,
                                                            int max_blocks, int num_blocks, unsigned* err,
                                                            const WindowSchedule schedule) {
  asm volatile("griddepcontrol.launch_dependents;");   // (the attention behind it may set up)
  if (schedule.prefix != nullptr && blockIdx.x == gridDim.x - 1) {
    window_schedule<128>(schedule);
    return;
  }
  const int b = blockIdx.x / R, j = blockIdx.x % R;
  const int ctx = ctx_lens[b];
  if (ctx < 0 || ctx > max_blocks * kBlock - R) {
    if (threadIdx.x == 0) raise_error(err, MTP_ERR_LENGTH);
    return;
  }
  const int blk = block_table[(int64_t)b * max_blocks + (ctx + j) / kBlock];
  if (blk < 0 || blk >= num_blocks) {
    if (threadIdx.x == 0) raise_error(err, MTP_ERR_BLOCK_ID);
    return;
  }
  const int64_t from = (int64_t)blockIdx.x * vecs, to = ((int64_t)blk * kBlock + (ctx + j) % kBlock) * vecs;
  for (int i = threadIdx.x; i < vecs; i += 128) {
    k_cache[to + i] = k_new[from + i];
    v_cache[to + i] = v_new[from + i];
  }
}

// -------------------------------------------------------------------- SIMT
// One CTA takes up to 16 query rows of one KV head and one range of the
// request's pages. A page's K and V are staged in shared memory as fp32 (K
// rows padded by 16 bytes, so that 8 lanes reading 16 bytes of 8 keys hit
// all banks). A warp owns two rows: for the scores each lane takes two keys,
// for the output each lane D/32 values of the row. Sums and statistics are
// fp32. Shared memory bounds it: each of a warp's rows reads K and V by itself
// (fp32 is the type of checks and small models; 32 requests of 1k-4k tokens, 16
// rows, 8 KV heads: 568 us, 9.5 TFLOP/s), and with little work the launches (4
// requests of 128 tokens: 12.9 us, of which the append is 4).
constexpr int kSimtRows = 16, kSimtWarps = 8;

template <typename T> struct KvLoad;
template <> struct KvLoad<float> {
  __device__ __forceinline__ static float4 get(const void* base, int64_t elem) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
  }
};
template <> struct KvLoad<uint8_t> {
  __device__ __forceinline__ static float4 get(const void* base, int64_t elem) {
    return e4m3x4_to_f(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + elem));
  }
};

template <int D>
constexpr int simt_smem_bytes() {
  return (kBlock * (D + 4) + kBlock * D + kSimtRows * D) * (int)sizeof(float);
}

template <typename T, typename KV, int D>
__global__ void __launch_bounds__(kSimtWarps* kWarp) window_simt_kernel(const WindowParams p) {
  constexpr int E = D / kWarp;
  extern __shared__ float smem[];
  float* ks = smem;                          // [64][D + 4]
  float* vs = ks + kBlock * (D + 4);         // [64][D]
  float* qs = vs + kBlock * D;               // [16][D]
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int split = blockIdx.y;
  const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x % p.Hkv;
  const int row0 = blockIdx.z * kSimtRows;
  const int ctx = p.ctx_lens[b];
  if (ctx < 0 || ctx > p.max_blocks * kBlock - p.R) {
    if (threadIdx.x == 0 && split == 0) raise_error(p.err, MTP_ERR_LENGTH);
    return;
  }
  const PageSpan span = page_span(ctx, p.R, p.window, p.sinks);
  const int i0 = (int)((int64_t)span.n * split / p.n_splits), i1 = (int)((int64_t)span.n * (split + 1) / p.n_splits);

  int64_t orow[2];
  int pos[2];
  bool live[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = row0 + warp + x * kSimtWarps;
    live[x] = r < p.rows;
    const int rc = min(r, p.rows - 1);
    pos[x] = ctx + rc / p.group;
    orow[x] = ((int64_t)b * p.R + rc / p.group) * p.Hq + kvh * p.group + rc % p.group;
    for (int e = lane; e < D; e += kWarp)
      qs[(warp + x * kSimtWarps) * D + e] = Num<T>::to_f(static_cast<const T*>(p.q)[orow[x] * D + e]);
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[2][E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[0][e] = o[1][e] = 0.0f;

  for (int i = i0; i < i1; ++i) {
    const int page = span.page(i);
    const int blk = p.block_table[(int64_t)b * p.max_blocks + page];
    if (blk < 0 || blk >= p.num_blocks) {      // the same for every thread
      if (threadIdx.x == 0) raise_error(p.err, MTP_ERR_BLOCK_ID);
      continue;
    }
    float sk = 1.0f, sv = 1.0f;
    if (p.k_scale != nullptr) {
      sk = p.k_scale[(int64_t)blk * p.Hkv + kvh];
      sv = p.v_scale[(int64_t)blk * p.Hkv + kvh];
      if (!scale_ok(sk) || !scale_ok(sv)) {
        if (threadIdx.x == 0) raise_error(p.err, MTP_ERR_SCALE);
        continue;
      }
    }
    // Only the slots between the first and the last that a row sees are read
    // (116 requests of 22 tokens, window 3: 57.0 us with whole pages, 28.4 us so).
    const int edge = p.window == 0 || page * kBlock < p.sinks ? 0 : ctx - p.window + 1 - page * kBlock;
    const int k0 = max(edge, 0), k1 = min(kBlock, ctx + p.R - page * kBlock);
    __syncthreads();                           // the last page has been read
    auto stage = [&](int x) {
      const int key = x / (D / 4), c = x % (D / 4) * 4;
      const int64_t elem = (((int64_t)blk * kBlock + key) * p.Hkv + kvh) * D + c;
      float4 k = KvLoad<KV>::get(p.k_cache, elem), v = KvLoad<KV>::get(p.v_cache, elem);
      k.x *= sk, k.y *= sk, k.z *= sk, k.w *= sk;
      v.x *= sv, v.y *= sv, v.z *= sv, v.w *= sv;
      *reinterpret_cast<float4*>(ks + key * (D + 4) + c) = k;
      *reinterpret_cast<float4*>(vs + key * D + c) = v;
    };
    if (k1 - k0 == kBlock) {
      for (int x = threadIdx.x; x < kBlock * (D / 4); x += kSimtWarps * kWarp) stage(x);
    } else {
      for (int x = k0 * (D / 4) + threadIdx.x; x < k1 * (D / 4); x += kSimtWarps * kWarp) stage(x);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!live[x]) continue;
      const float* q = qs + (warp + x * kSimtWarps) * D;
      float s[2] = {0.0f, 0.0f};
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        const float4 a = *reinterpret_cast<const float4*>(q + c);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float4 k = *reinterpret_cast<const float4*>(ks + (lane + y * kWarp) * (D + 4) + c);
          s[y] += a.x * k.x + a.y * k.y + a.z * k.z + a.w * k.w;
        }
      }
      // A slot the row may not see takes no part: not its score, and not its
      // value either (0 x NaN would spread from a stale slot).
      unsigned see[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const bool vis = slot_visible(page * kBlock + lane + y * kWarp, pos[x], p.window, p.sinks);
        see[y] = __ballot_sync(0xffffffffu, vis);
        s[y] = vis ? s[y] * p.sm_scale : -INFINITY;
      }
      const float mn = fmaxf(fmaxf(m[x], (see[0] | see[1]) != 0 ? kNoWeight : -INFINITY), warp_max(fmaxf(s[0], s[1])));
      const float base = mn == -INFINITY ? 0.0f : mn;
      const float c = expf(m[x] - base);
      const float p0 = expf(s[0] - base), p1 = expf(s[1] - base);
      m[x] = mn;
      l[x] = l[x] * c + warp_sum(p0 + p1);
#pragma unroll
      for (int e = 0; e < E; ++e) o[x][e] *= c;
      const float* v = vs + lane * E;
      if ((see[0] & see[1]) == 0xffffffffu) {
#pragma unroll 8
        for (int key = 0; key < kWarp; ++key) {
          const float w0 = __shfl_sync(0xffffffffu, p0, key), w1 = __shfl_sync(0xffffffffu, p1, key);
#pragma unroll
          for (int e = 0; e < E; ++e) o[x][e] += w0 * v[key * D + e] + w1 * v[(key + kWarp) * D + e];
        }
      } else {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          for (unsigned left = see[y]; left != 0; left &= left - 1) {
            const int key = __ffs(left) - 1;
            const float w = __shfl_sync(0xffffffffu, y == 0 ? p0 : p1, key);
#pragma unroll
            for (int e = 0; e < E; ++e) o[x][e] += w * v[(key + y * kWarp) * D + e];
          }
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    if (!live[x]) continue;
    // no weight: nothing seen (bad blocks only), or -inf only
    const float inv = l[x] != 0.0f ? 1.0f / l[x] : m[x] == -INFINITY || p.n_splits > 1 ? 0.0f : NAN;
    if (p.n_splits == 1) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        static_cast<T*>(p.out)[orow[x] * D + lane * E + e] = Num<T>::from_f(o[x][e] * inv);
    } else {
      float* po = p.part_o + (orow[x] * p.n_splits + split) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) po[e] = o[x][e] * inv;
      if (lane == 0) p.part_lse[orow[x] * p.n_splits + split] = l[x] == 0.0f ? m[x] : (m[x] + logf(l[x])) * kLog2e;
    }
  }
}

// out = sum_s 2^(lse_s - max) part_s / sum_s 2^(lse_s - max): one warp a row
// (few rows, a launch's latency bounds it). A part that saw nothing is left
// out; one of -inf scores has weight 0, and hands a NaN of V on.
template <typename T, int D>
__global__ void __launch_bounds__(128) window_merge_kernel(const WindowParams p, int64_t n_rows) {
  constexpr int E = D / kWarp;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / kWarp;
  if (row >= n_rows) return;
  const int lane = threadIdx.x % kWarp;
  const int ctx = p.ctx_lens[row / ((int64_t)p.R * p.Hq)];
  if (ctx < 0 || ctx > p.max_blocks * kBlock - p.R) return;   // flagged; its rows stay as they were
  const float* lse = p.part_lse + row * p.n_splits;
  float m = -INFINITY;
  for (int s = lane; s < p.n_splits; s += kWarp) m = fmaxf(m, lse[s]);
  m = warp_max(m);
  float o[E], l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int s = 0; s < p.n_splits; ++s) {
    const float x = lse[s];
    if (x == -INFINITY) continue;
    const float w = exp2f(x - m);
    l += w;
    const float* po = p.part_o + (row * p.n_splits + s) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += w * po[e];
  }
  const float inv = m == -INFINITY && l == 0.0f ? 0.0f : m == kNoWeight ? NAN : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) static_cast<T*>(p.out)[row * D + lane * E + e] = Num<T>::from_f(o[e] * inv);
}

template <typename T, typename KV, int D>
cudaError_t run_simt(const WindowParams& p, cudaStream_t s, int* launches) {
  const int smem = simt_smem_bytes<D>();
  cudaError_t e = cudaFuncSetAttribute(window_simt_kernel<T, KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.B * p.Hkv, p.n_splits, (p.rows + kSimtRows - 1) / kSimtRows);
  window_simt_kernel<T, KV, D><<<grid, kSimtWarps * kWarp, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  *launches = 1;
  return cudaSuccess;
}

template <typename T, int D>
cudaError_t run_merge(const WindowParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.B * p.R * p.Hq;
  window_merge_kernel<T, D><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(p, rows);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt(const WindowParams& p, int d, bool kv8, cudaStream_t s, int* launches) {
  cudaError_t e;
  if (kv8) e = d == 128 ? run_simt<T, uint8_t, 128>(p, s, launches) : run_simt<T, uint8_t, 64>(p, s, launches);
  else e = d == 128 ? run_simt<T, T, 128>(p, s, launches) : run_simt<T, T, 64>(p, s, launches);
  if (e != cudaSuccess || p.n_splits == 1) return e;
  *launches += 1;
  return d == 128 ? run_merge<T, 128>(p, s) : run_merge<T, 64>(p, s);
}

// ----------------------------------------------------------- checks and plan
int fail(const char* name, const char* msg) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", name, msg);
  return set_error(MTP_INVALID_ARG, buf);
}

int check_window(const mtp_window_attn_args* a, bool kv8) {
  const char* name = kv8 ? "mtp_verify_attention_kv8" : "mtp_verify_attention_window";
  if (!a) return fail(name, "args is NULL");
  if (a->B < 0) return fail(name, "B < 0");
  if (a->D < 0 || a->D > MTP_MAX_DRAFTS) return fail(name, "D outside [0, 15]");
  if (a->block_size != MTP_BLOCK_SIZE) return fail(name, "block_size must be 64");
  if (a->max_blocks <= 0 || a->max_blocks > (1 << 24) || a->num_blocks <= 0)
    return fail(name, "max_blocks outside [1, 2^24], or num_blocks <= 0");
  if (a->Hq <= 0 || a->Hkv <= 0 || a->Hkv > (1 << 16) || a->Hq % a->Hkv) return fail(name, "Hkv outside [1, 2^16], or Hq % Hkv != 0");
  if (a->dtype != MTP_F32 && a->dtype != MTP_BF16) return fail(name, "dtype");
  if (!(a->sm_scale > 0.0f && a->sm_scale <= 1e30f)) return fail(name, "sm_scale must be > 0 and finite");
  if (a->window < (kv8 ? 0 : 1)) return fail(name, kv8 ? "window must be >= 0" : "window must be >= 1");
  if (a->sinks < 0) return fail(name, "sinks must be >= 0");
  if (a->window == 0 && a->sinks > 0) return fail(name, "sinks need a window");
  if (a->d != 64 && a->d != 128) {
    char buf[128];
    snprintf(buf, sizeof buf, "%s: head dim must be 64 or 128", name);
    return set_error(MTP_UNSUPPORTED, buf);
  }
  if ((long long)a->B * (a->D + 1) * a->Hq > (1 << 29) || a->Hq / a->Hkv > (1 << 15)) {
    char buf[128];
    snprintf(buf, sizeof buf, "%s: B x R x Hq > 2^29, or Hq / Hkv > 2^15", name);
    return set_error(MTP_UNSUPPORTED, buf);
  }
  if ((long long)a->B * a->max_blocks > 0x7fffffffll) {
    char buf[128];
    snprintf(buf, sizeof buf, "%s: B x max_blocks >= 2^31", name);
    return set_error(MTP_UNSUPPORTED, buf);
  }
  if (a->B == 0) return MTP_OK;
  if (!a->q || !a->k_new || !a->v_new || !a->k_cache || !a->v_cache || !a->block_table || !a->ctx_lens || !a->out)
    return fail(name, "a required pointer is NULL");
  if (kv8 && (!a->k_scale || !a->v_scale)) return fail(name, "k_scale / v_scale is NULL");
  if (!kv8 && (a->k_scale || a->v_scale)) return fail(name, "k_scale and v_scale must be NULL");
  const uintptr_t any = (uintptr_t)a->q | (uintptr_t)a->k_new | (uintptr_t)a->v_new | (uintptr_t)a->k_cache |
                        (uintptr_t)a->v_cache | (uintptr_t)a->out;
  if (any % 16) return fail(name, "q, out, k_new, v_new and the caches must be 16-byte aligned");
  return MTP_OK;
}

// The tensor cores take bf16 rows, the SIMT kernel fp32 ones.
bool uses_mma(const mtp_window_attn_args& a) { return a.dtype == MTP_BF16; }

WindowPlan plan_window(const mtp_window_attn_args& a, bool kv8, int sm_count) {
  if (uses_mma(a)) return kv8 ? plan_kv8_tc(a, sm_count) : plan_window_mma(a, sm_count);
  WindowPlan p{};
  const int rows = a.Hq / a.Hkv * (a.D + 1);
  const long long ctas = (long long)a.B * a.Hkv * ((rows + kSimtRows - 1) / kSimtRows);
  // Two CTAs an SM where the batch alone has fewer, and at least four pages a
  // split (about what the merge's launch costs).
  const long long pages = a.window == 0 ? a.max_blocks
                                        : std::min<long long>(a.max_blocks, ((long long)a.window + a.sinks) / kBlock + 3);
  const long long want = std::max<long long>(1, (2ll * sm_count + ctas - 1) / std::max(ctas, 1ll));
  p.n_splits = (int)std::max<long long>(1, std::min({want, pages / 4, 64ll}));
  p.ws_bytes = 256;
  if (p.n_splits > 1) {
    const size_t n = (size_t)a.B * (a.D + 1) * a.Hq * p.n_splits;
    p.ws_partial_o = 0;
    p.ws_partial_lse = n * a.d * sizeof(float);
    p.ws_bytes = (p.ws_partial_lse + n * sizeof(float) + 255) / 256 * 256;
  }
  return p;
}

size_t workspace_size(const mtp_window_attn_args* a, bool kv8) {
  if (check_window(a, kv8) != MTP_OK) return 0;
  unsigned* err = nullptr;
  int sm_count = 0;
  if (device_context(&err, &sm_count) != MTP_OK) return 0;
  return plan_window(*a, kv8, sm_count).ws_bytes;
}

cudaError_t append(const mtp_window_attn_args& a, bool kv8, const WindowSchedule& sch, unsigned* err, cudaStream_t s) {
  if (kv8) {
    mtp_kv8_append_args k{};
    k.k_new = a.k_new;
    k.v_new = a.v_new;
    k.k_cache = a.k_cache;
    k.v_cache = a.v_cache;
    k.k_scale = a.k_scale;
    k.v_scale = a.v_scale;
    k.block_table = a.block_table;
    k.ctx_lens = a.ctx_lens;
    k.T = a.B * (a.D + 1);
    k.B = a.B;
    k.Hkv = a.Hkv;
    k.d = a.d;
    k.max_blocks = a.max_blocks;
    k.num_blocks = a.num_blocks;
    k.dtype = a.dtype;
    return launch_kv8_append(k, a.D + 1, sch, err, s);
  }
  const int vecs = a.Hkv * a.d * (a.dtype == MTP_BF16 ? 2 : 4) / 16;
  window_append_kernel<<<a.B * (a.D + 1) + (sch.prefix ? 1 : 0), 128, 0, s>>>(
      (const uint4*)a.k_new, (const uint4*)a.v_new, (uint4*)a.k_cache, (uint4*)a.v_cache, a.block_table, a.ctx_lens,
      a.D + 1, vecs, a.max_blocks, a.num_blocks, err, sch);
  return cudaGetLastError();
}

int attend(const mtp_window_attn_args* a, bool kv8, void* stream) {
  int rc = check_window(a, kv8);
  if (rc != MTP_OK) return rc;
  set_launch_count(0);
  if (a->B == 0) return MTP_OK;
  unsigned* err = nullptr;
  int sm_count = 0;
  if ((rc = device_context(&err, &sm_count)) != MTP_OK) return rc;
  const WindowPlan pl = plan_window(*a, kv8, sm_count);
  if (!a->workspace || a->workspace_bytes < pl.ws_bytes) {
    char buf[160];
    snprintf(buf, sizeof buf, "workspace of %zu bytes needed, %zu given", pl.ws_bytes, a->workspace ? a->workspace_bytes : (size_t)0);
    return set_error(MTP_INVALID_ARG, buf);
  }
  if ((uintptr_t)a->workspace % 256) return set_error(MTP_INVALID_ARG, "workspace must be 256-byte aligned");
  WindowParams p{};
  p.q = a->q;
  p.out = a->out;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.block_table = a->block_table;
  p.ctx_lens = a->ctx_lens;
  p.err = err;
  p.B = a->B;
  p.R = a->D + 1;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.group = a->Hq / a->Hkv;
  p.rows = p.group * p.R;
  p.max_blocks = a->max_blocks;
  p.num_blocks = a->num_blocks;
  // past these bounds a window or sinks hide nothing; the kernels add to them
  p.window = std::min(a->window, a->max_blocks * kBlock + kMaxRows);
  p.sinks = std::min(a->sinks, a->max_blocks * kBlock);
  p.n_splits = pl.n_splits;
  p.sm_scale = a->sm_scale;
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + pl.ws_partial_o);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + pl.ws_partial_lse);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto record = [&](void* ev) { return ev ? cudaEventRecord(static_cast<cudaEvent_t>(ev), s) : cudaSuccess; };
  WindowSchedule sch{};
  const bool mma = uses_mma(*a);
  if (mma) {
    p.row_tiles = pl.row_tiles;
    p.row_warps = pl.row_warps;
    p.key_parts = pl.key_parts;
    p.stages = pl.stages;
    sch.prefix = reinterpret_cast<int32_t*>(static_cast<char*>(a->workspace) + pl.ws_prefix);
    sch.shares = reinterpret_cast<Share*>(static_cast<char*>(a->workspace) + pl.ws_shares);
    sch.sharers = reinterpret_cast<int2*>(static_cast<char*>(a->workspace) + pl.ws_sharers);
    sch.arrived = reinterpret_cast<int32_t*>(static_cast<char*>(a->workspace) + pl.ws_arrived);
    sch.ctas = pl.ctas_per_head;
    sch.n_arrived = (int64_t)p.B * p.Hkv * pl.row_tiles * pl.row_warps;
    sch.ctx_lens = p.ctx_lens;
    sch.B = p.B;
    sch.R = p.R;
    sch.max_blocks = p.max_blocks;
    sch.window = p.window;
    sch.sinks = p.sinks;
    p.prefix = sch.prefix;
    p.shares = sch.shares;
    p.sharers = sch.sharers;
    p.arrived = sch.arrived;
  }
  cudaError_t e = append(*a, kv8, sch, err, s);
  if (e != cudaSuccess) return set_cuda_error(e, "kv append launch");
  if ((e = record(a->timing_events[0])) != cudaSuccess) return set_cuda_error(e, "cudaEventRecord");
  int launches = 0;
  if (mma) {
    launches = 1;
    e = kv8 ? launch_kv8_tc(*a, pl, p, s) : launch_window_mma(*a, pl, p, s);
  } else {
    e = launch_simt<float>(p, a->d, kv8, s, &launches);
  }
  if (e != cudaSuccess) return set_cuda_error(e, "attention launch");
  if ((e = record(a->timing_events[1])) != cudaSuccess) return set_cuda_error(e, "cudaEventRecord");
  set_launch_count(1 + launches);
  return MTP_OK;
}

}  // namespace
}  // namespace mtp

extern "C" {

size_t mtp_attention_kv8_workspace_size(const mtp_window_attn_args* a) { return mtp::workspace_size(a, true); }

int mtp_verify_attention_kv8(const mtp_window_attn_args* a, void* stream) { return mtp::attend(a, true, stream); }

size_t mtp_attention_window_workspace_size(const mtp_window_attn_args* a) { return mtp::workspace_size(a, false); }

int mtp_verify_attention_window(const mtp_window_attn_args* a, void* stream) { return mtp::attend(a, false, stream); }

}  // extern "C"
