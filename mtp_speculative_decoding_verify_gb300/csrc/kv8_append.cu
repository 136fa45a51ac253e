// mtp_kv8_append: K/V of a ragged batch of new tokens into the 8-bit paged
// cache (and, with R tokens a request, the append of mtp_verify_attention_kv8).
//
// "Multi Token Prediction" note, overall flow for K=3 draft tokens, step 2:
// the new tokens' K/V are written to the cache the next queries read. The
// pages keep the cache in the model's type; here a block's head is held as
// e4m3 bytes times one scale.
//
// One team of threads per (request, block, KV head, K or V): it reads the
// tokens of its block once, 16 bytes a lane, keeps them in registers while
// the largest magnitude is reduced, and writes the bytes. Every (block, head)
// has one team, so the scale needs no atomics and the result no order.
// A team is a warp when a request appends at most 16 tokens (verify: 16
// tokens x 128 values are 64 values a lane) and four warps otherwise.
//
// It should be bound by the bytes, and is by what it issues for each: the
// maximum is taken over magnitude bits, two bf16 at once, and what is not
// finite or needs a division takes a loop of its own that reads the values
// again. Prefill of 64 requests, 64k tokens: 130 us with both in the one
// pass, 67 us so, 86 % of the copy rate (fp32: 104 us, 92 %); a step's append
// takes 4 us. (Several units a team, the next one's values on their way: 147 us.
// The registers cost more warps than the chain of loads before a unit's values
// does.)
#include "kernels.h"
#include "kv8.cuh"

namespace mtp {
int device_context(unsigned** err, int* sm_count);
int set_error(int code, const char* msg);
int set_cuda_error(cudaError_t e, const char* what);
void set_launch_count(int n);

namespace {

constexpr int kThreads = 128;

template <typename T> struct Vec;   // 16 bytes of T as floats
template <> struct Vec<float> {
  static constexpr int N = 4;
  // The largest magnitude bits so far with those of w, and the largest of
  // both as a float; above kFinite something is not finite.
  static constexpr uint32_t kFinite = 0x7f7fffffu;
  __device__ __forceinline__ static uint32_t most(uint32_t m, const uint4& w) {
    return max(max(max(m, w.x & 0x7fffffffu), max(w.y & 0x7fffffffu, w.z & 0x7fffffffu)), w.w & 0x7fffffffu);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
  __device__ __forceinline__ static void unpack(const uint4& w, float (&f)[N]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kFinite = 0x7f7fffffu;
  __device__ __forceinline__ static uint32_t most(uint32_t m, const uint4& w) {   // two halves
    return __vmaxu2(__vmaxu2(__vmaxu2(m, w.x & 0x7fff7fffu), __vmaxu2(w.y & 0x7fff7fffu, w.z & 0x7fff7fffu)), w.w & 0x7fff7fffu);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  __device__ __forceinline__ static void unpack(const uint4& w, float (&f)[N]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
};

struct AppendParams {
  const void *k_new, *v_new;
  const int32_t* starts;       // [B+1] token offsets, nullptr: `uniform` tokens each
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const int32_t *block_table, *ctx_lens;
  int T, B, Hkv, uniform, max_blocks, num_blocks;
  long long units;             // teams of the grid that have work to look for
  unsigned* err;
  WindowSchedule schedule;     // for the last CTA, when asked for
};

// The request that slot `piece` of the piece numbering belongs to. A request
// of n tokens touches at most n/64 + 2 blocks, so numbering its blocks from
// starts[b]/64 + 2b leaves no two requests the same number, and b is the
// count of requests whose number is at most `piece` (less one).
__device__ __forceinline__ int piece_request(const AppendParams& p, int piece, int* first) {
  if (p.starts == nullptr) {   // at most 16 tokens: two blocks
    *first = piece / 2 * 2;
    return piece / 2;
  }
  // 32-ary search: every warp does it by itself
  const int lane = threadIdx.x % kWarp;
  int lo = 0, hi = p.B;        // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + kWarp - 1) / kWarp;
    const int b = lo + lane * step;
    const bool le = b < hi && (p.starts[b] >> 6) + 2 * b <= piece;
    const unsigned m = __ballot_sync(0xffffffffu, le || lane == 0);
    const int last = 31 - __clz(m);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  *first = (p.starts[lo] >> 6) + 2 * lo;
  return lo;
}

template <typename T, int D, int TEAM>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const AppendParams p) {
  constexpr int VE = Vec<T>::N;
  constexpr int LANES = D / VE;              // lanes a token row takes
  constexpr int ROWS = TEAM / LANES;         // rows of a pass
  constexpr int TOKENS = TEAM == kWarp ? kMaxRows : kBlock;
  constexpr int PASSES = (TOKENS + ROWS - 1) / ROWS;
  static_assert(TEAM % LANES == 0 && ROWS >= 1, "a token row is read by one team");
  __shared__ float s_max[kThreads / kWarp];
  const int tid = threadIdx.x % TEAM;
  asm volatile("griddepcontrol.launch_dependents;");   // (an attention behind it may set up)

  if (p.schedule.prefix != nullptr && blockIdx.x == gridDim.x - 1) {
    window_schedule<kThreads>(p.schedule);
    return;
  }
  if (p.starts != nullptr && blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      const int s0 = p.starts[b], s1 = p.starts[b + 1];
      if (s0 < 0 || s1 < s0 || s1 > p.T) raise_error(p.err, MTP_ERR_LENGTH);
    }
  }
  const long long unit = (long long)blockIdx.x * (kThreads / TEAM) + threadIdx.x / TEAM;
  // Everything up to the reduction depends on the unit alone: a team leaves whole.
  if (unit >= p.units) return;
  const bool is_v = unit & 1;
  const int h = (int)((unit >> 1) % p.Hkv);
  const int piece = (int)((unit >> 1) / p.Hkv);
  int first;
  const int b = piece_request(p, piece, &first);
  if (b >= p.B) return;
  const int s0 = p.starts ? p.starts[b] : b * p.uniform;
  const int n = (p.starts ? p.starts[b + 1] : s0 + p.uniform) - s0;
  if (s0 < 0 || n <= 0 || n > p.T - s0) return;   // empty, or flagged above
  const int ctx = p.ctx_lens[b];
  if (ctx < 0 || (long long)ctx + n > (long long)p.max_blocks * kBlock) {
    if (tid == 0) raise_error(p.err, MTP_ERR_LENGTH);
    return;
  }
  const int i = ctx / kBlock + (piece - first);
  if (piece < first || i > (ctx + n - 1) / kBlock) return;
  const int blk = p.block_table[(int64_t)b * p.max_blocks + i];
  if (blk < 0 || blk >= p.num_blocks) {
    if (tid == 0) raise_error(p.err, MTP_ERR_BLOCK_ID);
    return;
  }
  const int lo = max(ctx, i * kBlock), cnt = min(ctx + n, (i + 1) * kBlock) - lo, off = lo - i * kBlock;
  float* scale = (is_v ? p.v_scale : p.k_scale) + (int64_t)blk * p.Hkv + h;
  const float old = *scale;
  if (off > 0 && !scale_ok(old)) {
    if (tid == 0) raise_error(p.err, MTP_ERR_SCALE);
    return;
  }
  const int row = p.Hkv * D;                   // elements from a token to the next (64 rows fit 31 bits)
  const int r0 = tid / LANES, e0 = tid % LANES * VE;
  const T* src = static_cast<const T*>(is_v ? p.v_new : p.k_new) + (int64_t)(s0 + lo - ctx + r0) * row + h * D + e0;
  uint8_t* block = (is_v ? p.v_cache : p.k_cache) + ((int64_t)blk * kBlock) * row + h * D;
  uint8_t* dst = block + (off + r0) * row + e0;

  uint4 w[PASSES];
#pragma unroll
  for (int y = 0; y < PASSES; ++y)
    w[y] = y * ROWS + r0 < cnt ? __ldg(reinterpret_cast<const uint4*>(src + y * ROWS * row)) : make_uint4(0, 0, 0, 0);
  uint32_t top = 0;
#pragma unroll
  for (int y = 0; y < PASSES; ++y) top = Vec<T>::most(top, w[y]);
  top = Vec<T>::bits(top);
  bool finite = top <= Vec<T>::kFinite;
  float a = __uint_as_float(top);
  if (!finite) {                               // the largest of the finite ones
    a = 0.0f;
#pragma unroll 1
    for (int r = r0; r < cnt; r += ROWS) {
      float f[VE];
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(src + (r - r0) * row)), f);
#pragma unroll
      for (int e = 0; e < VE; ++e) a = fmaxf(a, fabsf(f[e]) <= FLT_MAX ? fabsf(f[e]) : 0.0f);
    }
  }
  a = warp_max(a);
  if (TEAM > kWarp) {
    if (threadIdx.x % kWarp == 0) s_max[threadIdx.x / kWarp] = a;
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kThreads / kWarp; ++y) a = fmaxf(a, s_max[y]);
  } else {
    __syncwarp();
  }
  int grow;
  const float s = grown_scale(old, off == 0, a, &grow);
  if (tid == 0) *scale = s;                    // every thread has read the old one
  if (off > 0 && grow > 0) {                   // the kept slots, to the new scale
    const float f = ldexpf(1.0f, -grow);
#pragma unroll 1
    for (int x = tid; x < off * (D / 4); x += TEAM) {
      uint32_t* at = reinterpret_cast<uint32_t*>(block + x / (D / 4) * row) + x % (D / 4);
      const float4 v = e4m3x4_to_f(*at);
      *at = f_to_e4m3x4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
  }
  auto store = [&](const float (&f)[VE], int y) {
    uint32_t* to = reinterpret_cast<uint32_t*>(dst + y * ROWS * row);
    if constexpr (VE == 8) {
      *reinterpret_cast<uint2*>(to) = make_uint2(f_to_e4m3x4(f[0], f[1], f[2], f[3]), f_to_e4m3x4(f[4], f[5], f[6], f[7]));
    } else {
      *to = f_to_e4m3x4(f[0], f[1], f[2], f[3]);
    }
  };
  // x / s to nearest: for a power of two (every scale this kernel began)
  // x * (1 / s) is the same number, without the division's cost.
  if (finite && (__float_as_uint(s) & 0x7fffffu) == 0) {
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));   // 1 / s
#pragma unroll
    for (int y = 0; y < PASSES; ++y) {
      if (y * ROWS + r0 >= cnt) break;
      float f[VE];
      Vec<T>::unpack(w[y], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] *= inv;
      store(f, y);
    }
  } else {
#pragma unroll 1
    for (int y = 0; y * ROWS + r0 < cnt; ++y) {
      float f[VE];
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(src + y * ROWS * row)), f);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        f[e] = fabsf(f[e]) <= FLT_MAX ? f[e] / s : __uint_as_float(0x7fffffffu);   // not finite: NaN, not 448
      store(f, y);
    }
  }
}

template <typename T, int D>
cudaError_t run_append(const AppendParams& p, cudaStream_t s) {
  if (p.starts == nullptr) {
    const long long grid = (p.units + kThreads / kWarp - 1) / (kThreads / kWarp) + (p.schedule.prefix ? 1 : 0);
    kv8_append_kernel<T, D, kWarp><<<(unsigned)grid, kThreads, 0, s>>>(p);
  } else {
    kv8_append_kernel<T, D, kThreads><<<(unsigned)p.units, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

int fail(const char* msg) { return set_error(MTP_INVALID_ARG, msg); }

int check_append(const mtp_kv8_append_args* a) {
  if (!a) return fail("mtp_kv8_append: args is NULL");
  if (a->B < 0 || a->T < 0) return fail("mtp_kv8_append: B and T must be >= 0");
  if (a->block_size != MTP_BLOCK_SIZE) return fail("mtp_kv8_append: block_size must be 64");
  if (a->max_blocks <= 0 || a->max_blocks > (1 << 24) || a->num_blocks <= 0)
    return fail("mtp_kv8_append: max_blocks outside [1, 2^24], or num_blocks <= 0");
  if (a->Hkv <= 0 || a->Hkv > (1 << 16)) return fail("mtp_kv8_append: Hkv outside [1, 2^16]");
  if (a->dtype != MTP_F32 && a->dtype != MTP_BF16) return fail("mtp_kv8_append: dtype");
  if (a->d != 64 && a->d != 128) return set_error(MTP_UNSUPPORTED, "mtp_kv8_append: head dim must be 64 or 128");
  if (a->B == 0 || a->T == 0) return MTP_OK;
  if (!a->k_new || !a->v_new || !a->starts || !a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale ||
      !a->block_table || !a->ctx_lens)
    return fail("mtp_kv8_append: a required pointer is NULL");
  const uintptr_t any = (uintptr_t)a->k_new | (uintptr_t)a->v_new | (uintptr_t)a->k_cache | (uintptr_t)a->v_cache;
  if (any % 16) return fail("mtp_kv8_append: k_new, v_new and the caches must be 16-byte aligned");
  if (((long long)a->T / kBlock + 2ll * a->B + 1) * a->Hkv * 2 > 0x7fffffffll)
    return set_error(MTP_UNSUPPORTED, "mtp_kv8_append: (T/64 + 2B) x Hkv x 2 exceeds 2^31");
  return MTP_OK;
}

}  // namespace

cudaError_t launch_kv8_append(const mtp_kv8_append_args& a, int uniform, const WindowSchedule& sch, unsigned* err,
                              cudaStream_t s) {
  AppendParams p;
  p.k_new = a.k_new;
  p.v_new = a.v_new;
  p.starts = uniform > 0 ? nullptr : a.starts;
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.T = a.T;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.uniform = uniform;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.err = err;
  p.schedule = sch;
  const long long pieces = uniform > 0 ? 2ll * a.B : (long long)a.T / kBlock + 2ll * a.B;
  p.units = pieces * a.Hkv * 2;
  if (a.dtype == MTP_BF16)
    return a.d == 128 ? run_append<__nv_bfloat16, 128>(p, s) : run_append<__nv_bfloat16, 64>(p, s);
  return a.d == 128 ? run_append<float, 128>(p, s) : run_append<float, 64>(p, s);
}

}  // namespace mtp

extern "C" int mtp_kv8_append(const mtp_kv8_append_args* a, void* stream) {
  int rc = mtp::check_append(a);
  if (rc != MTP_OK) return rc;
  mtp::set_launch_count(0);
  if (a->B == 0 || a->T == 0) return MTP_OK;
  unsigned* err = nullptr;
  int sm_count = 0;
  if ((rc = mtp::device_context(&err, &sm_count)) != MTP_OK) return rc;
  const cudaError_t e = mtp::launch_kv8_append(*a, 0, mtp::WindowSchedule{}, err, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return mtp::set_cuda_error(e, "8-bit append launch");
  mtp::set_launch_count(1);
  return MTP_OK;
}
