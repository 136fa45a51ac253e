// mtp_kv_append: K/V rows of new tokens into the paged cache at the slots that
// kv_block_assign gives ("Multi Token Prediction" note, K=3 flow step 2: the
// new tokens' K/V are added to the cache that later queries reuse).
//
// A copy: each row is read once and written once, so bytes bound a prompt's
// call and two dependent reads (the slot, the row) a step's. A team of lanes
// takes a token, 16 bytes a lane and access, K and V side by side, so that
// eight loads of a lane are on their way for rows of 2 KB. 65536 tokens of 8 x
// 128: 78 us, the rate of a plain copy; 1024: 2.7 us.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mtp {
int device_context(unsigned** err, int* sm_count);
int set_error(int code, const char* msg);
int set_cuda_error(cudaError_t e, const char* what);
void set_launch_count(int n);

namespace {

constexpr int kThreads = 256;

struct SlotAppendParams {
  const uint4 *k_new, *v_new;
  const int64_t* slots;
  uint4 *k_cache, *v_cache;
  int64_t k_stride, v_stride, n_slots;   // 16-byte units from a token to the next; slots of the cache
  int T, k_vecs, v_vecs;                 // 16-byte units of a row (v: 0 without V)
  unsigned* err;
};

template <int TEAM>
__global__ void __launch_bounds__(kThreads) kv_slot_append_kernel(const SlotAppendParams p) {
  const long long t = (long long)blockIdx.x * (kThreads / TEAM) + threadIdx.x / TEAM;
  if (t >= p.T) return;
  const int lane = threadIdx.x % TEAM;
  const int64_t slot = __ldg(p.slots + t);
  if (slot < 0) return;
  if (slot >= p.n_slots) {
    if (lane == 0) raise_error(p.err, MTP_ERR_BLOCK_ID);
    return;
  }
  const uint4 *ks = p.k_new + t * p.k_stride, *vs = p.v_new + t * p.v_stride;
  uint4 *kd = p.k_cache + slot * p.k_vecs, *vd = p.v_cache + slot * p.v_vecs;
  constexpr int U = 4;
  const int most = max(p.k_vecs, p.v_vecs);
  for (int c = lane; c < most; c += U * TEAM) {
    uint4 k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u * TEAM < p.k_vecs) k[u] = __ldg(ks + c + u * TEAM);
      if (c + u * TEAM < p.v_vecs) v[u] = __ldg(vs + c + u * TEAM);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u * TEAM < p.k_vecs) kd[c + u * TEAM] = k[u];
      if (c + u * TEAM < p.v_vecs) vd[c + u * TEAM] = v[u];
    }
  }
}

template <int TEAM>
cudaError_t launch(const SlotAppendParams& p, cudaStream_t s) {
  const long long teams = kThreads / TEAM;
  kv_slot_append_kernel<TEAM><<<(unsigned)((p.T + teams - 1) / teams), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

int fail(const char* msg) { return set_error(MTP_INVALID_ARG, msg); }

int check_kv_append(const mtp_kv_append_args* a) {
  if (!a) return fail("mtp_kv_append: args is NULL");
  if (a->T < 0) return fail("mtp_kv_append: T < 0");
  if (a->block_size != MTP_BLOCK_SIZE) return fail("mtp_kv_append: block_size must be 64");
  if (a->num_blocks <= 0) return fail("mtp_kv_append: num_blocks <= 0");
  if (a->dtype != MTP_F32 && a->dtype != MTP_BF16) return fail("mtp_kv_append: dtype");
  const bool mla = a->is_mla != 0;
  if (a->Hkv <= 0 || a->Hkv > (1 << 16) || (mla && a->Hkv != 1)) return fail("mtp_kv_append: Hkv outside [1, 2^16], or not 1 for MLA");
  if (a->d_qk <= 0 || a->d_qk > (1 << 12) || (!mla && (a->d_v <= 0 || a->d_v > (1 << 12))))
    return fail("mtp_kv_append: head dims outside [1, 2^12]");
  const int64_t size = a->dtype == MTP_BF16 ? 2 : 4, kn = (int64_t)a->Hkv * a->d_qk, vn = mla ? 0 : (int64_t)a->Hkv * a->d_v;
  if (kn * size % 16 || vn * size % 16) return set_error(MTP_UNSUPPORTED, "mtp_kv_append: a token's rows must be multiples of 16 bytes");
  if (a->T == 0) return MTP_OK;
  if (!a->k_new || !a->slot_map || !a->k_cache) return fail("mtp_kv_append: a required pointer is NULL");
  if (mla ? (a->v_new || a->v_cache) : (!a->v_new || !a->v_cache))
    return fail(mla ? "mtp_kv_append: MLA takes v_new = v_cache = NULL" : "mtp_kv_append: v_new / v_cache is NULL");
  if (a->k_stride < kn || (!mla && a->v_stride < vn)) return fail("mtp_kv_append: tokens overlap (stride < Hkv d)");
  if (a->k_stride > (1ll << 40) || (!mla && a->v_stride > (1ll << 40))) return fail("mtp_kv_append: stride > 2^40");
  uintptr_t any = (uintptr_t)a->k_new | (uintptr_t)a->k_cache | (uintptr_t)(a->k_stride * size);
  if (!mla) any |= (uintptr_t)a->v_new | (uintptr_t)a->v_cache | (uintptr_t)(a->v_stride * size);
  if (any % 16) return fail("mtp_kv_append: k_new, v_new, the caches and the strides must be 16-byte aligned");
  return MTP_OK;
}

}  // namespace
}  // namespace mtp

extern "C" int mtp_kv_append(const mtp_kv_append_args* a, void* stream) {
  int rc = mtp::check_kv_append(a);
  if (rc != MTP_OK) return rc;
  mtp::set_launch_count(0);
  if (a->T == 0) return MTP_OK;
  unsigned* err = nullptr;
  int sm_count = 0;
  if ((rc = mtp::device_context(&err, &sm_count)) != MTP_OK) return rc;
  const int per = a->dtype == MTP_BF16 ? 8 : 4;   // elements in 16 bytes
  const bool mla = a->is_mla != 0;
  mtp::SlotAppendParams p;
  p.k_new = static_cast<const uint4*>(a->k_new);
  p.v_new = static_cast<const uint4*>(a->v_new);
  p.slots = a->slot_map;
  p.k_cache = static_cast<uint4*>(a->k_cache);
  p.v_cache = static_cast<uint4*>(a->v_cache);
  p.k_stride = a->k_stride / per;
  p.v_stride = mla ? 0 : a->v_stride / per;
  p.n_slots = (int64_t)a->num_blocks * mtp::kBlock;
  p.T = a->T;
  p.k_vecs = a->Hkv * a->d_qk / per;
  p.v_vecs = mla ? 0 : a->Hkv * a->d_v / per;
  p.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int most = std::max(p.k_vecs, p.v_vecs);
  // Lanes a token: 8 for short rows, and for many tokens of middling ones, since warps cost more than loads there (us with 8
  // and with 32 lanes, K alone: 65536 tokens of 128 bytes 5.5, 13.7; of 1152 bytes 26.1, 29.5; 8192 of them 3.7, 3.8, 4096
  // 3.1, 2.7, 1024 2.9, 2.0. 1024 bytes cross between 4096 tokens (2.8, 2.9) and 2048 (2.9, 2.2), 1536 at 8192 (4.2, 4.2;
  // 65536 32.2, 34.3), 512 at 4096 (2.3, 2.5; 2048 2.3, 2.2). Close below 2 KB 32 lanes would be the better ones: 2032 bytes,
  // 8192 tokens 5.3, 4.7, 65536 42.8, 41.5).
  const bool few = most <= 16 || (p.T >= 8192 && most < 128);
  const cudaError_t e = few ? mtp::launch<8>(p, s) : mtp::launch<32>(p, s);
  if (e != cudaSuccess) return mtp::set_cuda_error(e, "kv append launch");
  mtp::set_launch_count(1);
  return MTP_OK;
}
