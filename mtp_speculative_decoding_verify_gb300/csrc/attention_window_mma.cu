// Windowed verify attention of bf16 rows over the bf16 cache.
//
// out = softmax(scale Q K^T) V over the slots each row sees, one pass over
// the cache with a running maximum and sum, fp32 accumulation (mma.sync
// m16n8k16). Pages arrive by TMA in a ring of shared-memory stages that one
// warp fills; a page of one KV head (64 keys) is a tile.
//
// What bounds it is the read of the cache (256 requests of 1k-32k tokens
// behind a window of 4096: 607 us, the copy rate), or, with little of it, the
// beginning and the end (16 requests x 48 rows behind 1000: 24.4 us, of which
// the read is 10). So the work is cut into shares of
// the same number of pages, whatever the lengths (Share). A CTA crosses from
// one request to the next without draining its ring. A request that several
// CTAs share is joined by the last of them to finish, in the order of the
// pages, so the result does not depend on who that is. Every KV head (and tile
// of its rows) has the same number of CTAs, as many as fit the device once: 19
// each for 8 heads, 152 in all, but 128 of the 152 for 32 heads and 80 for 80
// (their time is in attention_window.h). The KV heads of the same pages run
// side by side, which keeps their interleaved rows together in DRAM.
//
// A warp takes 16 query rows (row warp) and every key_parts-th tile; the
// parts join in shared memory at the end of a request. Registers hold Q, the
// scores and the output. Probabilities are rounded to bf16, the type of V that
// the product needs, as in mtp_verify_attention (rms error of an output 2.2e-3,
// of which its own rounding makes 1.66e-3); their sum is of the unrounded ones.
// Above 48 rows mma.sync bounds it (32 requests behind 4096: 64 rows 147 us of
// 81 for the read, 120 rows 295 us). A request of one page is left to its part, so that
// such requests run side by side (113 of them, 16 KV heads: 62 us with a join
// for each, 28 us so).
//
// Slots that not every row sees occur in the last pages, at the window's edge
// and behind the sinks. Only those tiles take the masked path: hidden scores
// become -inf, and values that are not finite are taken out of the product
// (0 x NaN) and put back into the rows that do see them (NaN where the weight is
// 0).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attention_window.h"
#include "kv8.cuh"
#include "mma_sync.cuh"
#include "sm100.cuh"

namespace mtp {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxWarps = 8;              // producer + consumers, two per SM sub-partition: up to 255 registers a thread
constexpr int kMaxStages = 16;
constexpr int kMaxSmem = 232448;          // 227 KB

template <int D>
struct Tile {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kBoxes = kRowBytes > 128 ? kRowBytes / 128 : 1;
  static constexpr int kBytes = kBlock * kRowBytes;      // K or V of a page's head
  static constexpr int kStage = 2 * kBytes;
  // byte offset of the 16-byte chunk c of a key's row
  __device__ __forceinline__ static uint32_t at(int key, int c) {
    return (c >> 3) * (kBlock * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4);   // boxes of 64 dims, 128-byte swizzle
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Take what is not finite out of a pair; true if there was any.
__device__ __forceinline__ bool take_out(uint32_t& w) {
  const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w), z = __hsub2(h, h);
  const uint32_t keep = __heq2_mask(z, z);
  w &= keep;
  return keep != 0xffffffffu;
}

template <int D>
__global__ void __launch_bounds__(kMaxWarps* kWarp, 1)
    window_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const WindowParams p) {
  using T = Tile<D>;
  constexpr int kVals = D / 2 + 4;        // fp32 values of a lane's partial result: output, two maxima, two sums
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* xchg = reinterpret_cast<float*>(smem + p.stages * T::kStage);     // [row warp][key_parts / 2][kVals][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(xchg + p.row_warps * (p.key_parts / 2) * kVals * kWarp);
  uint64_t* empty = full + kMaxStages;
  int* stage_valid = reinterpret_cast<int*>(empty + kMaxStages);           // 0: the table named no block
  int* last_flag = stage_valid + kMaxStages;                               // [row warp]
  volatile int* abort = last_flag + kMaxWarps;

  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int heads = p.Hkv * p.row_tiles;
  const int kvh = blockIdx.x % heads / p.row_tiles, row_tile = blockIdx.x % heads % p.row_tiles;
  const int g_cta = blockIdx.x / heads;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      sm100::mbar_init(&full[s], 1);
      sm100::mbar_init(&empty[s], p.row_warps);   // a tile is read by one part: a warp of every row warp
    }
    *abort = 0;
    sm100::fence_barrier_init();
    sm100::tma_prefetch_desc(&tm_k);
    sm100::tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  // Everything up to here may run while the append still does; what follows
  // reads what it writes.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Share share = load_share(p.shares, g_cta);
  const int t_end = share_end(p.shares, g_cta);
  if (g_cta >= share_count(p.shares)) return;
  // The request that is walked, pages p0 .. p1 - 1 of the line; the next one's
  // end and context are read while it is.
  int b = share.b, ctx = share.ctx, pos = share.begin, p0 = share.p0, p1 = p0 + share.n;
  int next_p1 = 0, next_ctx = 0;
  auto read_next = [&]() {
    if (b + 1 < p.B) {
      next_ctx = __ldg(p.ctx_lens + b + 1);
      next_p1 = __ldcg(p.prefix + b + 2);
    }
  };
  read_next();
  auto find = [&]() {
    while (p1 <= pos) {
      ++b;
      p0 = p1;
      p1 = next_p1;
      ctx = next_ctx;
      read_next();
    }
  };

  int stage = 0;             // of tile n (counted over the CTA's life): n % stages
  uint32_t phase = 0;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The warp reads the block ids of 32 pages at a time, one a lane, so that
    // their latency is paid once for 32 tiles.
    const uint64_t pol = sm100::l2_policy_evict_first();
    int n_fills = 0;
    bool ok = true;
    while (pos < t_end && ok) {
      find();
      const int i1 = min(t_end, p1) - p0;
      const PageSpan span = page_span(ctx, p.R, p.window, p.sinks);
      for (int i = pos - p0; i < i1 && ok; i += kWarp) {
        int blk = -1;
        if (i + lane < i1) {
          blk = p.block_table[(int64_t)b * p.max_blocks + span.page(i + lane)];
          if (blk < 0 || blk >= p.num_blocks) {
            raise_error(p.err, MTP_ERR_BLOCK_ID);
            blk = -1;
          }
        }
        const int n = min(kWarp, i1 - i);
        for (int x = 0; x < n; ++x) {
          const int id = __shfl_sync(0xffffffffu, blk, x);
          int go = 1;
          if (lane == 0) {
            go = sm100::mbar_wait(&empty[stage], phase ^ 1u, abort);
            if (go) {
              stage_valid[stage] = id >= 0;
              if (id >= 0) {
                uint8_t* ks = smem + stage * T::kStage;
                sm100::mbar_arrive_expect_tx(&full[stage], T::kStage);
#pragma unroll
                for (int c = 0; c < T::kBoxes; ++c) {
                  sm100::tma_load_4d(ks + c * kBlock * 128, &tm_k, &full[stage], c * 64, kvh, 0, id, pol);
                  sm100::tma_load_4d(ks + T::kBytes + c * kBlock * 128, &tm_v, &full[stage], c * 64, kvh, 0,
                                     id, pol);
                }
              } else {
                sm100::mbar_arrive(&full[stage]);
              }
            } else {
              *abort = 1;
              raise_error(p.err, MTP_ERR_TIMEOUT);
            }
          }
          ok = __shfl_sync(0xffffffffu, go, 0) != 0;
          if (!ok) break;
          ++n_fills;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      pos = p0 + i1;
    }
    // Every copy issued lands before the CTA may exit.
    if (lane == 0) {
      for (int x = max(0, n_fills - p.stages); x < n_fills; ++x)
        sm100::mbar_wait_timeout(&full[x % p.stages], (uint32_t)((x / p.stages) & 1), sm100::kWaitTimeoutNs);
    }
    return;
  }

  // ------------------------------------------------------------- consumers
  const int cw = warp - 1, rw = cw % p.row_warps, kp = cw / p.row_warps;
  const int g = lane >> 2, t = lane & 3, mi = lane >> 3;
  const int r_lo = (row_tile * p.row_warps + rw) * 16 + g, r_hi = r_lo + 8;
  const int c_lo = min(r_lo, p.rows - 1), c_hi = min(r_hi, p.rows - 1);     // padding rows repeat the last row
  const int j_lo = c_lo / p.group, j_hi = c_hi / p.group;
  const int q_lo = j_lo * p.Hq + kvh * p.group + c_lo % p.group;   // + b R Hq: the row of q and out
  const int q_hi = j_hi * p.Hq + kvh * p.group + c_hi % p.group;
  const int row_block = row_tile * p.row_warps + rw, row_blocks = p.row_tiles * p.row_warps;
  const int part_threads = p.key_parts * kWarp;
  float* my_xchg = xchg + (size_t)rw * (p.key_parts / 2) * kVals * kWarp + lane;
  auto xchg_of = [&](int part) { return my_xchg + part * (kVals * kWarp); };

  uint32_t qa[D / 16][4];
  float o[D / 8][4];
  float m_lo, m_hi, l_lo, l_hi;           // running maxima (log2 units, scaled) and this lane's part of the sums
  const float f = p.sm_scale * kLog2e;
  int tile = 0;                           // n % key_parts == kp: this part's tiles

  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    m_lo = m_hi = -INFINITY;
    l_lo = l_hi = 0.0f;
  };
  // Join another partial result (same fragment layout), read through `val`.
  auto fold = [&](auto&& val) {
    const float ml = val(D / 2), mh = val(D / 2 + 1);
    const float nl = fmaxf(m_lo, ml), nh = fmaxf(m_hi, mh);
    const float al = m_lo == -INFINITY ? 0.0f : ex2(m_lo - nl), bl = ml == -INFINITY ? 0.0f : ex2(ml - nl);
    const float ah = m_hi == -INFINITY ? 0.0f : ex2(m_hi - nh), bh = mh == -INFINITY ? 0.0f : ex2(mh - nh);
    l_lo = l_lo * al + val(D / 2 + 2) * bl;
    l_hi = l_hi * ah + val(D / 2 + 3) * bh;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      o[i][0] = o[i][0] * al + val(4 * i) * bl;
      o[i][1] = o[i][1] * al + val(4 * i + 1) * bl;
      o[i][2] = o[i][2] * ah + val(4 * i + 2) * bh;
      o[i][3] = o[i][3] * ah + val(4 * i + 3) * bh;
    }
    m_lo = nl;
    m_hi = nh;
  };
  auto spill = [&](float* to) {
#pragma unroll
    for (int i = 0; i < D / 2; ++i) to[i * kWarp] = o[i >> 2][i & 3];
    to[(D / 2) * kWarp] = m_lo;
    to[(D / 2 + 1) * kWarp] = m_hi;
    to[(D / 2 + 2) * kWarp] = l_lo;
    to[(D / 2 + 3) * kWarp] = l_hi;
  };
  auto part_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + rw), "r"(part_threads) : "memory"); };
  // Join the parts of this row warp into part 0, halving their number each time.
  auto join_parts = [&]() {
    for (int n = p.key_parts; n > 1;) {
      const int half = (n + 1) / 2;
      if (kp >= half && kp < n) spill(xchg_of(kp - half));
      part_sync();
      if (kp < n - half) {
        const float* from = xchg_of(kp);
        fold([&](int i) { return from[i * kWarp]; });
      }
      part_sync();
      n = half;
    }
  };

  auto consume = [&](int page, int ctx, auto masked_c) {
    constexpr bool kMasked = decltype(masked_c)::value;
    const uint32_t kbase = sm100::smem_u32(smem + stage * T::kStage), vbase = kbase + T::kBytes;
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t b0, b1, b2, b3;
        mma::ldsm_x4(kbase + T::at(np * 16 + (mi >> 1) * 8 + (lane & 7), kk * 2 + (mi & 1)), b0, b1, b2, b3);
        mma::mma_bf16_16816(s[2 * np], qa[kk], b0, b1);
        mma::mma_bf16_16816(s[2 * np + 1], qa[kk], b2, b3);
      }
    }
    if constexpr (kMasked) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int slot = page * kBlock + n * 8 + 2 * t + (e & 1);
          if (!slot_visible(slot, ctx + (e < 2 ? j_lo : j_hi), p.window, p.sinks)) s[n][e] = -INFINITY;
        }
      }
    }
    float x_lo = -INFINITY, x_hi = -INFINITY;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      x_lo = fmaxf(x_lo, fmaxf(s[n][0], s[n][1]));
      x_hi = fmaxf(x_hi, fmaxf(s[n][2], s[n][3]));
    }
    x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 1));
    x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 2));
    x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 1));
    x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 2));
    float n_lo = fmaxf(m_lo, x_lo * f), n_hi = fmaxf(m_hi, x_hi * f);
    if (!kMasked || page_seen(page, ctx + j_lo, p.window, p.sinks)) n_lo = fmaxf(n_lo, kNoWeight);
    if (!kMasked || page_seen(page, ctx + j_hi, p.window, p.sinks)) n_hi = fmaxf(n_hi, kNoWeight);
    const float z_lo = n_lo == -INFINITY ? 0.0f : n_lo, z_hi = n_hi == -INFINITY ? 0.0f : n_hi;
    const float k_lo = ex2(m_lo - z_lo), k_hi = ex2(m_hi - z_hi);
    m_lo = n_lo;
    m_hi = n_hi;
    float t_lo = 0.0f, t_hi = 0.0f;
    uint32_t pa[4][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float p0 = ex2(fmaf(s[n][0], f, -z_lo)), p1 = ex2(fmaf(s[n][1], f, -z_lo));
      const float p2 = ex2(fmaf(s[n][2], f, -z_hi)), p3 = ex2(fmaf(s[n][3], f, -z_hi));
      t_lo += p0 + p1;
      t_hi += p2 + p3;
      pa[n >> 1][(n & 1) * 2] = mma::pack_bf16(p0, p1);
      pa[n >> 1][(n & 1) * 2 + 1] = mma::pack_bf16(p2, p3);
    }
    l_lo = l_lo * k_lo + t_lo;
    l_hi = l_hi * k_hi + t_hi;
    bool out_of = false;
    uint32_t some = 0;        // probabilities that are not 0: of the i-th word of pa, bits 31 - i (upper half) and 15 - i
    if constexpr (kMasked) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) some |= ((pa[n >> 1][(n & 1) * 2 + e] + 0x7fff7fffu) & 0x80008000u) >> (2 * n + e);
      }
    }
    if (__any_sync(0xffffffffu, k_lo != 1.0f || k_hi != 1.0f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= k_lo;
        o[i][1] *= k_lo;
        o[i][2] *= k_hi;
        o[i][3] *= k_hi;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int dp = 0; dp < D / 16; ++dp) {
        uint32_t b0, b1, b2, b3;
        mma::ldsm_x4_trans(vbase + T::at(k * 16 + (mi & 1) * 8 + (lane & 7), dp * 2 + (mi >> 1)), b0, b1, b2, b3);
        if constexpr (kMasked) {
          out_of |= take_out(b0);
          out_of |= take_out(b1);
          out_of |= take_out(b2);
          out_of |= take_out(b3);
        }
        mma::mma_bf16_16816(o[2 * dp], pa[k], b0, b1);
        mma::mma_bf16_16816(o[2 * dp + 1], pa[k], b2, b3);
      }
    }
    if constexpr (kMasked) {
      if (__any_sync(0xffffffffu, out_of)) {       // rare: a NaN or infinity in V
        const uint8_t* vt = smem + stage * T::kStage + T::kBytes;
#pragma unroll 1
        for (int key = 0; key < kBlock; ++key) {
          // of the lane that holds the key's probabilities
          const uint32_t has = __shfl_sync(0xffffffffu, some, (lane & ~3) | (key % 8 / 2)) << (key / 8 * 2 + (key & 1 ? 0 : 16));
          const float none_lo = has >> 31 ? 0.0f : NAN, none_hi = (has >> 30) & 1 ? 0.0f : NAN;
          const bool see_lo = slot_visible(page * kBlock + key, ctx + j_lo, p.window, p.sinks);
          const bool see_hi = slot_visible(page * kBlock + key, ctx + j_hi, p.window, p.sinks);
          if (!see_lo && !see_hi) continue;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // the dim of o[i][e] and o[i][e + 2]
              const int dim = i * 8 + 2 * t + e;
              const float v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vt + T::at(key, dim / 8) + dim % 8 * 2));
              if (!(fabsf(v) <= FLT_MAX)) {
                if (see_lo) o[i][e] += v + none_lo;
                if (see_hi) o[i][e + 2] += v + none_hi;
              }
            }
          }
        }
      }
    }
  };

  while (pos < t_end) {
    find();
    const int i0 = pos - p0, i1 = min(t_end, p1) - p0, n_tiles = p1 - p0;
    const PageSpan span = page_span(ctx, p.R, p.window, p.sinks);
    const bool alone = n_tiles == 1;      // its part does the request by itself, and the others go on
    if (alone && tile != kp) {
      if (++tile == p.key_parts) tile = 0;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
      pos = p1;
      continue;
    }
    const int64_t row0 = (int64_t)b * p.R * p.Hq;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q);
    const uint32_t* lo = reinterpret_cast<const uint32_t*>(qp + (row0 + q_lo) * D);
    const uint32_t* hi = reinterpret_cast<const uint32_t*>(qp + (row0 + q_hi) * D);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][0] = __ldg(lo + kk * 8 + t);
      qa[kk][1] = __ldg(hi + kk * 8 + t);
      qa[kk][2] = __ldg(lo + kk * 8 + 4 + t);
      qa[kk][3] = __ldg(hi + kk * 8 + 4 + t);
    }
    clear();

    for (int i = i0; i < i1; ++i) {
      if (tile == kp) {
        if (!__all_sync(0xffffffffu, sm100::mbar_wait(&full[stage], phase, abort) ? 1 : 0)) {
          // the tiles that are left give up at once; the joins below still meet
          if (lane == 0) {
            *abort = 1;
            raise_error(p.err, MTP_ERR_TIMEOUT);
          }
        } else {
          if (stage_valid[stage]) {
            const int page = span.page(i), first = page * kBlock, last = first + kBlock - 1;
            const bool whole = last <= ctx && (p.window == 0 || first > ctx + p.R - 1 - p.window || last < p.sinks);
            if (whole) consume(page, ctx, std::false_type());
            else consume(page, ctx, std::true_type());
          }
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&empty[stage]);
        }
      }
      if (++tile == p.key_parts) tile = 0;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    pos = p0 + i1;

    if (!alone) join_parts();
    if (i0 > 0 || i1 < n_tiles) {
      // Shared with other CTAs: leave the partial result, and the last to
      // arrive at this (request, KV head, row block) joins them all. Slot 0
      // of a CTA is for a request it did not begin, slot 1 for one it began.
      const int2 in = __ldcg(p.sharers + b);
      const int g0 = in.x, g1 = in.y;
      const size_t stride = (size_t)kVals * kWarp;
      auto slot_of = [&](int gg, int which) {
        return p.part_o + ((((size_t)gg * 2 + which) * p.Hkv + kvh) * row_blocks + row_block) * stride + lane;
      };
      if (kp == 0) {
        spill(slot_of(g_cta, i0 > 0 ? 0 : 1));
        __syncwarp();
        if (lane == 0) last_flag[rw] = arrive_at(p.arrived + ((int64_t)b * p.Hkv + kvh) * row_blocks + row_block) == g1 - g0;
      }
      part_sync();
      const bool last = *const_cast<volatile int*>(last_flag + rw) != 0;
      if (!last) {
        part_sync();       // the flag has been read
        continue;
      }
      clear();
      for (int gg = g0 + kp; gg <= g1; gg += p.key_parts) {
        const float* from = slot_of(gg, gg == g0 ? 1 : 0);
        fold([&](int i) { return __ldcg(from + i * kWarp); });
      }
      part_sync();
      join_parts();
    }
    if (alone || kp == 0) {
      l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
      l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
      l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
      // no weight: nothing seen (bad blocks only), or -inf only
      const float v_lo = l_lo != 0.0f ? 1.0f / l_lo : m_lo == -INFINITY ? 0.0f : NAN;
      const float v_hi = l_hi != 0.0f ? 1.0f / l_hi : m_hi == -INFINITY ? 0.0f : NAN;
      __nv_bfloat16* out_lo = static_cast<__nv_bfloat16*>(p.out) + (row0 + q_lo) * D;
      __nv_bfloat16* out_hi = static_cast<__nv_bfloat16*>(p.out) + (row0 + q_hi) * D;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        if (r_lo < p.rows)
          *reinterpret_cast<uint32_t*>(out_lo + i * 8 + 2 * t) = mma::pack_bf16(o[i][0] * v_lo, o[i][1] * v_lo);
        if (r_hi < p.rows)
          *reinterpret_cast<uint32_t*>(out_hi + i * 8 + 2 * t) = mma::pack_bf16(o[i][2] * v_hi, o[i][3] * v_hi);
      }
    }
  }
}

// The layout of a launch: row warps and key parts of a CTA, stages, CTAs.
// A page of 64 keys keeps a warp busy for about as long as several pages take
// to arrive, so a CTA (one per SM: 227 KB of stages) needs around 8 warps;
// with few rows they come from key parts.
template <int D>
void layout(const mtp_window_attn_args& a, int sm_count, WindowPlan* pl) {
  using T = Tile<D>;
  const int blocks = (a.Hq / a.Hkv * (a.D + 1) + 15) / 16;     // of 16 rows
  pl->row_tiles = (blocks + kMaxWarps - 2) / (kMaxWarps - 1);
  pl->row_warps = (blocks + pl->row_tiles - 1) / pl->row_tiles;
  // Tile n sits in stage n % stages and goes to part n % key_parts. stages is
  // a multiple of key_parts, so that each stage serves one part, which meets
  // its phases one after the other, and two stages a part at least, so that
  // one fills while the other is read.
  for (pl->key_parts = (kMaxWarps - 1) / pl->row_warps;; --pl->key_parts) {
    const int fixed = pl->row_warps * (pl->key_parts / 2) * (D / 2 + 4) * kWarp * 4 + kMaxStages * 20 + (kMaxWarps + 1) * 4 + 1024;
    pl->stages = std::min(kMaxStages, (kMaxSmem - fixed) / T::kStage) / pl->key_parts * pl->key_parts;
    pl->smem = pl->stages * T::kStage + fixed;
    if (pl->key_parts == 1 || pl->stages >= 2 * pl->key_parts) break;
  }
  pl->ctas_per_head = head_ctas(a, sm_count, (long long)a.Hkv * pl->row_tiles);
}

template <int D>
cudaError_t launch(const mtp_window_attn_args& a, const WindowPlan& pl, const WindowParams& p, cudaStream_t s) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t elem = 2;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.Hkv, (cuuint64_t)kBlock, (cuuint64_t)a.num_blocks};
  const cuuint64_t strides[3] = {D * elem, a.Hkv * D * elem, (cuuint64_t)kBlock * a.Hkv * D * elem};
  const cuuint32_t box[4] = {64u, 1, (cuuint32_t)kBlock, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i) {
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               i == 0 ? a.k_cache : a.v_cache, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(window_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, pl.smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(pl.ctas_per_head * a.Hkv * pl.row_tiles);
  return launch_behind_append(window_mma_kernel<D>, grid, (pl.row_warps * pl.key_parts + 1) * kWarp, pl.smem, s, maps[0],
                              maps[1], p);
}

}  // namespace

WindowPlan plan_window_mma(const mtp_window_attn_args& a, int sm_count) {
  WindowPlan pl{};
  a.d == 128 ? layout<128>(a, sm_count, &pl) : layout<64>(a, sm_count, &pl);
  const size_t rows = (size_t)a.Hkv * pl.row_tiles * pl.row_warps;     // row blocks of a request
  pl.ws_partial_o = plan_schedule(&pl, a.B, a.Hkv);
  pl.ws_bytes = pl.ws_partial_o + (size_t)pl.ctas_per_head * 2 * rows * (a.d / 2 + 4) * kWarp * sizeof(float);
  pl.ws_bytes = (pl.ws_bytes + 255) / 256 * 256;
  return pl;
}

cudaError_t launch_window_mma(const mtp_window_attn_args& a, const WindowPlan& pl, const WindowParams& p, cudaStream_t s) {
  return a.d == 128 ? launch<128>(a, pl, p, s) : launch<64>(a, pl, p, s);
}

}  // namespace mtp
