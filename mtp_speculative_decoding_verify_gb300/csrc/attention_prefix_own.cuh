// The requests' own pages of mtp_verify_attention_prefix for bf16 rows: the
// part of prefix_kernel's CTAs that do them.
//
// A request has few rows of a KV head (R x group) and, behind a shared prefix,
// few pages, so the read of the pages bounds this part, as long as no warp waits
// for another at the many beginnings and ends. So warps work in teams that have
// nothing to do with each other: the row_warps warps of a team take 16 rows each
// of one (request, KV head), page after page, out of a ring of shared-memory
// stages of the team's own (32 or 64 keys of K and V each, by TMA; which, lay_out
// decides), and leave a partial result. The teams have an even share of the line
// of all pages (as the prefix's CTAs of theirs, attention_prefix.h), cut wherever
// it falls; what a cut parts is joined with the prefix's results, which have to be
// joined in any case. Products are mma.sync m16n8k16: 16 rows need no more.
//
// Alone on the device: 16 rows of 128 dims 6.0 TB/s; 48 rows 4.5 TB/s, 64 dims 3.8,
// bound by the chain from one stage's scores to its products (the tensor pipe is
// busy 40 % of the time; the next scores ahead of a stage's softmax cost more
// registers than they gave: 15 % slower). On 54 SMs, 16 rows get 90 GB/s an SM, of
// the 121 that loads alone get.
//
// Four warps load, a lane for each team: it looks whether the team's next slot is
// free, loads it, and has the block id after that on its way.
//
// Hidden slots (behind a row's own token, or off its path in a tree) occur in the
// last stages only; those take the masked path of attention_window_mma.cu:
// hidden scores become -inf, and values that are not finite are taken out of the
// product (0 x NaN) and put back into the rows that see them.
#pragma once

#include <float.h>

#include <type_traits>

#include "attention_prefix.h"
#include "attention_window.h"
#include "mma_sync.cuh"
#include "sm100.cuh"

namespace mtp {
namespace own {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBox = 32;                  // keys of a box
constexpr int kWarps = 8, kLoaders = 4;   // consumers, warps that load
constexpr int kMaxStages = 8;             // of a team

template <int D, int KEYS>
struct Stage {
  static constexpr int kHalf = KEYS * D * 2, kBytes = 2 * kHalf;    // K or V; both
  // byte offset of the 16-byte chunk c of a key's row: boxes of 64 dims, 128-byte swizzle
  __device__ __forceinline__ static uint32_t at(int key, int c) {
    return (c >> 3) * (KEYS * 128) + key * 128 + (((c & 7) ^ (key & 7)) << 4);
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

// A team's place in the line: pages pos .. end - 1, of which the next belong to
// item (request b, head and row tile hr) with `pages` pages from unit u0 on.
// What it needs of the request after b is on its way before it is asked for.
struct OwnWalk {
  const PrefixParams& p;
  int pos, end, b, hr, pages, u0, heads, ctx, first;
  int sum1, sum2, ctx1, first1;           // own pages of the requests up to b and b + 1; of request b + 1
  struct Seg {
    int b, hr, i0, i1;                    // pages i0 .. i1 - 1 of the request's own
    int ctx, first;                       // its context, the first page of its own
  };
  __device__ __forceinline__ void look_ahead() {
    const int n = min(b + 1, p.B - 1);
    sum2 = __ldcg(p.view.pages + n + 1);
    ctx1 = __ldg(p.ctx_lens + n);
    first1 = __ldcg(p.view.first + n);
  }
  __device__ __forceinline__ OwnWalk(const PrefixParams& params, int team) : p(params) {   // (team: of all CTAs')
    heads = p.Hkv * p.row_tiles;
    pos = end = b = hr = pages = u0 = ctx = first = sum1 = 0;
    if (team >= __ldcg(&p.view.own->ctas)) return;
    const OwnStart* at = p.view.own_starts + team;
    const int4 v = __ldcg(reinterpret_cast<const int4*>(at));
    pages = __ldcg(&at->pages);
    pos = v.x;
    end = v.y;
    b = v.z;
    look_ahead();
    ctx = __ldg(p.ctx_lens + b);
    first = __ldcg(p.view.first + b);
    sum1 = v.w + pages;
    hr = (pos - v.w * heads) / pages;
    u0 = v.w * heads + hr * pages;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (pos >= end) return false;
    while (pos >= u0 + pages) {
      u0 += pages;
      if (++hr == heads) {
        hr = 0;
        ++b;
        pages = sum2 - sum1;
        sum1 = sum2;
        ctx = ctx1;
        first = first1;
        look_ahead();
      }
    }
    s.b = b;
    s.hr = hr;
    s.i0 = pos - u0;
    s.i1 = min(pages, s.i0 + end - pos);
    s.ctx = ctx;
    s.first = first;
    pos += s.i1 - s.i0;
    return true;
  }
};

// Boxes of a page: 1 when the last verify token is in its first half.
__device__ __forceinline__ int boxes_of(int page, int ctx, int R) { return ctx + R - page * kBlock > kBox ? 2 : 1; }
// .. and stages.
template <int KEYS>
__device__ __forceinline__ int stages_of(int page, int ctx, int R) {
  return KEYS == kBlock ? 1 : boxes_of(page, ctx, R);
}

// Barriers and flags of the teams' stages, behind the stages. K and V of a stage
// are slots of their own (2 x and 2 x + 1), so that a K is replaced as soon as the
// scores are there: of two stages' four slots, three are on their way at any time.
struct Control {
  uint64_t *full, *empty;                 // [team][stage][2]
  volatile int* valid;                    // [team][stage] 0: the table named no block
  volatile int* abort;
};

// The warps that load: a lane of warp w for each of the teams w, w + 4, .. (one warp
// for all is the slowest part of the CTA); cta: among those that do own pages. A
// lane must not wait for global memory, since the others wait with it: the next
// segment and the next block id are read ahead.
template <int D, int KEYS>
__device__ __forceinline__ void producer(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PrefixParams& p, uint8_t* smem,
                                         const Control& c, int cta) {
  using T = Stage<D, KEYS>;
  const int team = threadIdx.x % kWarp * kLoaders + threadIdx.x / kWarp;
  volatile int* abort = c.abort;
  if (team < p.teams) {
    const uint64_t pol = sm100::l2_policy_evict_first();
    OwnWalk walk(p, cta * p.teams + team);
    OwnWalk::Seg seg, after;
    const int slots = 2 * p.stages;
    uint8_t* ring = smem + (size_t)team * p.stages * T::kBytes;
    uint64_t *my_full = c.full + team * slots, *my_empty = c.empty + team * slots;
    volatile int* my_valid = c.valid + team * p.stages;
    int n = 0, slot = 0, i = 0, half = 0, halves = 0, id = 0, next_id = 0, kvh = 0;
    uint32_t phase = 1;                   // of `empty`: the first round needs no wait
    bool more = walk.next(seg), more_after = false;
    auto read_id = [&](const OwnWalk::Seg& s, int x) { return __ldg(p.block_table + (int64_t)s.b * p.max_blocks + s.first + x); };
    auto begin = [&]() {                  // of a segment, whose first id has been asked for
      kvh = seg.hr / p.row_tiles;
      i = seg.i0;
      more_after = walk.next(after);
    };
    auto begin_page = [&]() {
      id = next_id;
      half = 0;
      halves = stages_of<KEYS>(seg.first + i, seg.ctx, p.R);
      if (i + 1 < seg.i1) next_id = read_id(seg, i + 1);
      else if (more_after) next_id = read_id(after, after.i0);
    };
    if (more) {
      next_id = read_id(seg, seg.i0);
      begin();
      begin_page();
    }
    uint64_t t0 = sm100::globaltimer();
    for (uint32_t spin = 1; more; ++spin) {
      if (sm100::mbar_test_wait(&my_empty[slot], phase)) {
        const bool good = id >= 0 && id < p.num_blocks, is_v = slot & 1;
        if (!is_v) my_valid[slot / 2] = good;
        if (good) {
          uint8_t* to = ring + slot * T::kHalf;
          // (of a page that is one stage, the half that is needed: what lies in the other is masked)
          const int boxes = KEYS == kBox ? 1 : boxes_of(seg.first + i, seg.ctx, p.R);
          sm100::mbar_arrive_expect_tx(&my_full[slot], boxes * kBox * D * 2);
          const CUtensorMap* map = is_v ? &tm_v : &tm_k;
          for (int y = 0; y < boxes; ++y) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              sm100::tma_load_4d(to + (x * KEYS + y * kBox) * 128, map, &my_full[slot], x * 64, kvh, (half + y) * kBox, id, pol);
          }
        } else {
          raise_error(p.err, MTP_ERR_BLOCK_ID);
          sm100::mbar_arrive(&my_full[slot]);
        }
        ++n;
        if (++slot == slots) {
          slot = 0;
          phase ^= 1u;
        }
        if (is_v && ++half == halves) {
          if (++i == seg.i1) {
            more = more_after;
            seg = after;
            if (more) begin();
          }
          if (more) begin_page();
        }
        spin = 0;
      } else if ((spin & 255u) == 0) {
        if (spin == 256) t0 = sm100::globaltimer();
        if (*abort) break;
        if (sm100::globaltimer() - t0 > sm100::kWaitTimeoutNs) {
          *abort = 1;
          raise_error(p.err, MTP_ERR_TIMEOUT);
          break;
        }
      }
    }
    // Every copy issued lands before the CTA may exit.
    for (int x = max(0, n - slots); x < n; ++x)
      sm100::mbar_wait_timeout(&my_full[x % slots], (uint32_t)((x / slots) & 1), sm100::kWaitTimeoutNs);
  }
  __syncwarp();
}

// Consumer warp cw of the CTA's.
template <int D, int KEYS>
__device__ __forceinline__ void consumer(const PrefixParams& p, uint8_t* smem, const Control& c, int cta, int cw) {
  using T = Stage<D, KEYS>;
  if (cw >= p.teams * p.row_warps) return;
  const int lane = threadIdx.x % kWarp;
  volatile int* abort = c.abort;
  const int team = cw / p.row_warps, rw = cw % p.row_warps;
  const int g = lane >> 2, t = lane & 3, mi = lane >> 3;
  uint8_t* ring = smem + (size_t)team * p.stages * T::kBytes;
  uint64_t *my_full = c.full + team * 2 * p.stages, *my_empty = c.empty + team * 2 * p.stages;
  volatile int* my_valid = c.valid + team * p.stages;
  const float f = p.sm_scale * kLog2e;
  const int tile_rows = p.row_warps * 16;
  OwnWalk walk(p, cta * p.teams + team);
  OwnWalk::Seg seg;
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;

  // Q of the item after this one, on its way into L1: a line of it a lane.
  auto ask_for_q = [&]() {
    if (walk.pos >= walk.end) return;
    const bool same = walk.hr + 1 < walk.heads;
    const int b = same ? walk.b : min(walk.b + 1, p.B - 1), hr = same ? walk.hr + 1 : 0, row = rw * 16 + lane / (D / 64);
    const int r = min(hr % p.row_tiles * tile_rows + row, p.rows - 1);
    const char* at = static_cast<const char*>(p.q) +
                     (((int64_t)b * p.R + r / p.group) * p.Hq + hr / p.row_tiles * p.group + r % p.group) * (D * 2) + lane % (D / 64) * 128;
    if (lane < 16 * (D / 64)) asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
  };

  while (ok && walk.next(seg)) {
    const int b = seg.b, kvh = seg.hr / p.row_tiles, ctx = seg.ctx, first = seg.first;
    const int r_lo = seg.hr % p.row_tiles * tile_rows + rw * 16 + g, r_hi = r_lo + 8;
    const int c_lo = min(r_lo, p.rows - 1), c_hi = min(r_hi, p.rows - 1);     // padding rows repeat the last row
    const int j_lo = c_lo / p.group, j_hi = c_hi / p.group;
    uint32_t qa[D / 16][4];
    {
      const int64_t row0 = (int64_t)b * p.R * p.Hq + kvh * p.group;
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q);
      const uint32_t* lo = reinterpret_cast<const uint32_t*>(qp + (row0 + j_lo * p.Hq + c_lo % p.group) * D);
      const uint32_t* hi = reinterpret_cast<const uint32_t*>(qp + (row0 + j_hi * p.Hq + c_hi % p.group) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qa[kk][0] = __ldg(lo + kk * 8 + t);
        qa[kk][1] = __ldg(hi + kk * 8 + t);
        qa[kk][2] = __ldg(lo + kk * 8 + 4 + t);
        qa[kk][3] = __ldg(hi + kk * 8 + 4 + t);
      }
    }
    ask_for_q();
    const uint32_t path_lo = tree_path_mask(p.view.parents, b, p.R, j_lo, p.err);
    const uint32_t path_hi = tree_path_mask(p.view.parents, b, p.R, j_hi, p.err);
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.0f, l_hi = 0.0f;   // maxima (log2 units), this lane's part of the sums

    auto wait = [&](int slot) {                      // (most often there is nothing to wait for: a test takes less than a wait)
      return __all_sync(0xffffffffu, sm100::mbar_test_wait(&my_full[slot], phase)) ||
             __all_sync(0xffffffffu, sm100::mbar_wait(&my_full[slot], phase, abort) ? 1 : 0);
    };
    auto release = [&](int slot) {
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&my_empty[slot]);
    };
    // keys_c keys at slots slot0 and up, the stage's from key0 on; `begins` and `ends`: the stage's first, its last
    auto consume = [&](int slot0, int key0, bool begins, bool ends, auto keys_c, auto masked_c) {
      constexpr bool kMasked = decltype(masked_c)::value;
      constexpr int kKeys = decltype(keys_c)::value;
      const uint32_t kbase = sm100::smem_u32(ring + stage * T::kBytes) + key0 * 128, vbase = kbase + T::kHalf;
      float s[kKeys / 8][4];
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int np = 0; np < kKeys / 16; ++np) {
          uint32_t b0, b1, b2, b3;
          mma::ldsm_x4(kbase + T::at(np * 16 + (mi >> 1) * 8 + (lane & 7), kk * 2 + (mi & 1)), b0, b1, b2, b3);
          mma::mma_bf16_16816(s[2 * np], qa[kk], b0, b1);
          mma::mma_bf16_16816(s[2 * np + 1], qa[kk], b2, b3);
        }
      }
      if (ends) release(2 * stage);
      bool some_lo = true, some_hi = true;           // the row sees a slot of the stage
      if constexpr (kMasked) {
        const int rel = slot0 - ctx;                 // (node 0, at slot ctx, is on every path)
        some_lo = rel <= 0 || (rel < 32 && path_lo >> rel != 0);
        some_hi = rel <= 0 || (rel < 32 && path_hi >> rel != 0);
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (tree_hidden(slot0 + n * 8 + 2 * t + (e & 1), ctx, e < 2 ? path_lo : path_hi)) s[n][e] = -INFINITY;
        }
      }
      float x_lo = -INFINITY, x_hi = -INFINITY;
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n) {
        x_lo = fmaxf(x_lo, fmaxf(s[n][0], s[n][1]));
        x_hi = fmaxf(x_hi, fmaxf(s[n][2], s[n][3]));
      }
      x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 1));
      x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 2));
      x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 1));
      x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 2));
      float n_lo = fmaxf(m_lo, x_lo * f), n_hi = fmaxf(m_hi, x_hi * f);
      if (some_lo) n_lo = fmaxf(n_lo, kNoWeight);
      if (some_hi) n_hi = fmaxf(n_hi, kNoWeight);
      const float z_lo = n_lo == -INFINITY ? 0.0f : n_lo, z_hi = n_hi == -INFINITY ? 0.0f : n_hi;
      const float k_lo = ex2(m_lo - z_lo), k_hi = ex2(m_hi - z_hi);
      m_lo = n_lo;
      m_hi = n_hi;
      float t_lo = 0.0f, t_hi = 0.0f;
      uint32_t pa[kKeys / 16][4];
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n) {
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
        for (int n = 0; n < kKeys / 8; ++n) {
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
      if (begins && !(ok = wait(2 * stage + 1))) return;
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k) {
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
          const uint8_t* vt = ring + stage * T::kBytes + T::kHalf;
#pragma unroll 1
          for (int key = 0; key < kKeys; ++key) {
            // of the lane that holds the key's probabilities
            const uint32_t has = __shfl_sync(0xffffffffu, some, (lane & ~3) | (key % 8 / 2)) << (key / 8 * 2 + (key & 1 ? 0 : 16));
            const float none_lo = has >> 31 ? 0.0f : NAN, none_hi = (has >> 30) & 1 ? 0.0f : NAN;
            const bool see_lo = !tree_hidden(slot0 + key, ctx, path_lo), see_hi = !tree_hidden(slot0 + key, ctx, path_hi);
            if (!see_lo && !see_hi) continue;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // the dim of o[i][e] and o[i][e + 2]
                const int dim = i * 8 + 2 * t + e;
                const float v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vt + T::at(key0 + key, dim / 8) + dim % 8 * 2));
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

    for (int i = seg.i0; i < seg.i1 && ok; ++i) {
      const int page = first + i, halves = stages_of<KEYS>(page, ctx, p.R);
      for (int half = 0; half < halves; ++half) {
        if (!(ok = wait(2 * stage))) break;
        if (my_valid[stage]) {
          const int slot0 = page * kBlock + half * KEYS;
          // (where some keys are hidden, 32 at a time: there are few such stages, and twice the keys do not fit the registers)
          using One = std::integral_constant<int, kBox>;
          if (KEYS > kBox && slot0 + KEYS - 1 <= ctx) {
            consume(slot0, 0, true, true, std::integral_constant<int, KEYS>(), std::false_type());
          } else {
            const int boxes = KEYS == kBox ? 1 : boxes_of(page, ctx, p.R);
            for (int y = 0; y < boxes && ok; ++y) {
              const int at = slot0 + y * kBox;
              if (KEYS == kBox && at + kBox - 1 <= ctx) consume(at, y * kBox, y == 0, y + 1 == boxes, One(), std::false_type());
              else consume(at, y * kBox, y == 0, y + 1 == boxes, One(), std::true_type());
            }
          }
          if (!ok) break;
        } else {
          if (!(ok = wait(2 * stage + 1))) break;
          release(2 * stage);
        }
        release(2 * stage + 1);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) break;
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
    const int64_t part = (int64_t)b * walk.heads + seg.hr + cta * p.teams + team;
    const int at = rw * 16 + g;
    if (t == 0) {
      p.view.own_stats[part * tile_rows + at] = make_float2(m_lo, l_lo);
      p.view.own_stats[part * tile_rows + at + 8] = make_float2(m_hi, l_hi);
    }
    float* lo = p.view.own_parts + (part * tile_rows + at) * D + 2 * t;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      *reinterpret_cast<float2*>(lo + i * 8) = make_float2(o[i][0], o[i][1]);
      *reinterpret_cast<float2*>(lo + 8 * D + i * 8) = make_float2(o[i][2], o[i][3]);
    }
  }
  if (!ok) {
    *abort = 1;
    if (lane == 0) raise_error(p.err, MTP_ERR_TIMEOUT);
  }
}

}  // namespace own
}  // namespace mtp
