// mtp_verify_attention_prefix for bf16 rows: the groups' prefixes on the
// 5th-generation tensor cores, and beside them, on other CTAs of the same
// launch, the requests' own pages (attention_prefix_own.cuh). The first is bound by
// products and the second by the read of the cache, and neither needs the whole
// device for that: side by side they take less than one after the other. How many
// CTAs do which is worked out with the shares (prefix_schedule).
//
// The prefix. For every item (attention_prefix.h: up to 256 rows of a group and KV head)
// and the tiles of 128 keys in this CTA's share of it,
//   S = Q K^T,  P = 2^(scale log2e S - m),  O += P V,  l += sum P,
// left as partial results (O, m, l). The rows of all requests of a group are
// one matrix, so products bound it (4 d flops a row and key) once the group
// has a few hundred rows, and the read of the prefix before that.
//
// Both products are tcgen05.mma with M = 128 rows: S from shared memory, N =
// 128 keys; O with P from TMEM and V MN-major from shared memory, N = d dims.
// TMEM holds S and O of two tiles of rows, all 512 columns at d = 128; P (bf16,
// half the columns) takes the place of the S it came from. While one tile's
// softmax runs on its four warps, the tensor cores do P V and the next S of
// the other. The MMAs are issued by one thread in the order P V(i), S(i+1) for
// each tile, and run in that order: S is there only when the P V before it is
// done, so O may then be rescaled, and S may overwrite P without a wait.
//
// A thread of a softmax warp has one row. Its maximum moves only when a tile
// passes it by 2^8 (O is then rescaled in TMEM, a rare branch): P and l stay
// relative to it, and fp32 and bf16 have the room.
//
// A unit (256 rows x 128 keys) takes 1.70 us at 128 dims, which is 1.5 PFLOP/s on
// all SMs; its products without the softmax 1.52, at 64 dims 1.41 and 1.11. 4096
// rows of 8 KV heads behind 8192 tokens are 92 us of all SMs by that; the whole call
// takes 131 (256 requests with one own page each, append and join), and a profile
// of this kernel, with cold caches, 116, tensor pipe 55 % of the time.
//
// Warps: 0 TMA (Q by boxes of whole tokens, K and V pages in a ring of tiles),
// 1 MMA, 4-7 and 8-11 softmax.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "attention_prefix_own.cuh"
#include "attention_window.h"
#include "sm100.cuh"

namespace mtp {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
bool make_bf16_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 384;
constexpr int kRows = kPrefixTcRows, kKeys = 2 * kBlock;
constexpr int kInfo = 8;               // tiles whose pages' marks are held
constexpr float kLazy = 8.0f;          // log2: how far a tile may pass the maximum that P is relative to
constexpr uint32_t kColO = 256;        // S (and P) of the two tiles at columns 0 and 128, O at 256 and 384

template <int D>
struct Smem {
  static constexpr int kChunk = 128 * 128;                      // 128 rows or keys x 64 dims
  static constexpr int kTile = D / 64 * kChunk;                 // Q of 128 rows, K or V of 128 keys
  static constexpr int kQ = 0, kRing = 2 * kTile;
  static constexpr int kSlots = D == 128 ? 5 : 12;              // K and V tiles in turn
  static constexpr int kBar = kRing + kSlots * kTile;           // behind the stages of the own pages, too
  static constexpr int kBars = 2 * kSlots + 2 + 8 + kInfo + 1;
  static constexpr int kMisc = kBar + kBars * 8;                // marks [kInfo], abort, TMEM base
  static constexpr int kOwnStages = kBar / own::Stage<D, own::kBox>::kBytes;   // of 32 keys
  static constexpr int kOwn = kMisc + kInfo * 4 + 8;            // own::Control
  static constexpr int kBytes = kOwn + kOwnStages * 36 + 1024;
  static_assert(kBytes <= 232448, "227 KB of shared memory");
  static_assert(kOwn % 8 == 0, "barriers are 8 bytes");
};

// ------------------------------------------------------------- instructions
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// (a, b) += (c, d) and (a, b) = (a, b) f + g as one instruction each.
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n  .reg .b64 p, q;\n  mov.b64 p, {%0, %1};\n  mov.b64 q, {%2, %3};\n  add.rn.f32x2 p, p, q;\n  mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void fma2(float& a, float& b, float f, float g) {
  asm("{\n  .reg .b64 p, q, r;\n  mov.b64 p, {%0, %1};\n  mov.b64 q, {%2, %2};\n  mov.b64 r, {%3, %3};\n"
      "  fma.rn.f32x2 p, p, q, r;\n  mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(f), "f"(g));
}

// D[tmem] (+)= A[tmem, two bf16 a column] x B[smem]^T.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand with 128-byte swizzling: 64-element MN blocks `lbo` bytes
// apart, 8-row K groups 1024 B apart.
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 consecutive columns from registers.
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---------------------------------------------------------------------- walk
// This CTA's part of an item: tiles u0 .. u1 - 1 of keys.
struct Seg {
  int first, blocks;                   // the group's first request, blocks of its prefix
  int kvh, sub0, nsub;                 // KV head; first tile of rows in the group and how many there are
  int u0, u1;
  int64_t part;                        // the partial result
};

struct Walk {
  const PrefixParams& p;
  PrefixGroup g;
  int pos, end, gi, cta;
  __device__ __forceinline__ Walk(const PrefixParams& params, int prefix_cta) : p(params), cta(prefix_cta) {
    pos = end = gi = 0;
    if (cta >= __ldcg(&p.view.head->ctas)) return;
    const PrefixStart* at = p.view.starts + cta;
    g = load_group(&at->group);
    const int4 v = __ldcg(reinterpret_cast<const int4*>(&at->gi));
    gi = v.x;
    pos = v.y;
    end = v.z;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (pos >= end) return false;
    while (g.units == 0 || pos >= g.line + g.tiles * p.Hkv * g.units) g = load_group(p.view.groups + ++gi);
    const int k = (pos - g.line) / g.units, rt = k % g.tiles;
    s.first = g.first;
    s.blocks = g.blocks;
    s.kvh = k / g.tiles;
    s.sub0 = rt * 2;
    s.nsub = min(2, g.sub_tiles - s.sub0);
    s.u0 = pos - g.line - k * g.units;
    s.u1 = min(g.units, s.u0 + end - pos);
    s.part = (int64_t)g.item + k + cta;
    pos += s.u1 - s.u0;
    return true;
  }
};

template <int D, int OWN_KEYS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PrefixParams p) {
  using S = Smem<D>;
  constexpr int kSlots = S::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBar);   // [kSlots] the tile has landed
  uint64_t* empty = full + kSlots;                                // [kSlots] .. and has been read
  uint64_t* q_full = empty + kSlots;
  uint64_t* q_empty = q_full + 1;                                 // the last S of a segment is done
  uint64_t* s_full = q_empty + 1;                                 // [2] S, and the P V before it
  uint64_t* p_full = s_full + 2;                                  // [2][2] a half of P has replaced S (and the last segment's O was read)
  uint64_t* o_full = p_full + 4;                                  // [2] the segment's O
  uint64_t* info_full = o_full + 2;                               // [kInfo]
  uint64_t* final_bar = info_full + kInfo;
  volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(smem + S::kMisc);   // bit h: page h of the tile is there
  volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kMisc + kInfo * 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc + kInfo * 4 + 4);

  const int n_own = 2 * p.teams * p.stages;
  own::Control oc;
  oc.full = reinterpret_cast<uint64_t*>(smem + S::kOwn);
  oc.empty = oc.full + n_own;
  oc.valid = reinterpret_cast<volatile int*>(oc.empty + n_own);
  oc.abort = abort;

  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  if (warp == 2) {
    for (int i = lane; i < n_own; i += kWarp) {
      sm100::mbar_init(&oc.full[i], 1);
      sm100::mbar_init(&oc.empty[i], p.row_warps);
    }
    sm100::fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], 1);
    }
    sm100::mbar_init(q_full, 1);
    sm100::mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&p_full[2 * i], 4);
      sm100::mbar_init(&p_full[2 * i + 1], 4);
      sm100::mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) sm100::mbar_init(&info_full[i], 1);
    sm100::mbar_init(final_bar, 1);
    *abort = 0;
    sm100::fence_barrier_init();
    sm100::tma_prefetch_desc(&tm_q);
    sm100::tma_prefetch_desc(&tm_k);
    sm100::tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    sm100::tmem_alloc(tmem_slot, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot, sbase = sm100::smem_u32(smem);
  // Everything up to here may run while the append still does; what follows
  // reads what it writes.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // Prefix or own pages: pairs of CTAs do the same, spread evenly over the grid.
  // (A cluster of two has the two SMs of a TPC, which share a way to L2: a
  // prefix CTA beside one that reads own pages took 177 us instead of 147, 256
  // requests behind 8192 shared tokens.)
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int own_pairs = pairs - (__ldcg(&p.view.head->ctas) + 1) / 2;
  const int own_before = pair * own_pairs / pairs;
  if ((pair + 1) * own_pairs / pairs > own_before) {
    // ----------------------------------------------------------- own pages
    // (72 + 2 x 216 = 3 x 168 registers a thread)
    const int cta = own_before * 2 + blockIdx.x % 2;
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      own::producer<D, OWN_KEYS>(tm_k, tm_v, p, smem, oc, cta);
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      own::consumer<D, OWN_KEYS>(p, smem, oc, cta, warp - 4);
    }
    __syncthreads();
    if (warp == 1) sm100::tmem_dealloc(tmem, 512);
    return;
  }
  const int prefix_cta = blockIdx.x - own_before * 2;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {   // the whole warp
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort) ? 1 : 0) != 0;
  };

  // Registers: 168 a thread at launch; the softmax warps take what the others
  // leave (88 + 2 x 208 = 3 x 168).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA
      Walk walk(p, prefix_cta);
      Seg seg;
      const uint64_t keep = sm100::l2_policy_evict_last();
      const PrefixShape& shape = p.view.shape;
      const int heads = min(p.group, kRows);
      int n = 0, tile = 0, sn = 0;               // tiles filled, tiles of keys, segments
      while (ok && walk.next(seg)) {
        if (sn > 0) ok = wait(q_empty, (uint32_t)((sn - 1) & 1));
        if (!ok) break;
        if (lane == 0) {
          sm100::mbar_arrive_expect_tx(q_full, (uint32_t)(seg.nsub * (D / 64) * heads * shape.tokens * 128));
          for (int x = 0; x < seg.nsub; ++x) {
            const int sub = seg.sub0 + x;
            const int token = seg.first * p.R + (shape.chunks > 1 ? sub / shape.chunks : sub * shape.tokens);
            const int head = shape.chunks > 1 ? sub % shape.chunks * kRows : 0;
            for (int c = 0; c < D / 64; ++c)
              sm100::tma_load_4d(smem + S::kQ + x * S::kTile + c * S::kChunk, &tm_q, q_full, c * 64, head, seg.kvh, token, keep);
          }
        }
        ++sn;
        for (int u = seg.u0; u < seg.u1 && ok; u += 16) {
          // the ids of 32 pages, one a lane; a page that is not there reads as zeros (beyond the cache)
          int id = -1;
          const int page = u * 2 + lane;
          if (page < seg.blocks && page < seg.u1 * 2) {
            id = p.block_table[(int64_t)seg.first * p.max_blocks + page];
            if (id < 0 || id >= p.num_blocks) {
              raise_error(p.err, MTP_ERR_BLOCK_ID);
              id = -1;
            }
          }
          for (int y = 0; y < min(16, seg.u1 - u) && ok; ++y, ++tile) {
            const int id0 = __shfl_sync(0xffffffffu, id, 2 * y), id1 = __shfl_sync(0xffffffffu, id, 2 * y + 1);
            for (int kv = 0; kv < 2 && ok; ++kv, ++n) {
              const int slot = n % kSlots;
              ok = n < kSlots || wait(&empty[slot], (uint32_t)((n / kSlots - 1) & 1));
              if (!ok) break;
              if (lane == 0) {
                if (kv == 0) {
                  info[tile % kInfo] = (id0 >= 0 ? 1u : 0u) | (id1 >= 0 ? 2u : 0u);
                  sm100::mbar_arrive(&info_full[tile % kInfo]);
                }
                sm100::mbar_arrive_expect_tx(&full[slot], S::kTile);
                uint8_t* to = smem + S::kRing + slot * S::kTile;
                const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;   // boxes of 32 keys x 64 dims
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int id = x < 2 ? id0 : id1;
                    sm100::tma_load_4d(to + c * S::kChunk + x * (S::kChunk / 4), map, &full[slot], c * 64, seg.kvh, x % 2 * own::kBox,
                                       id < 0 ? p.num_blocks : id, keep);
                  }
                }
              }
              __syncwarp();
            }
          }
        }
      }
      if (!ok) {
        *abort = 1;
        if (lane == 0) raise_error(p.err, MTP_ERR_TIMEOUT);
      }
      // Every copy issued lands before the CTA may exit.
      if (lane == 0) {
        for (int x = max(0, n - kSlots); x < n; ++x)
          sm100::mbar_wait_timeout(&full[x % kSlots], (uint32_t)((x / kSlots) & 1), sm100::kWaitTimeoutNs);
        if (sn > 0) sm100::mbar_wait_timeout(q_full, (uint32_t)((sn - 1) & 1), sm100::kWaitTimeoutNs);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA
      // (The whole warp walks, so that descriptors stay uniform; one elected
      // lane issues.)
      Walk walk(p, prefix_cta);
      Seg seg;
      constexpr uint32_t idesc_s = sm100::idesc_bf16_f32(128, kKeys);
      constexpr uint32_t idesc_o = sm100::idesc_bf16_f32(128, D) | (1u << 16);   // V MN-major
      const uint64_t qd = sm100::smem_desc_sw128_kmajor(sbase + S::kQ);
      const uint64_t kd = sm100::smem_desc_sw128_kmajor(sbase + S::kRing);
      const uint64_t vd = desc_mnmajor(sbase + S::kRing, S::kChunk);
      auto issue_s = [&](int x, int slot) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t at = (uint64_t)((kk >> 2) * (S::kChunk >> 4) + (kk & 3) * 2);
          sm100::tc_mma_bf16(tmem + x * 128, qd + (uint64_t)(x * (S::kTile >> 4)) + at, kd + (uint64_t)(slot * (S::kTile >> 4)) + at,
                             idesc_s, kk > 0 ? 1u : 0u);
        }
      };
      int n = 0, sn = 0;                         // tiles of the ring that have been waited for
      uint32_t p_phase[2] = {0, 0};
      while (ok && walk.next(seg)) {
        const int tiles = seg.u1 - seg.u0, last_x = seg.nsub - 1;
        ok = wait(q_full, (uint32_t)(sn & 1)) && wait(&full[n % kSlots], (uint32_t)((n / kSlots) & 1));
        if (!ok) break;
        ++sn;
        sm100::tc_fence_after();
        if (sm100::elect_one()) {
          for (int x = 0; x < seg.nsub; ++x) {
            issue_s(x, n % kSlots);
            sm100::tc_commit(&s_full[x]);
          }
          sm100::tc_commit(&empty[n % kSlots]);
          if (tiles == 1) sm100::tc_commit(q_empty);
        }
        __syncwarp();
        ++n;
        for (int i = 0; i < tiles && ok; ++i) {
          const int v_slot = n % kSlots, k_slot = (n + 1) % kSlots;
          const bool more = i + 1 < tiles;
          ok = wait(&full[v_slot], (uint32_t)((n / kSlots) & 1));
          for (int x = 0; x < seg.nsub && ok; ++x) {
            for (int h = 0; h < 2; ++h) {
              ok = wait(&p_full[2 * x + h], p_phase[x]);
              if (!ok) break;
              sm100::tc_fence_after();
              if (sm100::elect_one()) {
#pragma unroll
                for (int kk = h * 4; kk < h * 4 + 4; ++kk)
                  mma_ts(tmem + kColO + x * 128, tmem + x * 128 + kk * 8, vd + (uint64_t)(v_slot * (S::kTile >> 4) + kk * 128),
                         idesc_o, i > 0 || kk > 0 ? 1u : 0u);
                if (h == 1) {
                  if (x == last_x) sm100::tc_commit(&empty[v_slot]);
                  if (!more) sm100::tc_commit(&o_full[x]);
                }
              }
              __syncwarp();
            }
            if (!ok) break;
            p_phase[x] ^= 1u;
            if (more) {
              if (x == 0) {
                ok = wait(&full[k_slot], (uint32_t)(((n + 1) / kSlots) & 1));
                if (!ok) break;
                sm100::tc_fence_after();
              }
              if (sm100::elect_one()) {
                issue_s(x, k_slot);
                sm100::tc_commit(&s_full[x]);
                if (x == last_x) {
                  sm100::tc_commit(&empty[k_slot]);
                  if (i + 2 == tiles) sm100::tc_commit(q_empty);
                }
              }
              __syncwarp();
            }
          }
          n += more ? 2 : 1;
        }
      }
      if (!ok) {
        *abort = 1;
        if (lane == 0) raise_error(p.err, MTP_ERR_TIMEOUT);
      }
      // Every MMA has completed before shared memory and TMEM go.
      if (sm100::elect_one()) sm100::tc_commit(final_bar);
      __syncwarp();
      sm100::mbar_wait_timeout(final_bar, 0, sm100::kWaitTimeoutNs);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------- softmax
    Walk walk(p, prefix_cta);
    Seg seg;
    const int x = (warp - 4) / 4, row = threadIdx.x % 128;       // TMEM lanes of warp w: 32 (w % 4) and up
    const uint32_t lane0 = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * 128 + lane0, to = tmem + kColO + x * 128 + lane0;
    const float f = p.sm_scale * kLog2e;
    int tile = 0;
    uint32_t s_phase = 0, o_phase = 0;
    while (ok && walk.next(seg)) {
      if (x >= seg.nsub) {
        tile += seg.u1 - seg.u0;
        continue;
      }
      float m = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      for (int u = seg.u0; u < seg.u1; ++u, ++tile) {
        // (the marks second: S is there only when they are, and the TMA warp is at most seven tiles ahead)
        ok = wait(&s_full[x], s_phase) && wait(&info_full[tile % kInfo], (uint32_t)((tile / kInfo) & 1));
        if (!ok) break;
        s_phase ^= 1u;
        const uint32_t mark = info[tile % kInfo];
        sm100::tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          sm100::tmem_ld_32x32b_x32(ts + c * 32, r);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(r[i]);
        }
        sm100::tmem_ld_wait();
        if (mark != 3u) {                      // rare: an odd end, a bad id
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (!((mark >> (i >> 6)) & 1u)) s[i] = -INFINITY;
        }
        float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 128; i += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = i + e + 4 < 128 ? fmaxf(fmaxf(t[e], s[i + e]), s[i + e + 4]) : fmaxf(t[e], s[i + e]);
        }
        float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * f;
        if (mark != 0) top = fmaxf(top, kNoWeight);
        if (u == seg.u0) {
          m = top;
        } else {
          const bool move = top > m + kLazy || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, move)) {
            const float a = !move ? 1.0f : m == -INFINITY ? 0.0f : ex2(m - top);
            if (move) m = top;
            l0 *= a;
            l1 *= a;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              sm100::tmem_ld_32x32b_x32(to + c * 32, r);
              sm100::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * a);
              tmem_st_x32(to + c * 32, r);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : -m;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float &a = s[c * 32 + 2 * i], &b = s[c * 32 + 2 * i + 1];
            fma2(a, b, f, base);
            a = ex2(a);
            b = ex2(b);
            w[i] = pack_bf16(a, b);
          }
          tmem_st_x16(ts + c * 16, w);
          if (c % 2 == 1) {                    // a half of the keys: its P V may begin
            tmem_st_wait();
            sm100::tc_fence_before();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&p_full[2 * x + c / 2]);
          }
        }
        // (the sums while the products run)
        float l2 = 0.0f, l3 = 0.0f;
#pragma unroll
        for (int i = 0; i < 128; i += 4) {
          add2(l0, l1, s[i], s[i + 1]);
          add2(l2, l3, s[i + 2], s[i + 3]);
        }
        l0 += l2;
        l1 += l3;
      }
      if (!ok) break;
      ok = wait(&o_full[x], o_phase);
      if (!ok) break;
      o_phase ^= 1u;
      sm100::tc_fence_after();
      const int64_t at = seg.part * 2 + x;
      p.view.stats[at * kRows + row] = make_float2(m, l0 + l1);
      float4* parts = reinterpret_cast<float4*>(p.view.parts + at * kRows * D) + row;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        sm100::tmem_ld_32x32b_x32(to + c * 32, r);
        sm100::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          parts[(c * 8 + i) * kRows] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                   __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
      }
      sm100::tc_fence_before();
    }
    if (!ok) {
      *abort = 1;
      if (lane == 0) raise_error(p.err, MTP_ERR_TIMEOUT);
    }
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const mtp_prefix_attn_args& a, const PrefixParams& p, int ctas, cudaStream_t s) {
  const PrefixShape& shape = p.view.shape;
  CUtensorMap tq, tk, tv;
  const cuuint64_t group = (cuuint64_t)p.group, Hkv = (cuuint64_t)a.Hkv;
  const cuuint64_t qdims[4] = {(cuuint64_t)D, group, Hkv, (cuuint64_t)a.B * p.R};
  const cuuint64_t qstrides[3] = {D * 2, group * D * 2, (cuuint64_t)a.Hq * D * 2};
  const cuuint32_t qbox[4] = {64, (cuuint32_t)std::min(p.group, kRows), 1, (cuuint32_t)shape.tokens};
  const cuuint64_t dims[4] = {(cuuint64_t)D, Hkv, (cuuint64_t)kBlock, (cuuint64_t)a.num_blocks};
  const cuuint64_t strides[3] = {D * 2, Hkv * D * 2, kBlock * Hkv * D * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)own::kBox, 1};
  if (!make_bf16_map(&tq, a.q, 4, qdims, qstrides, qbox) || !make_bf16_map(&tk, a.k_cache, 4, dims, strides, box) ||
      !make_bf16_map(&tv, a.v_cache, 4, dims, strides, box))
    return cudaErrorInvalidValue;
  const auto kernel = p.own_keys == kBlock ? prefix_kernel<D, kBlock> : prefix_kernel<D, own::kBox>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_behind_append(kernel, (unsigned)ctas, kThreads, Smem<D>::kBytes, s, tq, tk, tv, p);
}

template <int D>
void lay_out(const mtp_prefix_attn_args& a, OwnPlan* pl) {
  const int blocks = (a.Hq / a.Hkv * (a.D + 1) + 15) / 16;     // of 16 rows
  pl->row_tiles = (blocks + own::kWarps - 1) / own::kWarps;
  pl->row_warps = (blocks + pl->row_tiles - 1) / pl->row_tiles;
  // As many teams as there are warps for, with two stages each at least. Stages of 64 keys where that takes no team away: a
  // warp then waits, and goes through a softmax, half as often, which is most of what it does (128 requests of 48 rows,
  // 1000 own tokens: 147 us with 32, 128 so; 48 rows of 64 dims: 53 and 46; of 100 tokens: 42.9 and 43.2, 21.5 and 21.4).
  // Or one team of eight where there is work for all: without a prefix (16 rows of 64 dims, us with 32 keys and with 64) 1024
  // items of 1000 tokens 65.2, 54.5, of 500 to 1500 69.6, 68.5; 512 of 1000 37.8, 33.9; 64 of 8000 36.1, 38.3, of 500 to 1500
  // 17.7, 18.0. Behind a prefix it can lose, since the SMs are shared out by costs that do not know the stages: 1024 items of
  // 1000 behind 2048 tokens 69.5, 87.3; 2048 of 250 behind 4096 68.9, 74.6, of 1000 144.7, 143.6.
  constexpr int kStages = Smem<D>::kOwnStages, kManyItems = 1024;
  const int teams = std::min(own::kWarps / pl->row_warps, kStages / 2), fewer = std::min(teams, kStages / 4);
  const bool many = (long long)a.B * a.Hkv * pl->row_tiles >= kManyItems;
  pl->keys = fewer == teams || (many && fewer * 8 >= teams * 7) ? kBlock : own::kBox;
  pl->teams = pl->keys == kBlock ? fewer : teams;
  pl->stages = std::min(own::kMaxStages, kStages * own::kBox / pl->keys / pl->teams);
}

}  // namespace

OwnPlan plan_prefix_own(const mtp_prefix_attn_args& a) {
  OwnPlan pl{};
  a.d == 128 ? lay_out<128>(a, &pl) : lay_out<64>(a, &pl);
  return pl;
}

cudaError_t launch_prefix_tc(const mtp_prefix_attn_args& a, const PrefixParams& p, int ctas, cudaStream_t s) {
  return a.d == 128 ? launch<128>(a, p, ctas, s) : launch<64>(a, p, ctas, s);
}

}  // namespace mtp
