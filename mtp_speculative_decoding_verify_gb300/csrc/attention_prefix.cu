// mtp_verify_attention_prefix: verify attention of requests whose tables begin
// with the same blocks. The C entry, the append, the plan, and the kernels of
// fp32 rows.
//
// "Multi Token Prediction" note, overall flow for K=3 draft tokens, step 2, as
// in mtp_verify_attention: the R verify rows of a request attend the reused
// cache and each other. A softmax over slots falls into one over the group's
// prefix and one over the request's own slots,
//   o = (o_p 2^(m_p - m) + o_w 2^(m_w - m)) / (l_p 2^(m_p - m) + l_w 2^(m_w - m)),
// m the larger maximum. Over the prefix the rows of all requests of the group
// are one matrix, so K and V are read once for all of them and the product
// is as tall as the group is large.
//
// Launches: the append, which also works out the shares of work in one more
// CTA; prefix and own pages (fp32 rows: one after the other); the join.
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "attention_prefix.h"
#include "attention_prefix_own.cuh"
#include "attention_window.h"

namespace mtp {
int device_context(unsigned** err, int* sm_count);
int set_error(int code, const char* msg);
int set_cuda_error(cudaError_t e, const char* what);
void set_launch_count(int n);

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------- append
// One CTA per (request, verify token): its K and V rows go to slot ctx+j of the
// cache, 16 bytes a thread; a request that its group's prefix rules out is left
// alone. The last CTA works out the shares.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) prefix_append_kernel(const uint4* __restrict__ k_new,
                                                                       const uint4* __restrict__ v_new,
                                                                       uint4* __restrict__ k_cache, uint4* __restrict__ v_cache,
                                                                       const int32_t* __restrict__ block_table, int vecs,
                                                                       int num_blocks, const PrefixSchedule prefix) {
  asm volatile("griddepcontrol.launch_dependents;");   // (the kernels behind it may set up)
  if (blockIdx.x == 0) {                       // first, since the others wait for it
    prefix_schedule<kAppendThreads>(prefix);
    return;
  }
  const int R = prefix.R, bj = blockIdx.x - 1, b = bj / R, j = bj % R;
  const int ctx = prefix.ctx_lens[b];
  bool bad;
  const int g = find_group(prefix.group_starts, prefix.G, prefix.B, b, &bad);
  const int first = own_first(g < 0 ? 0 : prefix.prefix_blocks[g], ctx, prefix.max_blocks, R);
  if (first < 0) {
    if (threadIdx.x == 0) raise_error(prefix.err, MTP_ERR_LENGTH);
    return;
  }
  const int blk = block_table[(int64_t)b * prefix.max_blocks + (ctx + j) / kBlock];
  if (blk < 0 || blk >= num_blocks) {
    if (threadIdx.x == 0) raise_error(prefix.err, MTP_ERR_BLOCK_ID);
    return;
  }
  const int64_t from = (int64_t)bj * vecs, to = ((int64_t)blk * kBlock + (ctx + j) % kBlock) * vecs;
  for (int i = threadIdx.x; i < 2 * vecs; i += kAppendThreads) {
    if (i < vecs) k_cache[to + i] = k_new[from + i];
    else v_cache[to + i - vecs] = v_new[from + i - vecs];
  }
}

// ---------------------------------------------------------------- fp32 rows
// Prefix and own pages on FFMA, by the same kernel: a CTA walks its share of the
// line (attention_prefix.h): for each item ROWS rows of one KV head, page after
// page. A thread holds RPT rows x 4 keys of the scores and RPT rows x D/16 dims of
// the output, so that a value from shared memory serves several products; P takes
// K's place once the scores are there, and two (64 rows) or three (16 rows) CTAs
// share an SM, one loading while the others compute. Own pages, of few rows,
// take 16 a tile; the prefix 64 where a KV head has more than 32 over all
// requests, else 16, and then one launch does both lines (2 rows of 8 KV heads
// behind 6400 tokens: 84 us with 64, 47 us with 16; 4 requests of 4 rows behind
// 1024: 15.4 us in two launches, 13.6 in one). FFMA and shared memory bound it: 32
// TFLOP/s (512 rows a KV head behind 2048 tokens), 1.4 TB/s over own pages of 16
// rows.
// Own pages: a hidden slot's P is held as -1 and takes no part in the products (0
// x NaN), and slots behind the last token are read as 0.
template <int D, int ROWS>
struct SimtCfg {
  static constexpr int kThreads = ROWS == 64 ? 256 : 128, kRpt = ROWS * 16 / kThreads, kCtas = ROWS == 64 ? 2 : 3;
  static constexpr int kQ = 0, kK = kQ + ROWS * (D + 4), kV = kK + kBlock * (D + 4), kFloats = kV + kBlock * D;
  static constexpr int kBytes = kFloats * (int)sizeof(float);
  static_assert(ROWS * (kBlock + 4) <= kBlock * (D + 4), "P fits in K's place");
  static_assert(kCtas * (kBytes + 1024) <= 228 * 1024, "the CTAs fit an SM");
};

// An item of either line.
struct SimtItem {
  int table;                                   // the request whose table row names the pages
  int page0, page1;                            // pages of it
  int kvh, tile;                               // KV head; tile of rows of the group, or of the request
  int ctx;                                     // own pages: the request's
  int64_t part;
};

// The CTAs of one line; cta: among them.
template <int D, int ROWS, bool kOwn>
__device__ __forceinline__ void simt_line(const PrefixParams& p, int cta) {
  using S = SimtCfg<D, ROWS>;
  constexpr int kThreads = S::kThreads, RPT = S::kRpt;
  constexpr int QS = D + 4, PS = kBlock + 4, E = D / 16;   // row strides; output dims of a thread
  extern __shared__ float smem[];
  float *qs = smem + S::kQ, *ks = smem + S::kK, *vs = smem + S::kV, *ps = ks;
  const PrefixView& v = p.view;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const float f = p.sm_scale * kLog2e;
  const float *q = static_cast<const float*>(p.q), *kc = static_cast<const float*>(p.k_cache), *vc = static_cast<const float*>(p.v_cache);
  auto load4 = [](const float* at) { return __ldg(reinterpret_cast<const float4*>(at)); };

  // What the two lines have apart: the next item.
  PrefixStart start{};
  int pos = 0, end = 0;
  if constexpr (!kOwn) {
    if (cta < __ldcg(&v.head->ctas)) {
      start.group = load_group(&v.starts[cta].group);
      start.gi = __ldcg(&v.starts[cta].gi);
      pos = __ldcg(&v.starts[cta].pos);
      end = __ldcg(&v.starts[cta].end);
    }
  }
  own::OwnWalk walk(p, kOwn ? cta : 0x7fffffff);
  auto next = [&](SimtItem& it) -> bool {
    if constexpr (kOwn) {
      own::OwnWalk::Seg s;
      if (!walk.next(s)) return false;
      it = SimtItem{s.b, s.first + s.i0, s.first + s.i1, s.hr / p.row_tiles, s.hr % p.row_tiles, s.ctx,
                    (int64_t)s.b * walk.heads + s.hr + cta};
    } else {
      if (pos >= end) return false;
      PrefixGroup& g = start.group;
      while (g.units == 0 || pos >= g.line + g.tiles * p.Hkv * g.units) g = load_group(v.groups + ++start.gi);
      const int k = (pos - g.line) / g.units, u0 = pos - g.line - k * g.units, u1 = min(g.units, u0 + end - pos);
      it = SimtItem{g.first, u0, u1, k / g.tiles, k % g.tiles, 0, (int64_t)g.item + k + cta};
      pos += u1 - u0;
    }
    return true;
  };

  SimtItem it;
  while (next(it)) {
    __syncthreads();                           // the last item's Q has been read
    for (int x = tid; x < ROWS * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      int64_t token;                           // (request, verify token)
      int hh;
      bool in;
      if constexpr (kOwn) {
        const int row = it.tile * ROWS + r;
        token = (int64_t)it.table * p.R + row / p.group;
        hh = row % p.group;
        in = row < p.rows;
      } else {
        token = (int64_t)it.table * p.R + (v.shape.chunks > 1 ? it.tile / v.shape.chunks : it.tile * v.shape.tokens + r / p.group);
        hh = v.shape.chunks > 1 ? it.tile % v.shape.chunks * ROWS + r : r % p.group;
        in = token < (int64_t)p.B * p.R && hh < p.group && (v.shape.chunks > 1 || r < v.shape.tokens * p.group);
      }
      float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // other rows compute on 0
      if (in) w = load4(q + (token * p.Hq + it.kvh * p.group + hh) * D + c);
      *reinterpret_cast<float4*>(qs + r * QS + c) = w;
    }
    uint32_t path[RPT];                        // own pages: the verify keys that the row sees
    float m[RPT], l[RPT], o[RPT][E];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      path[i] = 0;
      if constexpr (kOwn)
        path[i] = tree_path_mask(v.parents, it.table, p.R, min(it.tile * ROWS + RPT * ty + i, p.rows - 1) / p.group, p.err);
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.0f;
    }
    for (int page = it.page0; page < it.page1; ++page) {
      const int blk = __ldg(p.block_table + (int64_t)it.table * p.max_blocks + page);
      if (blk < 0 || blk >= p.num_blocks) {    // the same for every thread
        if (tid == 0) raise_error(p.err, MTP_ERR_BLOCK_ID);
        continue;
      }
      const int keys = kOwn ? min(kBlock, it.ctx + p.R - page * kBlock) : kBlock;
      const bool masked = kOwn && page * kBlock + kBlock - 1 > it.ctx;
      __syncthreads();                         // the last page's P and V have been read
#pragma unroll 4
      for (int x = tid; x < kBlock * (D / 4); x += kThreads) {
        const int key = x / (D / 4), c = x % (D / 4) * 4;
        const int64_t at = (((int64_t)blk * kBlock + key) * p.Hkv + it.kvh) * D + c;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
        if (key < keys) a = __ldcg(reinterpret_cast<const float4*>(kc + at)), b = __ldcg(reinterpret_cast<const float4*>(vc + at));
        *reinterpret_cast<float4*>(ks + key * QS + c) = a;
        *reinterpret_cast<float4*>(vs + key * D + c) = b;
      }
      __syncthreads();
      float s[RPT][4];                         // rows RPT ty + i, keys tx + 16 x
#pragma unroll
      for (int i = 0; i < RPT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 a[RPT], b[4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) a[i] = *reinterpret_cast<const float4*>(qs + (RPT * ty + i) * QS + c);
#pragma unroll
        for (int x = 0; x < 4; ++x) b[x] = *reinterpret_cast<const float4*>(ks + (tx + 16 * x) * QS + c);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
#pragma unroll
          for (int x = 0; x < 4; ++x) s[i][x] += a[i].x * b[x].x + a[i].y * b[x].y + a[i].z * b[x].z + a[i].w * b[x].w;
        }
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        unsigned hidden = 0;                   // of this thread's keys
        if (kOwn && masked) {
#pragma unroll
          for (int x = 0; x < 4; ++x) hidden |= (tree_hidden(page * kBlock + tx + 16 * x, it.ctx, path[i]) ? 1u : 0u) << x;
        }
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[i][x] = (hidden >> x) & 1 ? -INFINITY : s[i][x] * f;
          top = fmaxf(top, s[i][x]);
        }
        bool seen = hidden != 15u;             // the row sees a slot of the page
#pragma unroll
        for (int z = 8; z > 0; z >>= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
          if (kOwn) seen |= __shfl_xor_sync(0xffffffffu, (int)seen, z) != 0;
        }
        const float n = fmaxf(fmaxf(m[i], top), seen ? kNoWeight : -INFINITY);
        const float base = n == -INFINITY ? 0.0f : n;
        const float a = m[i] == -INFINITY ? 0.0f : exp2f(m[i] - base);
        m[i] = n;
        l[i] *= a;                             // (of this thread's keys; joined at the end)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float w = exp2f(s[i][x] - base);
          s[i][x] = (hidden >> x) & 1 ? -1.0f : w;
          if (!((hidden >> x) & 1)) l[i] += w;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] *= a;
      }
      __syncthreads();                         // K has been read
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
#pragma unroll
        for (int x = 0; x < 4; ++x) ps[(RPT * ty + i) * PS + tx + 16 * x] = s[i][x];
      }
      __syncwarp();                            // (a row's P is written and read by one warp)
      auto products = [&](auto masked_c) {
        constexpr bool kMasked = decltype(masked_c)::value;
#pragma unroll 2
        for (int key = 0; key < kBlock; key += 4) {
          float a[RPT][4];
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(ps + (RPT * ty + i) * PS + key);
            a[i][0] = w.x, a[i][1] = w.y, a[i][2] = w.z, a[i][3] = w.w;
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float b[E];                        // dims 4 tx + 64 (e / 4) + e % 4
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const float4 w = *reinterpret_cast<const float4*>(vs + (key + y) * D + 4 * tx + e * 16);
              b[e] = w.x, b[e + 1] = w.y, b[e + 2] = w.z, b[e + 3] = w.w;
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              if (kMasked && a[i][y] < 0.0f) continue;
#pragma unroll
              for (int e = 0; e < E; ++e) o[i][e] += a[i][y] * b[e];
            }
          }
        }
      };
      if (kOwn && masked) products(std::true_type());
      else products(std::false_type());
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
      for (int z = 8; z > 0; z >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], z);
      const int r = RPT * ty + i;
      if (tx == 0) (kOwn ? v.own_stats : v.stats)[it.part * ROWS + r] = make_float2(m[i], l[i]);
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        float* to = kOwn ? v.own_parts + (it.part * ROWS + r) * D + (tx + e * 4) * 4
                         : v.parts + it.part * ROWS * D + ((tx + e * 4) * ROWS + r) * 4;
        *reinterpret_cast<float4*>(to) = make_float4(o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3]);
      }
    }
  }
}

// kPrefix, kOwn or kBoth, some CTAs each (as many as the schedule gives the prefix).
enum SimtLines { kPrefix, kOwn, kBoth };

template <int D, int ROWS, SimtLines kLines>
__global__ void __launch_bounds__((SimtCfg<D, ROWS>::kThreads), (SimtCfg<D, ROWS>::kCtas))
    prefix_simt_kernel(const PrefixParams p, int behind_prefix) {
  // (Own pages: the append is complete when the prefix's kernel, which waited for it, lets this grid begin. What that
  // kernel writes is not read here.)
  if (!behind_prefix) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");   // (the next one reads what the append left before it waits)
  if constexpr (kLines == kPrefix) {
    simt_line<D, ROWS, false>(p, blockIdx.x);
  } else if constexpr (kLines == kOwn) {
    simt_line<D, ROWS, true>(p, blockIdx.x);
  } else {
    const int ctas = (__ldcg(&p.view.head->ctas) + 1) / 2 * 2;
    if ((int)blockIdx.x < ctas) simt_line<D, ROWS, false>(p, blockIdx.x);
    else simt_line<D, ROWS, true>(p, blockIdx.x - ctas);
  }
  if (behind_prefix) asm volatile("griddepcontrol.wait;" ::: "memory");   // whoever waits for this grid waits for that one too
}

// ----------------------------------------------------------- checks and plan
int fail(const char* msg) {
  char buf[256];
  snprintf(buf, sizeof buf, "mtp_verify_attention_prefix: %s", msg);
  return set_error(MTP_INVALID_ARG, buf);
}
int unsupported(const char* msg) {
  char buf[256];
  snprintf(buf, sizeof buf, "mtp_verify_attention_prefix: %s", msg);
  return set_error(MTP_UNSUPPORTED, buf);
}

int check_prefix(const mtp_prefix_attn_args* a) {
  if (!a) return fail("args is NULL");
  if (a->B < 0 || a->G < 0) return fail("B and G must be >= 0");
  if (a->D < 0 || a->D > MTP_MAX_DRAFTS) return fail("D outside [0, 15]");
  if (a->block_size != MTP_BLOCK_SIZE) return fail("block_size must be 64");
  if (a->max_blocks <= 0 || a->max_blocks > (1 << 24) || a->num_blocks <= 0)
    return fail("max_blocks outside [1, 2^24], or num_blocks <= 0");
  if (a->Hq <= 0 || a->Hkv <= 0 || a->Hkv > (1 << 16) || a->Hq % a->Hkv) return fail("Hkv outside [1, 2^16], or Hq % Hkv != 0");
  if (a->dtype != MTP_F32 && a->dtype != MTP_BF16) return fail("dtype");
  if (!(a->sm_scale > 0.0f && a->sm_scale <= 1e30f)) return fail("sm_scale must be > 0 and finite");
  if (a->d != 64 && a->d != 128) return unsupported("head dim must be 64 or 128");
  if ((long long)a->B * (a->D + 1) * a->Hq > (1 << 29) || a->Hq / a->Hkv > (1 << 15))
    return unsupported("B x R x Hq > 2^29, or Hq / Hkv > 2^15");
  if ((long long)a->B * a->max_blocks > 0x7fffffffll) return unsupported("B x max_blocks >= 2^31");
  if (a->G > (1 << 20)) return unsupported("G > 2^20");
  if (a->B == 0) return MTP_OK;
  if (!a->q || !a->k_new || !a->v_new || !a->k_cache || !a->v_cache || !a->block_table || !a->ctx_lens || !a->out)
    return fail("a required pointer is NULL");
  if (a->G > 0 && (!a->group_starts || !a->prefix_blocks)) return fail("group_starts / prefix_blocks is NULL");
  const uintptr_t any = (uintptr_t)a->q | (uintptr_t)a->k_new | (uintptr_t)a->v_new | (uintptr_t)a->k_cache |
                        (uintptr_t)a->v_cache | (uintptr_t)a->out;
  if (any % 16) return fail("q, out, k_new, v_new and the caches must be 16-byte aligned");
  return MTP_OK;
}

bool fp32_rows(const mtp_prefix_attn_args& a) { return a.dtype == MTP_F32; }

struct PrefixPlan {
  PrefixShape shape;
  int ctas;                            // of the prefix (bf16: and the own pages)
  int own_ctas;                        // fp32
  OwnPlan own;
  // byte offsets in the workspace
  size_t head, groups, group_of, first, starts, own_starts, parts, stats, own_head, pages, own_parts, own_stats, bytes;
};

// False: more units of work than 31 bits count. (A KV head has at most B R group / 8 tiles of rows, B + 2 G more of which
// are only part full, and a tile at most max_blocks units.)
constexpr const char* kTooMany = "(B R Hq / 8 + (B + 2 G) Hkv) max_blocks is too large: more units of work than 31 bits count";
bool plan_prefix(const mtp_prefix_attn_args& a, int sm_count, PrefixPlan* pl) {
  const int group = a.Hq / a.Hkv, R = a.D + 1, G = std::min(a.G, a.B);   // (empty groups have no items)
  const bool fp32 = fp32_rows(a);
  if (fp32) {
    const int rows = a.B * R * group > 32 ? 64 : 16;
    pl->shape = prefix_shape(rows, 1, 1, group);
    pl->ctas = rows == 64 ? 2 * sm_count : std::max(4, 3 * sm_count / 2 * 2);
    pl->own_ctas = rows == 64 ? 3 * sm_count : 0;
    pl->own = OwnPlan{(R * group + 15) / 16, 1, 1, 0, 0};
  } else {
    pl->shape = prefix_shape(kPrefixTcRows, 2, 2, group);
    pl->ctas = std::max(4, sm_count / 2 * 2);   // pairs
    pl->own_ctas = 0;
    pl->own = plan_prefix_own(a);
  }
  const long long limit = 0x7fffffffll - 0x10000;
  // Items of all groups: the tiles of all rows, and the ones that each group leaves part of empty.
  const long long tiles = ((long long)a.B * R / pl->shape.tokens + G) * pl->shape.chunks;
  const long long items = G == 0 ? 0 : (tiles / pl->shape.subs + G) * a.Hkv;
  if (items * a.max_blocks > limit) return false;
  const size_t results = G == 0 ? 0 : ((size_t)items + pl->ctas) * pl->shape.subs * pl->shape.rows;   // rows of partial results
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += (n + 255) / 256 * 256;
    return was;
  };
  pl->head = take(sizeof(PrefixHead));
  pl->groups = take((size_t)a.G * sizeof(PrefixGroup));
  pl->group_of = take((size_t)a.B * sizeof(int32_t));
  pl->first = take((size_t)a.B * sizeof(int32_t));
  pl->starts = take((size_t)pl->ctas * sizeof(PrefixStart));
  pl->stats = take(results * sizeof(float2));
  pl->parts = take(results * a.d * sizeof(float));
  const long long own_items = (long long)a.B * a.Hkv * pl->own.row_tiles;
  if (own_items * a.max_blocks > limit) return false;
  const size_t own_shares = (size_t)(pl->own_ctas > 0 ? pl->own_ctas : pl->ctas) * pl->own.teams;
  const size_t n = ((size_t)own_items + own_shares) * pl->own.row_warps * 16;
  pl->own_head = take(sizeof(PrefixHead));
  pl->pages = take(((size_t)a.B + 1) * sizeof(int32_t));
  pl->own_starts = take(own_shares * sizeof(OwnStart));
  pl->own_stats = take(n * sizeof(float2));
  pl->own_parts = take(n * a.d * sizeof(float));
  pl->bytes = at;
  return true;
}

template <int D, int ROWS, SimtLines kLines>
cudaError_t launch_simt(const PrefixParams& p, int ctas, int behind_prefix, cudaStream_t s) {
  using S = SimtCfg<D, ROWS>;
  const auto kernel = prefix_simt_kernel<D, ROWS, kLines>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  return launch_behind_append(kernel, (unsigned)ctas, S::kThreads, S::kBytes, s, p, behind_prefix);
}

template <int D>
cudaError_t launch_fp32(const PrefixParams& p, const PrefixPlan& pl, bool groups, cudaStream_t s) {
  if (pl.own_ctas == 0) return launch_simt<D, 16, kBoth>(p, pl.ctas, 0, s);
  if (groups) {
    const cudaError_t e = launch_simt<D, 64, kPrefix>(p, pl.ctas, 0, s);
    if (e != cudaSuccess) return e;
  }
  return launch_simt<D, 16, kOwn>(p, pl.own_ctas, groups, s);
}

}  // namespace
}  // namespace mtp

extern "C" {

size_t mtp_attention_prefix_workspace_size(const mtp_prefix_attn_args* a) {
  using namespace mtp;
  if (check_prefix(a) != MTP_OK) return 0;
  unsigned* err = nullptr;
  int sm_count = 0;
  if (device_context(&err, &sm_count) != MTP_OK) return 0;
  PrefixPlan pl;
  if (!plan_prefix(*a, sm_count, &pl)) {
    unsupported(kTooMany);
    return 0;
  }
  return pl.bytes;
}

int mtp_verify_attention_prefix(const mtp_prefix_attn_args* a, void* stream) {
  using namespace mtp;
  int rc = check_prefix(a);
  if (rc != MTP_OK) return rc;
  set_launch_count(0);
  if (a->B == 0) return MTP_OK;
  unsigned* err = nullptr;
  int sm_count = 0;
  if ((rc = device_context(&err, &sm_count)) != MTP_OK) return rc;
  PrefixPlan pl;
  if (!plan_prefix(*a, sm_count, &pl)) return unsupported(kTooMany);
  if (!a->workspace || a->workspace_bytes < pl.bytes) {
    char buf[160];
    snprintf(buf, sizeof buf, "workspace of %zu bytes needed, %zu given", pl.bytes, a->workspace ? a->workspace_bytes : (size_t)0);
    return set_error(MTP_INVALID_ARG, buf);
  }
  if ((uintptr_t)a->workspace % 256) return set_error(MTP_INVALID_ARG, "workspace must be 256-byte aligned");
  const bool fp32 = fp32_rows(*a);
  char* ws = static_cast<char*>(a->workspace);
  auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
  PrefixSchedule ps{};
  ps.head = reinterpret_cast<PrefixHead*>(ws + pl.head);
  ps.groups = reinterpret_cast<PrefixGroup*>(ws + pl.groups);
  ps.group_of = i32(pl.group_of);
  ps.first = i32(pl.first);
  ps.starts = reinterpret_cast<PrefixStart*>(ws + pl.starts);
  ps.group_starts = a->group_starts;
  ps.prefix_blocks = a->prefix_blocks;
  ps.ctx_lens = a->ctx_lens;
  ps.G = a->G;
  ps.B = a->B;
  ps.R = a->D + 1;
  ps.Hkv = a->Hkv;
  ps.max_blocks = a->max_blocks;
  ps.ctas = pl.ctas;
  ps.shape = pl.shape;
  ps.err = err;
  PrefixParams p{};
  p.q = a->q;
  p.out = a->out;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.block_table = a->block_table;
  p.ctx_lens = a->ctx_lens;
  p.err = err;
  p.B = a->B;
  p.R = ps.R;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.group = a->Hq / a->Hkv;
  p.rows = p.group * p.R;
  p.max_blocks = a->max_blocks;
  p.num_blocks = a->num_blocks;
  p.sm_scale = a->sm_scale;
  p.view.head = ps.head;
  p.view.groups = ps.groups;
  p.view.group_of = ps.group_of;
  p.view.first = ps.first;
  p.view.starts = ps.starts;
  p.view.parts = reinterpret_cast<float*>(ws + pl.parts);
  p.view.stats = reinterpret_cast<float2*>(ws + pl.stats);
  p.view.parents = a->parents;
  p.view.shape = pl.shape;
  ps.own = reinterpret_cast<PrefixHead*>(ws + pl.own_head);
  ps.pages = i32(pl.pages);
  ps.own_starts = reinterpret_cast<OwnStart*>(ws + pl.own_starts);
  ps.own_heads = p.Hkv * pl.own.row_tiles;
  ps.own_ctas = pl.own_ctas;
  ps.teams = pl.own.teams;
  if (fp32) {                          // (a page of 16 rows either way)
    ps.unit_cost = ps.page_cost = 2;
    ps.item_cost = 1;
  } else {
    // As measured, and tried 20 % up and down: 64 dims, 256 requests of 16 rows: 95 us with 2700, 82.6 with 1500, 86 with
    // 1200; 48 of 48 rows: 53.0 with 2700, 50.3 with 2000, 55.4 with 1500.
    ps.unit_cost = a->d == 128 ? 1800 : 1400;
    ps.page_cost = (a->d == 128 ? 2700 : pl.own.teams < 4 ? 2100 : 1500) / pl.own.teams;
    ps.item_cost = 1900 / pl.own.teams;
  }
  p.row_tiles = pl.own.row_tiles;
  p.row_warps = pl.own.row_warps;
  p.teams = pl.own.teams;
  p.stages = pl.own.stages;
  p.own_keys = pl.own.keys;
  p.view.own = ps.own;
  p.view.pages = ps.pages;
  p.view.own_starts = ps.own_starts;
  p.view.own_parts = reinterpret_cast<float*>(ws + pl.own_parts);
  p.view.own_stats = reinterpret_cast<float2*>(ws + pl.own_stats);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto record = [&](void* ev) { return ev ? cudaEventRecord(static_cast<cudaEvent_t>(ev), s) : cudaSuccess; };
  const int vecs = a->Hkv * a->d * (fp32 ? 4 : 2) / 16;
  prefix_append_kernel<<<a->B * p.R + 1, kAppendThreads, 0, s>>>((const uint4*)a->k_new, (const uint4*)a->v_new, (uint4*)a->k_cache,
                                                     (uint4*)a->v_cache, a->block_table, vecs, a->num_blocks, ps);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_cuda_error(e, "kv append launch");
  if ((e = record(a->timing_events[0])) != cudaSuccess) return set_cuda_error(e, "cudaEventRecord");
  if (fp32) e = a->d == 128 ? launch_fp32<128>(p, pl, a->G > 0, s) : launch_fp32<64>(p, pl, a->G > 0, s);
  else e = launch_prefix_tc(*a, p, pl.ctas, s);
  if (e != cudaSuccess) return set_cuda_error(e, "attention launch");
  e = launch_prefix_join(*a, p, s);
  if (e != cudaSuccess) return set_cuda_error(e, "attention join launch");
  if ((e = record(a->timing_events[1])) != cudaSuccess) return set_cuda_error(e, "cudaEventRecord");
  set_launch_count(pl.own_ctas > 0 && a->G > 0 ? 4 : 3);
  return MTP_OK;
}

}  // extern "C"
