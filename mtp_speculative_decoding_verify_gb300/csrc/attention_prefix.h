// Launch parameters and the shares of work of mtp_verify_attention_prefix,
// between attention_prefix.cu (entry, append, fp32 rows), attention_prefix_tc.cu
// and attention_prefix_own.cuh (bf16 rows) and attention_prefix_join.cu.
//
// The query rows of a group that share a KV head are numbered token after
// token (request, verify token), the heads of a token side by side, and cut
// into tiles of `rows` rows that hold whole tokens (rows / group of them; of
// a token with more heads than that, `rows` heads at a time). An item is
// `subs` such tiles of one group and KV head against all of the group's
// prefix. The items form a line in units of `pages` pages of keys, cut into
// an even share for each CTA. Item i's part from CTA c is partial result i + c:
// along the line, i and c never go down together, so the number is its own.
//
// The own pages of the requests form a line the same way, in pages, with
// (request, KV head, tile of rows) for items and warp teams for CTAs.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace mtp {

struct alignas(16) PrefixGroup {
  int32_t first;                    // its first request: whose table row names the prefix's blocks
  int32_t blocks;                   // of the prefix
  int32_t units, tiles;             // of an item; items of a KV head
  int32_t line, item;               // its first unit of the line and its first item
  int32_t sub_tiles, pad;           // tiles of rows of a KV head
};
struct alignas(16) PrefixHead {
  int32_t total, ctas;              // units of the line, shares
  int32_t narrow, pad;              // total x ctas fits 32 bits (a division of 64 costs what the join's other steps do together)
};
// Where a share begins.
struct alignas(16) PrefixStart {
  PrefixGroup group;
  int32_t gi;                       // which group that is
  int32_t pos, end;                 // units of the line
  int32_t pad;
};
struct alignas(16) OwnStart {
  int32_t pos, end;                 // pages of the line
  int32_t b, before, pages;         // the request, own pages of those before it (of one head), its own
  int32_t pad[3];
};

constexpr int kPrefixTcRows = 128;  // of a tile on the tensor cores: two tiles an item, two pages a unit

// Of one launch, the same on the host and on the device.
struct PrefixShape {
  int rows, subs, pages;            // rows of a tile, tiles of an item, pages of a unit
  int tokens, chunks;               // tokens that a tile holds; tiles that a token needs
};
__host__ __device__ inline PrefixShape prefix_shape(int rows, int subs, int pages, int group) {
  PrefixShape s{rows, subs, pages, 0, 0};
  s.tokens = group <= rows ? rows / group : 1;
  s.chunks = group <= rows ? 1 : (group + rows - 1) / rows;
  return s;
}

struct PrefixView {
  const PrefixHead* head;
  const PrefixGroup* groups;
  const int32_t* group_of;          // [B] group of a request that has a prefix, else -1
  const int32_t* first;             // [B] first page of a request's own; -1: the request is skipped
  const PrefixStart* starts;        // [ctas]
  float* parts;                     // [partial result][sub][d/4][rows][4]: sums of p v, not divided
  float2* stats;                    // [partial result][sub][rows]: maximum (log2 units), sum of p
  const int32_t* parents;           // [B, R] or NULL
  PrefixShape shape;
  const PrefixHead* own;            // the own pages
  const int32_t* pages;             // [B+1] own pages of the requests before each
  const OwnStart* own_starts;       // [teams]
  float* own_parts;                 // [partial result][rows of a tile][d]
  float2* own_stats;                // [partial result][rows of a tile]
};

struct PrefixParams {
  const void* q;
  void* out;
  const void *k_cache, *v_cache;
  const int32_t *block_table, *ctx_lens;
  unsigned* err;
  int B, R, Hq, Hkv, group, rows;   // rows = query rows per (request, KV head)
  int max_blocks, num_blocks;
  float sm_scale;
  int row_tiles, row_warps;         // own pages: tiles of 16 row_warps rows of a request
  int teams, stages, own_keys;      // .. bf16: teams of a CTA, stages of a team, keys of a stage
  PrefixView view;
};

struct OwnPlan {
  int row_tiles, row_warps, teams, stages, keys;
};
OwnPlan plan_prefix_own(const mtp_prefix_attn_args& a);
// bf16 rows: prefix and own pages.
cudaError_t launch_prefix_tc(const mtp_prefix_attn_args& a, const PrefixParams& p, int ctas, cudaStream_t s);
cudaError_t launch_prefix_join(const mtp_prefix_attn_args& a, const PrefixParams& p, cudaStream_t s);

// Written by one more CTA of the append.
struct PrefixSchedule {
  PrefixHead* head;                 // nullptr: nothing to prepare
  PrefixGroup* groups;
  int32_t *group_of, *first;
  PrefixStart* starts;
  const int32_t *group_starts, *prefix_blocks, *ctx_lens;
  int G, B, R, Hkv, max_blocks, ctas;
  PrefixShape shape;
  PrefixHead* own;
  int32_t* pages;
  OwnStart* own_starts;
  int own_heads, own_ctas;          // items of a request; CTAs that do own pages, 0: some of `ctas`
  int teams;                        // of such a CTA
  int unit_cost, page_cost, item_cost;   // of a CTA, for a unit of the prefix, a page and an item of the requests' own (ns)
  unsigned* err;
};

// Shares are cut as evenly as can be, so that where there are as many for each KV
// head they are the same stretches of each: the heads' interleaved rows of a page
// are then read at about the same time, which DRAM likes (a prefix of 32768
// tokens, 16 rows, 8 KV heads: 46.7 us with uneven cuts, 41.9 us so).
__device__ __forceinline__ int prefix_cut(const PrefixHead& h, int c) {
  if (h.narrow) return (int)((uint32_t)c * (uint32_t)h.total / (uint32_t)max(h.ctas, 1));
  return (int)((long long)c * h.total / max(h.ctas, 1));
}
__device__ __forceinline__ int prefix_cta_of(const PrefixHead& h, int unit) {
  if (h.narrow) return (int)((((uint32_t)unit + 1u) * (uint32_t)h.ctas - 1u) / (uint32_t)max(h.total, 1));
  return (int)((((long long)unit + 1) * h.ctas - 1) / max(h.total, 1));
}

__device__ __forceinline__ PrefixHead load_head(const PrefixHead* at) {
  const int4 v = __ldcg(reinterpret_cast<const int4*>(at));
  return PrefixHead{v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ PrefixGroup load_group(const PrefixGroup* at) {
  const int4 v = __ldcg(reinterpret_cast<const int4*>(at));
  const int4 w = __ldcg(reinterpret_cast<const int4*>(&at->line));
  return PrefixGroup{v.x, v.y, v.z, v.w, w.x, w.y, w.z, 0};
}

// Where the partial results of a row over its group's prefix lie: n of them,
// the first at `o` and `ml`, each next one `step` tiles on.
struct PrefixRow {
  const float* o;
  const float2* ml;
  int n, step;
};

// Row r (verify token r / group, head r % group of KV head kvh) of request b.
__device__ __forceinline__ PrefixRow prefix_row(const PrefixView& v, const PrefixHead& h, const PrefixGroup& g, int R, int group,
                                                int b, int kvh, int r, int d) {
  const PrefixShape& s = v.shape;
  const int token = (b - g.first) * R + r / group, head = r % group;
  const int tile = token / s.tokens * s.chunks + head / s.rows;
  const int row = s.chunks > 1 ? head % s.rows : token % s.tokens * group + head;
  const int k = kvh * g.tiles + tile / s.subs;
  const int u0 = g.line + k * g.units, c0 = prefix_cta_of(h, u0), c1 = prefix_cta_of(h, u0 + g.units - 1);
  const int64_t at = (int64_t)(g.item + k + c0) * s.subs + tile % s.subs;
  return PrefixRow{v.parts + at * s.rows * d + row * 4, v.stats + at * s.rows + row, c1 - c0 + 1, s.subs};
}

// --------------------------------------------------------------- scheduling
// The group of request b, for a CTA of any size: -1 none, and *bad (for all of
// the CTA the same) when the starts decrease or leave [0, B].
__device__ __forceinline__ int find_group(const int32_t* starts, int G, int B, int b, bool* bad) {
  __shared__ int s_found;
  int wrong = 0;
  if (threadIdx.x == 0) s_found = -1;
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    const int s0 = starts[g], s1 = starts[g + 1];
    wrong |= s0 < 0 || s1 < s0 || s1 > B;
    if (s0 <= b && b < s1) s_found = g;        // (one at most, where the starts are right)
  }
  *bad = __syncthreads_or(wrong) != 0;
  return *bad ? -1 : s_found;
}

// The first page of request b's own, -1 when the request cannot be done.
__device__ __forceinline__ int own_first(int blocks, int ctx, int max_blocks, int R) {
  if (ctx < 0 || ctx > max_blocks * kBlock - R) return -1;
  return blocks < 0 || blocks > max_blocks || ctx < blocks * kBlock ? -1 : blocks;
}

// The last of n entries (n >= 1, not decreasing) that is at most x, else 0.
__device__ __forceinline__ int last_at_most(const int32_t* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    (v[mid] <= x ? lo : hi) = mid;
  }
  return lo;
}

__device__ __forceinline__ PrefixHead make_shares(int total, int ctas) {
  const int n = min(ctas, total);
  return PrefixHead{total, n, (long long)total * n < 0x7fffffffll, 0};
}

// The work of one CTA of THREADS threads. It stands between the lengths and
// the attention: each input is read once, in parallel, and searches go through
// copies in shared memory (of up to kCopy groups and requests).
template <int THREADS>
__device__ void prefix_schedule(const PrefixSchedule& w) {
  constexpr int kWarps = THREADS / kWarp, kCopy = 1024;
  __shared__ int2 s_sum[kWarps];
  __shared__ int32_t s_start[kCopy + 1], s_blocks[kCopy], s_line[kCopy], s_pages[kCopy + 1];
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  // Sums of v over the threads before this one, and over all of them.
  auto scan = [&](int2 v, int2* total) {
    int2 incl = v;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) incl.x += x, incl.y += y;
    }
    __syncthreads();                           // the last totals have been read
    if (lane == kWarp - 1) s_sum[warp] = incl;
    __syncthreads();
    incl.x -= v.x, incl.y -= v.y;
    *total = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int2 t = s_sum[i];
      if (i < warp) incl.x += t.x, incl.y += t.y;
      total->x += t.x, total->y += t.y;
    }
    return incl;
  };

  const int ctx0 = tid < w.B ? w.ctx_lens[tid] : 0;   // (on its way while the groups are looked at)
  int wrong = 0;
  for (int g = tid; g < w.G; g += THREADS) {
    const int s0 = w.group_starts[g], s1 = w.group_starts[g + 1], blocks = w.prefix_blocks[g];
    wrong |= s0 < 0 || s1 < s0 || s1 > w.B;
    if (w.G <= kCopy) {
      s_start[g] = s0;
      s_start[g + 1] = s1;                     // (its neighbour writes the same)
      s_blocks[g] = blocks;
    }
  }
  const bool bad = __syncthreads_or(wrong) != 0;
  if (bad && tid == 0) raise_error(w.err, MTP_ERR_LENGTH);
  const int G = bad ? 0 : w.G;                 // every request by itself
  const int32_t *starts = w.G <= kCopy ? s_start : w.group_starts, *blocks_of = w.G <= kCopy ? s_blocks : w.prefix_blocks;

  int2 base = make_int2(0, 0);                 // units of the line, items
  for (int g0 = 0; g0 < G; g0 += THREADS) {
    const int g = g0 + tid;
    PrefixGroup e{0, 0, 0, 0, 0, 0, 0, 0};
    int2 mine = make_int2(0, 0);
    if (g < G) {
      e.first = starts[g];
      const int n = starts[g + 1] - e.first;
      e.blocks = blocks_of[g];
      if (n > 0 && e.blocks > 0 && e.blocks <= w.max_blocks) {
        e.units = (e.blocks + w.shape.pages - 1) / w.shape.pages;
        e.sub_tiles = (n * w.R + w.shape.tokens - 1) / w.shape.tokens * w.shape.chunks;
        e.tiles = (e.sub_tiles + w.shape.subs - 1) / w.shape.subs;
        mine = make_int2(e.tiles * w.Hkv * e.units, e.tiles * w.Hkv);
      } else if (n > 0 && e.blocks != 0) {
        raise_error(w.err, MTP_ERR_LENGTH);
      }
    }
    int2 total;
    const int2 before = scan(mine, &total);
    e.line = base.x + before.x;
    e.item = base.y + before.y;
    base.x += total.x, base.y += total.y;
    if (g < G) {
      w.groups[g] = e;
      if (G <= kCopy) s_line[g] = e.line;
    }
  }

  int own = 0;                                 // own pages of the requests so far
  for (int b0 = 0; b0 < w.B; b0 += THREADS) {
    const int b = b0 + tid;
    int n = 0;
    if (b < w.B) {
      const int ctx = b0 == 0 ? ctx0 : w.ctx_lens[b];
      int g = -1;                              // the last group that begins at or before b, if b is in it
      if (G > 0) {
        const int lo = last_at_most(starts, G, b);
        if (starts[lo] <= b && b < starts[lo + 1]) g = lo;
      }
      const int first = own_first(g < 0 ? 0 : blocks_of[g], ctx, w.max_blocks, w.R);
      w.first[b] = first;
      w.group_of[b] = first > 0 ? g : -1;
      if (first >= 0) n = (ctx + w.R + kBlock - 1) / kBlock - first;
    }
    int2 total;
    const int end = own + scan(make_int2(n, 0), &total).x + n;
    own += total.x;
    if (b < w.B) {
      w.pages[b + 1] = end;
      if (w.B <= kCopy) s_pages[b + 1] = end;
    }
  }
  if (tid == 0) w.pages[0] = s_pages[0] = 0;
  own *= w.own_heads;
  // CTAs for the prefix and for the own pages: so that both should end at once.
  int ctas = w.ctas;
  if (w.own_ctas == 0 && own > 0 && base.x > 0) {
    const float a = (float)base.x * w.unit_cost, z = (float)own * w.page_cost + (float)w.B * w.own_heads * w.item_cost;
    ctas = max(2, min(w.ctas - 2, 2 * (int)(w.ctas * a / (a + z) * 0.5f + 0.5f)));   // (pairs of CTAs do the same)
  }
  // (of one group as many for each KV head, where that leaves few CTAs out)
  int n = min(ctas, base.x);
  if (G == 1 && n % w.Hkv * 10 <= n) n -= n % w.Hkv;
  const PrefixHead h = make_shares(base.x, n);
  if (tid == 0) *w.head = h;
  __syncthreads();                             // (writes to global memory too, for this CTA)
  for (int c = tid; c < h.ctas; c += THREADS) {
    PrefixStart s;
    s.pos = prefix_cut(h, c);
    s.end = prefix_cut(h, c + 1);
    if (G <= kCopy) {
      s.gi = last_at_most(s_line, G, s.pos);   // (the last group whose line begins there or before has items)
    } else {
      int lo = 0, hi = G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (w.groups[mid].line <= s.pos ? lo : hi) = mid;
      }
      s.gi = lo;
    }
    s.group = w.groups[s.gi];
    s.pad = 0;
    w.starts[c] = s;
  }
  const PrefixHead o = make_shares(own, (w.own_ctas > 0 ? w.own_ctas : w.ctas - (h.ctas + 1) / 2 * 2) * w.teams);
  if (tid == 0) *w.own = o;
  const int32_t* pages = w.B <= kCopy ? s_pages : w.pages;
  for (int c = tid; c < o.ctas; c += THREADS) {
    OwnStart s;
    s.pos = prefix_cut(o, c);
    s.end = prefix_cut(o, c + 1);
    s.b = last_at_most(pages, w.B, s.pos / w.own_heads);   // (the last request whose line begins there or before has pages)
    s.before = pages[s.b];
    s.pages = pages[s.b + 1] - s.before;
    s.pad[0] = s.pad[1] = s.pad[2] = 0;
    w.own_starts[c] = s;
  }
}

}  // namespace mtp
