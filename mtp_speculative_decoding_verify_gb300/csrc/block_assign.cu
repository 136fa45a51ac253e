// kv_block_assign: blocks for the tokens that requests are about to append,
// from the free list into the block tables, and the cache slot of each token.
// The other direction of kv_rollback and kv_window_release.
//
// need_b = number of entries < 0 among blocks ceil(L/64) .. (L+n-1)/64 of
// request b; with c_b the sum of need up to and with b, b is served iff need_b
// = 0 or c_b <= free_count, and its k-th missing entry becomes
// free_list[free_count - 1 - (c_b - need_b) - k]. The sum is monotone, so
// what is taken has no gaps.
//
// A step's call (a few tokens a request) is one CTA, a thread a request: a
// chain of five dependent reads bounds it (256 requests: 3.5 us). Longer appends
// go by pieces of 32 blocks, one entry a lane: the first launch counts each
// piece's missing entries, the second sums the counts before its own (they are
// few, and in L2), takes its blocks and writes the slots, 8 bytes a token (64
// requests of 500-1500 tokens: 5.8 us, 32 of 5000-65000: 8.5). Where there are
// many pieces, so that each piece's sum would take as long as the rest, the first
// launch also counts by groups of pieces, and a sum is of those and of a part of
// one group. A CTA then counts 256 pieces, not 8, which costs more until there are
// some 14000 (us one by one and by groups: 2056 pieces 12, 32; 8200 39, 52; 16420 89,
// 75; 32840 244, 124; 131200 2970, 474).
#include <algorithm>

#include "attention_window.h"
#include "common.cuh"
#include "kernels.h"

namespace mtp {
int device_context(unsigned** err, int* sm_count);
int set_error(int code, const char* msg);
int set_cuda_error(cudaError_t e, const char* what);
void set_launch_count(int n);

namespace {

constexpr int kPieceBlocks = kWarp, kPieceTokens = kPieceBlocks * kBlock;
constexpr int kStepThreads = 1024, kPieceThreads = 256;
constexpr int kGroup = kPieceThreads;    // pieces of a group
constexpr int kManyPieces = 16384;       // from which on there are groups

struct AssignParams {
  int32_t* table;
  const int32_t *seq_lens, *starts, *free_list;
  int32_t* free_count;
  int64_t* slots;
  int32_t* taken;
  int32_t* counts;             // [1 + pieces]: the free list's length, missing entries of each piece
  int32_t* sums;               // [groups]: missing entries of the pieces of each group, if they are counted
  int B, T, max_blocks, capacity, pieces;
  unsigned* err;
};

// Request b: its tokens s0 .. s0 + n - 1 of the batch at positions L and up.
struct Req {
  int s0, n, L;
  unsigned error;              // 0: it can be served
};

// (of starts that starts_ok has passed)
__device__ __forceinline__ Req load_request(const AssignParams& p, int b) {
  Req r;
  r.s0 = p.starts[b];
  r.n = p.starts[b + 1] - r.s0;
  r.L = p.seq_lens[b];
  r.error = 0;
  if (r.L < 0 || (long long)r.L + r.n > (long long)p.max_blocks * kBlock) {
    r.error = MTP_ERR_LENGTH;
    r.L = 0;                   // (its slots are written all the same, as -1)
  } else if (r.n > 0 && r.L % kBlock != 0 && p.table[(int64_t)b * p.max_blocks + r.L / kBlock] < 0) {
    r.error = MTP_ERR_BLOCK_ID;   // the block that holds its last tokens (no call writes that entry)
  }
  return r;
}

// No start decreases or leaves [0, T]. The whole CTA.
__device__ __forceinline__ bool starts_ok(const AssignParams& p) {
  int bad = 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int s0 = p.starts[b], s1 = p.starts[b + 1];
    bad |= s0 < 0 || s1 < s0 || s1 > p.T;
  }
  return __syncthreads_or(bad) == 0;
}

__device__ __forceinline__ int64_t slot_of(int id, int pos) { return id < 0 ? -1 : (int64_t)id * kBlock + pos % kBlock; }

__device__ __forceinline__ int free_blocks(const AssignParams& p, int count) {   // a bad count holds nothing
  return count >= 0 && count <= p.capacity ? count : 0;
}

// -------------------------------------------------------------------- a step
// A lane walks its own request's entries and slots when they are a step's; a
// longer one among them (a prompt's chunk) is the whole warp's.
constexpr int kStepTokens = kMaxRows, kStepBlocks = kMaxRows / kBlock + 1;

__global__ void __launch_bounds__(kStepThreads) assign_step_kernel(const AssignParams p) {
  __shared__ int s_warp[kStepThreads / kWarp];
  __shared__ int s_used;       // blocks taken
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  const int listed = *p.free_count, free0 = free_blocks(p, listed);
  if (tid == 0) {
    s_used = 0;
    if (free0 != listed) raise_error(p.err, MTP_ERR_FREE_LIST);
  }
  if (!starts_ok(p)) {
    if (tid == 0) raise_error(p.err, MTP_ERR_LENGTH);
    for (int b = tid; b < p.B; b += kStepThreads) p.taken[b] = -1;
    return;
  }
  long long base = 0;          // what the requests of the chunks before need
  for (int b0 = 0; b0 < p.B; b0 += kStepThreads) {
    const int b = b0 + tid;
    Req r{0, 0, 0, 0};
    int i0 = 0, i1 = 0, need = 0;              // entries i0 .. i1 - 1 may be missing
    int32_t* row = p.table + (int64_t)b * p.max_blocks;
    if (b < p.B) {
      r = load_request(p, b);
      if (r.error) raise_error(p.err, r.error);
      else if (r.n > 0) {
        i0 = (r.L + kBlock - 1) / kBlock;
        i1 = (r.L + r.n - 1) / kBlock + 1;
      }
    }
    const bool long_row = i1 - i0 > kStepBlocks;
    if (!long_row)
      for (int i = i0; i < i1; ++i) need += row[i] < 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, long_row); todo != 0; todo &= todo - 1) {
      const int who = __ffs(todo) - 1, j0 = __shfl_sync(0xffffffffu, i0, who), j1 = __shfl_sync(0xffffffffu, i1, who);
      const int32_t* r2 = p.table + (int64_t)(b - lane + who) * p.max_blocks;
      int c = 0;
      for (int i = j0 + lane; i < j1; i += kWarp) c += r2[i] < 0;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == who) need = c;
    }
    int incl = need;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();           // the last chunk's totals have been read
    if (lane == kWarp - 1) s_warp[warp] = incl;
    __syncthreads();
    const int mine = s_warp[lane];             // one total a lane: 32 warps
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
    const int total = __reduce_add_sync(0xffffffffu, mine);
    const long long end = base + before + incl;
    base += total;
    const bool served = b < p.B && r.error == 0 && (need == 0 || end <= free0);
    if (b < p.B) p.taken[b] = served ? need : -1;
    const int at = served ? free0 - 1 - (int)(end - need) : 0;   // place of its first block in the list
    if (served && need > 0) atomicMax(&s_used, (int)end);
    auto take = [&](int32_t* entry, int place) {
      const int id = p.free_list[place];
      if (id < 0) raise_error(p.err, MTP_ERR_BLOCK_ID);
      *entry = id;
    };
    if (served && need > 0 && !long_row) {
      int place = at;
      for (int i = i0; i < i1; ++i)
        if (row[i] < 0) take(row + i, place--);
    }
    const bool long_slots = r.n > kStepTokens;
    if (!long_slots) {
      int id = -1, block = -1;                 // the block whose id is held
      for (int x = 0; x < r.n; ++x) {
        const int pos = r.L + x;
        if (served && pos / kBlock != block) {
          block = pos / kBlock;
          id = row[block];
        }
        p.slots[r.s0 + x] = slot_of(id, pos);
      }
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, long_slots); todo != 0; todo &= todo - 1) {
      const int who = __ffs(todo) - 1;
      const int j0 = __shfl_sync(0xffffffffu, i0, who), j1 = __shfl_sync(0xffffffffu, i1, who);
      const int ok = __shfl_sync(0xffffffffu, served, who), some = __shfl_sync(0xffffffffu, need, who);
      const int L = __shfl_sync(0xffffffffu, r.L, who), n = __shfl_sync(0xffffffffu, r.n, who);
      const int s0 = __shfl_sync(0xffffffffu, r.s0, who);
      int place = __shfl_sync(0xffffffffu, at, who);
      int32_t* r2 = p.table + (int64_t)(b - lane + who) * p.max_blocks;
      if (ok && some > 0 && j1 - j0 > kStepBlocks) {
        for (int i = j0; i < j1; i += kWarp) {
          const bool miss = i + lane < j1 && r2[i + lane] < 0;
          const unsigned m = __ballot_sync(0xffffffffu, miss);
          if (miss) take(r2 + i + lane, place - __popc(m & ((1u << lane) - 1u)));
          place -= __popc(m);
        }
      }
      __syncwarp();            // the entries are there for all lanes
      for (int x = lane; x < n; x += kWarp) p.slots[s0 + x] = slot_of(ok ? r2[(L + x) / kBlock] : -1, L + x);
    }
  }
  __syncthreads();
  if (tid == 0 && s_used > 0) *p.free_count = free0 - s_used;
}

// -------------------------------------------------------------------- pieces
// Request b's blocks L/64 .. in pieces of 32. A request of n tokens has at
// most n / 2048 + 2 of them, so numbering them from starts[b] / 2048 + 2 b
// on leaves no two requests the same number, and b is the last request whose
// number is at most `piece`.
__device__ __forceinline__ int piece_request(const AssignParams& p, int piece, int* first) {
  const int lane = threadIdx.x % kWarp;
  int lo = 0, hi = p.B;        // the answer is in [lo, hi)
  while (hi - lo > 1) {        // 32-ary search: every warp does it by itself
    const int step = (hi - lo + kWarp - 1) / kWarp;
    const int b = lo + lane * step;
    const bool le = b < hi && p.starts[b] / kPieceTokens + 2 * b <= piece;
    const unsigned m = __ballot_sync(0xffffffffu, le || lane == 0);
    const int last = 31 - __clz(m);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  *first = p.starts[lo] / kPieceTokens + 2 * lo;
  return lo;
}

// Entry of lane `lane` in a piece: its block index, or -1 outside the request.
__device__ __forceinline__ int piece_block(const Req& r, int k, int lane) {
  const int i = r.L / kBlock + k * kPieceBlocks + lane;
  return k >= 0 && r.n > 0 && i <= (r.L + r.n - 1) / kBlock ? i : -1;
}

// GROUPS: a CTA counts a group of kGroup pieces; else a piece a warp.
template <bool GROUPS>
__global__ void __launch_bounds__(kPieceThreads) assign_count_kernel(const AssignParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_sum;
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, warps = kPieceThreads / kWarp;
  const int b_taken = blockIdx.x * kPieceThreads + threadIdx.x;   // (as many CTAs have B threads: a request has two pieces)
  if (GROUPS && threadIdx.x == 0) s_sum = 0;   // (starts_ok is a barrier)
  const bool ok = starts_ok(p);
  if (blockIdx.x == 0 && threadIdx.x == 0) {   // the second launch lowers it while others still need it
    const int listed = *p.free_count, free0 = free_blocks(p, listed);
    p.counts[0] = ok ? free0 : -1;
    if (free0 != listed) raise_error(p.err, MTP_ERR_FREE_LIST);
    if (!ok) raise_error(p.err, MTP_ERR_LENGTH);
  }
  if (b_taken < p.B) {         // until its first piece knows better
    Req r{0, 1, 0, 0};
    if (ok) r = load_request(p, b_taken);
    if (r.error) raise_error(p.err, r.error);
    p.taken[b_taken] = r.error || r.n > 0 ? -1 : 0;
  }
  if (!ok) return;
  int sum = 0;
  for (int x = warp; x < (GROUPS ? kGroup : warps); x += warps) {
    const int piece = blockIdx.x * (GROUPS ? kGroup : warps) + x;
    if (piece >= p.pieces) break;
    int first;
    const int b = piece_request(p, piece, &first);
    const Req r = load_request(p, b);
    const int i = piece_block(r, piece - first, lane);
    const bool miss = r.error == 0 && i * (int64_t)kBlock >= r.L && i >= 0 && p.table[(int64_t)b * p.max_blocks + i] < 0;
    const int c = __popc(__ballot_sync(0xffffffffu, miss));
    if (lane == 0) p.counts[1 + piece] = c;
    sum += c;
  }
  if constexpr (GROUPS) {
    if (lane == 0 && sum != 0) atomicAdd(&s_sum, sum);
    __syncthreads();
    if (threadIdx.x == 0) p.sums[blockIdx.x] = s_sum;
  }
}

template <bool GROUPS>
__global__ void __launch_bounds__(kPieceThreads) assign_pieces_kernel(const AssignParams p) {
  __shared__ int s_id[kPieceBlocks];
  __shared__ long long s_sum[2][kPieceThreads / kWarp];
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp, piece = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int free0 = __ldcg(p.counts);
  if (free0 < 0) return;       // bad starts
  int first;
  const int b = piece_request(p, piece, &first);
  const Req r = load_request(p, b);
  const int k = piece - first, i0 = piece_block(r, k, 0);
  if (i0 < 0) return;
  const int last = (r.L + r.n - 1) / kBlock, n_pieces = (last - r.L / kBlock) / kPieceBlocks + 1;
  // What the pieces before this one need, and those up to the request's last.
  const int stop = first + n_pieces;
  long long before = 0, end = 0;
  int own = 0;                 // of this request
  if constexpr (GROUPS) {      // the groups before piece's and before the last, then the pieces of these two
    for (int g = tid; g < stop / kGroup; g += kPieceThreads) {
      const int c = __ldcg(p.sums + g);
      end += c;
      if (g < piece / kGroup) before += c;
    }
    for (int x = piece / kGroup * kGroup + tid; x < piece; x += kPieceThreads) before += __ldcg(p.counts + 1 + x);
    for (int x = stop / kGroup * kGroup + tid; x < stop; x += kPieceThreads) end += __ldcg(p.counts + 1 + x);
    for (int x = first + tid; x < stop; x += kPieceThreads) own += __ldcg(p.counts + 1 + x);
  } else {
    for (int x = tid; x < stop; x += kPieceThreads) {
      const int c = __ldcg(p.counts + 1 + x);
      end += c;
      if (x < piece) before += c;
      if (x >= first) own += c;
    }
  }
  own = __syncthreads_or(own);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    end += __shfl_xor_sync(0xffffffffu, end, o);
  }
  if (lane == 0) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = end;
  }
  __syncthreads();
  before = end = 0;
#pragma unroll
  for (int w = 0; w < kPieceThreads / kWarp; ++w) {
    before += s_sum[0][w];
    end += s_sum[1][w];
  }
  const bool served = r.error == 0 && (own == 0 || end <= free0);
  if (warp == 0) {
    const int i = piece_block(r, k, lane);
    int id = -1;
    if (served && i >= 0) id = p.table[(int64_t)b * p.max_blocks + i];
    const bool miss = served && i >= 0 && id < 0 && i * (int64_t)kBlock >= r.L;
    const unsigned m = __ballot_sync(0xffffffffu, miss);
    if (miss) {
      id = p.free_list[free0 - 1 - (int)before - __popc(m & ((1u << lane) - 1u))];
      if (id < 0) raise_error(p.err, MTP_ERR_BLOCK_ID);
      p.table[(int64_t)b * p.max_blocks + i] = id;
    }
    s_id[lane] = id;
  }
  if (tid == 0 && k == 0 && served) {
    long long of_request = 0;
    for (int x = first; x < stop; ++x) of_request += __ldcg(p.counts + 1 + x);
    p.taken[b] = (int)of_request;
    if (own != 0) atomicMin(p.free_count, free0 - (int)end);
  }
  __syncthreads();
  // Positions count from the piece's first: a refused request may have up to 2^31 - 1 tokens, and the piece's end is then
  // beyond 31 bits.
  const int at = i0 * kBlock, x0 = max(r.L - at, 0), x1 = min(r.L + r.n - at, kPieceTokens);
  for (int x = x0 + tid; x < x1; x += kPieceThreads) p.slots[r.s0 + (at - r.L) + x] = slot_of(s_id[x / kBlock], x);
}

int pieces_of(int B, int T) { return T / kPieceTokens + 2 * B; }

template <bool GROUPS>
cudaError_t launch_pieces(const AssignParams& p, cudaStream_t s) {
  const int of_cta = GROUPS ? kGroup : kPieceThreads / kWarp;
  assign_count_kernel<GROUPS><<<(p.pieces + of_cta - 1) / of_cta, kPieceThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_behind_append(assign_pieces_kernel<GROUPS>, p.pieces, kPieceThreads, 0, s, p);
}

int fail(const char* msg) { return set_error(MTP_INVALID_ARG, msg); }

int check_assign(const mtp_block_assign_args* a) {
  if (!a) return fail("kv_block_assign: args is NULL");
  if (a->B < 0 || a->T < 0) return fail("kv_block_assign: B and T must be >= 0");
  if (a->block_size != MTP_BLOCK_SIZE) return fail("kv_block_assign: block_size must be 64");
  if (a->max_blocks <= 0 || a->max_blocks > (1 << 24) || a->free_capacity < 0)
    return fail("kv_block_assign: max_blocks outside [1, 2^24], or free_capacity < 0");
  if (a->B > (1 << 20)) return set_error(MTP_UNSUPPORTED, "kv_block_assign: B > 2^20");
  if (a->B == 0) return MTP_OK;
  if (!a->block_table || !a->seq_lens || !a->starts || !a->free_count || !a->taken || (a->T > 0 && !a->slot_map) ||
      (a->free_capacity > 0 && !a->free_list))
    return fail("kv_block_assign: a required pointer is NULL");
  if (!a->workspace || a->workspace_bytes < mtp_block_assign_workspace_size(a->B, a->T))
    return fail("kv_block_assign: workspace too small (mtp_block_assign_workspace_size)");
  if ((uintptr_t)a->workspace % 256) return fail("workspace must be 256-byte aligned");
  return MTP_OK;
}

}  // namespace
}  // namespace mtp

extern "C" {

size_t mtp_block_assign_workspace_size(int32_t B, int32_t T) {
  if (B < 0 || T < 0 || B > (1 << 20)) return 0;
  const size_t pieces = mtp::pieces_of(B, T);
  return ((1 + pieces + pieces / mtp::kGroup + 1) * sizeof(int32_t) + 255) / 256 * 256;
}

int kv_block_assign(const mtp_block_assign_args* a, void* stream) {
  int rc = mtp::check_assign(a);
  if (rc != MTP_OK) return rc;
  mtp::set_launch_count(0);
  if (a->B == 0) return MTP_OK;
  unsigned* err = nullptr;
  int sm_count = 0;
  if ((rc = mtp::device_context(&err, &sm_count)) != MTP_OK) return rc;
  mtp::AssignParams p;
  p.table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.starts = a->starts;
  p.free_list = a->free_list;
  p.free_count = a->free_count;
  p.slots = a->slot_map;
  p.taken = a->taken;
  p.counts = static_cast<int32_t*>(a->workspace);
  p.B = a->B;
  p.T = a->T;
  p.max_blocks = a->max_blocks;
  p.capacity = a->free_capacity;
  p.pieces = mtp::pieces_of(a->B, a->T);
  p.sums = p.counts + 1 + p.pieces;
  p.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  // (us in one CTA and by pieces: 256 requests of 16 tokens 5.4, 6.4, of 48 10.9, 6.5; 1024 of 16 12.2, 11.5; 4096 of 16
  // 44.5, 38.5, of 4 16.5, 38.8; 16384 of 4 61, 122. Up to 65536 tokens, since one long request may be among them, and a
  // warp walks it alone, which the rule does not see: 256 requests, 255 of one token and one of 3841, 11.1, 6.2; 1024, one
  // of 15361, 36, 12; 8192, one of 8000, 38, 74, one of 30000 83, 74, one of 57000 143, 74.)
  if ((a->T <= 16 * (long long)a->B && a->T <= 16384) || (a->T <= 8 * (long long)a->B && a->T <= 65536)) {
    mtp::assign_step_kernel<<<1, mtp::kStepThreads, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return mtp::set_cuda_error(e, "block assign launch");
    mtp::set_launch_count(1);
    return MTP_OK;
  }
  e = p.pieces > mtp::kManyPieces ? mtp::launch_pieces<true>(p, s) : mtp::launch_pieces<false>(p, s);
  if (e != cudaSuccess) return mtp::set_cuda_error(e, "block assign launch");
  mtp::set_launch_count(2);
  return MTP_OK;
}

}  // extern "C"
