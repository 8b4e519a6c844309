// The prompts' blocks and their order: what the prompt attention works on, laid out by a block of the
// few-row kernel that runs before it.
//
// An item is a block and one of its key/value heads.  The items, longest first, go to the pairs of CTAs in
// rounds, forward and back.  What the last, incomplete round holds is poured over the pairs up to a common
// level: an item weighs kItemStart, what its start and end cost, and one unit per tile of 128 cached tokens
// that its rows see; in a line of these units each pair has a stretch as long as it is below the level.
// An item that lies on several stretches is cut along the cache.  Where even the longest of the round is
// short, a cut costs more than it saves (1000 tokens of 32 / 8 heads, 8 tiles at most: 36 us instead of 27),
// and every pair takes one.
#pragma once

#include <algorithm>
#include <climits>

#include "kv_device.cuh"

namespace moe {

constexpr int kBlockRows = 512;              // of a pair of CTAs
constexpr int kCtaRows = 256;
constexpr int kMaxBlocks = 1 << 16;           // blocks of a call, without the heads
constexpr int kBins = 1024;                   // lengths that the order tells apart

constexpr int kPromptCtas = 152;              // at most (SMs)
constexpr int kPromptPairs = kPromptCtas / 2;
constexpr int kItemStart = 3;                 // units
constexpr int kCutTiles = 12;                 // of the longest item of the last round, at least, for cuts

// The last round: item i has units from start[i] on, pair c those from bound[c] on.
struct PromptTail {
  int rounds, rest, pour;                     // full rounds, items after them, whether they are poured
  int start[kPromptPairs + 1], bound[kPromptPairs + 1];
};
struct PromptPlan {
  PromptTail* tail;
  int4* list;                  // blocks (request, block, tiles), longest first
  int2* bins;                  // scratch of the order: place of its length, tiles
  int min_n;                   // requests with more tokens than this
  int pairs;
};
constexpr size_t kPlanList = (sizeof(PromptTail) + 255) & ~(size_t)255;
constexpr size_t kPlanBytes = kPlanList + kMaxBlocks * (sizeof(int4) + sizeof(int2));
constexpr int kPlanSmem = (2 * kPromptPairs + kMaxRequests + 1 + kBins + 32) * 4;

inline PromptPlan prompt_plan_at(void* space) {
  uint8_t* p = static_cast<uint8_t*>(space);
  PromptPlan pl;
  pl.tail = reinterpret_cast<PromptTail*>(p);
  pl.list = reinterpret_cast<int4*>(p + kPlanList);
  pl.bins = reinterpret_cast<int2*>(p + kPlanList + kMaxBlocks * sizeof(int4));
  pl.min_n = 0;
  pl.pairs = std::min(kPromptCtas, sm_count()) / 2;
  return pl;
}

// One block's rows and the tokens that they see; tiles [t0, t1) of it for this pair of CTAs.
struct PromptWork {
  int b, h, row0, rows, q0, pos0, lo, hi, t0, t1;
  int part;                    // workspace part, -1: the whole block is here
};

// The k-th item of pair c in rounds forward and back.
__device__ __forceinline__ long long round_item(int k, int c, int pairs) {
  return (long long)k * pairs + ((k & 1) ? pairs - 1 - c : c);
}

// Tiles of an item of n that lie before a cut x units behind its first tile.
__device__ __forceinline__ int prompt_cut(int x, int n) { return min(max(x, 0), n); }

// Block blk of request b, with all the tiles that its rows see.
__device__ __forceinline__ void prompt_block(const moe_kv_attention_args& a, int G, int page_shift, int b, int blk,
                                             PromptWork& w) {
  w.b = b;
  w.q0 = a.tok_start[b];
  const int n = min(a.tok_start[b + 1] - w.q0, a.max_q);
  const int L = min(max(a.kv_len[b], 0), a.max_pages << page_shift);
  w.pos0 = L - (a.tok_start[b + 1] - w.q0);
  w.row0 = blk * kBlockRows;
  w.rows = n * G;
  const int i0 = w.row0 / G, i1 = (min(w.rows, w.row0 + kBlockRows) - 1) / G;
  w.hi = max(0, min(L, w.pos0 + i1 + 1));
  w.lo = a.window > 0 ? max(0, w.pos0 + i0 - a.window + 1) : 0;
  w.t0 = min(w.lo, max(w.hi - 1, 0)) / kTile;
  w.t1 = max(w.t0 + 1, (w.hi + kTile - 1) / kTile);
}

// Blocks of all requests with more than min_n tokens, longest first; equal lengths keep the order of
// requests and rows, so the order never depends on timing.  One block of threads, kPlanSmem bytes.
__device__ __forceinline__ void prompt_plan(const moe_kv_attention_args& a, const PromptPlan& pl, int G, int page_shift,
                                            int* smem) {
  long long* load = reinterpret_cast<long long*>(smem);   // [pairs] units of the full rounds
  int* first = smem + 2 * kPromptPairs;       // blocks before request b
  int* hist = first + kMaxRequests + 1;
  int* sums = hist + kBins;
  const int threads = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto blocks_of = [&](int b) {
    const int q0 = a.tok_start[b], q1 = a.tok_start[b + 1];
    if (q0 < 0 || q1 <= q0 || q1 > a.T || q1 - q0 <= pl.min_n) return 0;
    return (min(q1 - q0, a.max_q) * G + kBlockRows - 1) / kBlockRows;
  };
  auto scan = [&](int v) {                    // inclusive sum over the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(~0u, v, d);
      if (lane >= d) v += t;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += sums[w];
    __syncthreads();
    return base + v;
  };
  const int per = (a.B + threads - 1) / threads;
  int mine = 0;
  for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) mine += blocks_of(b);
  int at = scan(mine) - mine;
  for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
    first[b] = at;
    at += blocks_of(b);
    if (b == a.B - 1) first[a.B] = at;
  }
  for (int i = tid; i < kBins; i += threads) hist[i] = 0;
  __syncthreads();
  const int total = min(first[a.B], kMaxBlocks);
  int shift = 0;                              // tiles per bin
  while (((a.max_pages << page_shift) / kTile + 1) >> shift >= kBins) ++shift;
  auto owner = [&](int x) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  for (int x = tid; x < total; x += threads) {
    const int b = owner(x);
    PromptWork w;
    prompt_block(a, G, page_shift, b, x - first[b], w);
    const int bin = kBins - 1 - min((w.t1 - w.t0) >> shift, kBins - 1);
    pl.bins[x] = make_int2(bin, w.t1 - w.t0);
    atomicAdd(&hist[bin], 1);
  }
  __syncthreads();
  // the bins' first places: an exclusive sum, consecutive bins per thread
  const int nb = (kBins + threads - 1) / threads, b0 = min(kBins, tid * nb), b1 = min(kBins, b0 + nb);
  int sum = 0;
  for (int i = b0; i < b1; ++i) sum += hist[i];
  int start = scan(sum) - sum;
  for (int i = b0; i < b1; ++i) {
    const int n = hist[i];
    hist[i] = start;
    start += n;
  }
  __syncthreads();
  if (warp == 0) {
    for (int x0 = 0; x0 < total; x0 += 32) {
      const int x = x0 + lane;
      const int2 bt = x < total ? pl.bins[x] : make_int2(-1, 0);
      const int bin = bt.x;
      const uint32_t same = __match_any_sync(~0u, bin);
      if (x < total) {
        const int b = owner(x);
        pl.list[hist[bin] + __popc(same & ((1u << lane) - 1))] = make_int4(b, x - first[b], bt.y, 0);
      }
      __syncwarp();
      if (x < total && lane == __ffs(same) - 1) hist[bin] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // ------------------------------------------------------------------------ the last round
  const int pairs = pl.pairs;
  const long long items = (long long)total * a.Hkv;
  const int rounds = (int)(items / pairs), rest = (int)(items - (long long)rounds * pairs);
  auto tiles_of = [&](long long item) { return pl.list[item / a.Hkv].z; };
  const long long own = (long long)rounds * pairs + tid;
  const int tiles = tid < rest ? tiles_of(own) : 0;
  const int weight = tid < rest ? tiles + kItemStart : 0;
  const bool pour = rest > 0 && tiles_of((long long)rounds * pairs) >= kCutTiles;
  if (tid == 0) {
    pl.tail->rounds = rounds;
    pl.tail->rest = rest;
    pl.tail->pour = pour;
  }
  if (!pour) return;
  if (tid < pairs) {
    long long sum_of = 0;
#pragma unroll 4
    for (int k = 0; k < rounds; ++k) sum_of += tiles_of(round_item(k, tid, pairs)) + kItemStart;
    load[tid] = sum_of;
  }
  const int begin = scan(weight) - weight;
  if (tid < rest) pl.tail->start[tid] = begin;
  if (tid == rest - 1) first[0] = begin + weight;
  __syncthreads();
  const int units = first[0];
  if (warp == 0) {
    // the level that the poured units reach: pairs above it get none
    constexpr int kPer = (kPromptPairs + 31) / 32;
    long long mine_of[kPer], level = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine_of[i] = lane + 32 * i < pairs ? load[lane + 32 * i] : LLONG_MAX;
    long long below = LLONG_MAX - 1;          // pairs whose load is at most this get some
    for (int turn = 0; turn < kPromptPairs; ++turn) {
      long long all = 0;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (mine_of[i] <= below) {
          all += mine_of[i];
          ++n;
        }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        all += __shfl_xor_sync(~0u, all, d);
        n += __shfl_xor_sync(~0u, n, d);
      }
      level = (all + units + n - 1) / n;
      bool out = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) out |= mine_of[i] <= below && mine_of[i] > level;
      if (!__any_sync(~0u, out)) break;
      below = level;
    }
    int base = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int room = mine_of[i] <= below ? (int)min(max(level - mine_of[i], 0ll), (long long)units) : 0;
      int upto = room;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += t;
      }
      const int at_c = min(units, base + upto - room);
      if (lane + 32 * i < pairs) pl.tail->bound[lane + 32 * i] = at_c;
      base = min(units, base + __shfl_sync(~0u, upto, 31));
    }
    if (lane == 0) pl.tail->bound[pairs] = units;
  }
}

// What pair c works on, piece by piece.  One warp, all lanes alike.
struct PromptWalk {
  int rounds, rest, pour, k, i, u0, u1;

  __device__ __forceinline__ void start(const PromptPlan& pl, int c, int lane) {
    rounds = pl.tail->rounds;
    rest = pl.tail->rest;
    pour = pl.tail->pour;
    k = i = u0 = u1 = 0;
    if (!pour) return;
    u0 = pl.tail->bound[c];
    u1 = pl.tail->bound[c + 1];
    // the last item that starts at or before u0
    int n = 0;
    for (int j = lane; j < kPromptPairs; j += 32) n += j < rest && pl.tail->start[j] <= u0;
    i = max(0, (int)__reduce_add_sync(~0u, (unsigned)n) - 1);
  }

  __device__ __forceinline__ bool next(const moe_kv_attention_args& a, const PromptPlan& pl, int G, int page_shift,
                                       int c, PromptWork& w) {
    auto look = [&](long long item) {
      const int4 e = pl.list[item / a.Hkv];
      prompt_block(a, G, page_shift, e.x, e.y, w);
      w.h = (int)(item % a.Hkv);
      w.part = -1;
    };
    if (k < rounds) {
      look(round_item(k++, c, pl.pairs));
      return true;
    }
    if (!pour) {
      const long long item = round_item(k, c, pl.pairs);
      if (k++ > rounds || item >= (long long)rounds * pl.pairs + rest) return false;
      look(item);
      return true;
    }
    for (; i < rest; ++i) {
      const int at = pl.tail->start[i] + kItemStart;
      if (at > u1) return false;
      look((long long)rounds * pl.pairs + i);
      const int t0 = w.t0, n = w.t1 - w.t0, ta = prompt_cut(u0 - at, n), tb = prompt_cut(u1 - at, n);
      if (tb <= ta) continue;
      w.t0 = t0 + ta;
      w.t1 = t0 + tb;
      // a pair's first piece may be a later part of its item, the last one a first part
      w.part = ta > 0 ? 2 * c : tb < n ? 2 * c + 1 : -1;
      ++i;
      return true;
    }
    return false;
  }
};
}  // namespace moe
