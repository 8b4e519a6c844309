// The prompts' blocks and their order: what the prompt attention works on, laid out by a block of the
// few-row kernel that runs before it.
#pragma once

#include "kv_device.cuh"

namespace moe {

constexpr int kBlockRows = 512;              // of a pair of CTAs
constexpr int kCtaRows = 256;
constexpr int kMaxBlocks = 1 << 16;           // blocks of a call, without the heads
constexpr int kBins = 1024;                   // lengths that the order tells apart

struct PromptPlan {
  int2* list;                  // blocks (request, block), longest first
  int* bins;                   // scratch of the order
  int* count;                  // blocks
  int min_n;                   // requests with more tokens than this
};
constexpr size_t kPlanBytes = 256 + kMaxBlocks * (sizeof(int2) + sizeof(int));
constexpr int kPlanSmem = (kMaxRequests + 1 + kBins + 32) * 4;

inline PromptPlan prompt_plan_at(void* space) {
  uint8_t* p = static_cast<uint8_t*>(space);
  PromptPlan pl;
  pl.count = reinterpret_cast<int*>(p);
  pl.list = reinterpret_cast<int2*>(p + 256);
  pl.bins = reinterpret_cast<int*>(p + 256 + kMaxBlocks * sizeof(int2));
  pl.min_n = 0;
  return pl;
}

// One block's rows and the tokens that they see; tiles [t0, t1) of it for this pair of CTAs.
struct PromptWork {
  int b, h, row0, rows, q0, pos0, lo, hi, t0, t1;
  int part;                    // workspace part, -1: the whole block is here
};

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
  int* first = smem;                          // blocks before request b
  int* hist = first + kMaxRequests + 1;
  int* sums = hist + kBins;
  const int threads = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto blocks_of = [&](int b) {
    const int q0 = a.tok_start[b], n = a.tok_start[b + 1] - q0;
    if (n <= pl.min_n || q0 < 0 || q0 + n > a.T) return 0;
    return (min(n, a.max_q) * G + kBlockRows - 1) / kBlockRows;
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
    pl.bins[x] = bin;
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
      const int bin = x < total ? pl.bins[x] : -1;
      const uint32_t same = __match_any_sync(~0u, bin);
      if (x < total) {
        const int b = owner(x);
        pl.list[hist[bin] + __popc(same & ((1u << lane) - 1))] = make_int2(b, x - first[b]);
      }
      __syncwarp();
      if (x < total && lane == __ffs(same) - 1) hist[bin] += __popc(same);
      __syncwarp();
    }
    if (lane == 0) *pl.count = total;
  }
}
}  // namespace moe
