// Block tables, free stack, slot map and page runs from request lengths.
//
// Everything follows from four prefix sums over the requests: pages released, pages needed, tokens
// added, page runs.  The outputs go to buffers of their own and the inputs are only read, so CTAs
// share nothing: each one scans the (at most 4096) requests again into its shared memory, about 1 us
// from L2, and then writes its share of every output.  One launch, no atomics, no order of arrival.
// The call is bound by latency: launch, one load of the lengths, two block scans, one binary search
// per token or run.  8 requests: 4.8 us back to back as a graph; 1024 requests with 1500-token prompts among
// them, 5.2 MB of tables: 7.6 us, 0.69 TB/s.
#include "kv_internal.h"

namespace moe {

constexpr int kTabThreads = 512;
constexpr int kTabItems = kMaxRequests / kTabThreads;   // requests per thread, at most
constexpr int kTabPerThread = 4;                        // output entries per thread that size the grid
constexpr int kTabCtas = 304;                           // at most
static_assert((long long)kMaxList + kTabCtas * kTabThreads <= 0x7FFFFFFF, "the loops' counters");

struct Scan3 {
  int rel, need, tok;
};

// Exclusive prefix of v over the block; total in *sum.  red: one Scan3 per warp.
__device__ __forceinline__ Scan3 block_scan3(Scan3 v, Scan3* red, Scan3* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Scan3 x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(~0u, x.rel, d), b = __shfl_up_sync(~0u, x.need, d),
              c = __shfl_up_sync(~0u, x.tok, d);
    if (lane >= d) {
      x.rel += a;
      x.need += b;
      x.tok += c;
    }
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  Scan3 base = {0, 0, 0}, all = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    const Scan3 t = red[w];
    if (w < warp) {
      base.rel += t.rel;
      base.need += t.need;
      base.tok += t.tok;
    }
    all.rel += t.rel;
    all.need += t.need;
    all.tok += t.tok;
  }
  __syncthreads();
  *sum = all;
  return Scan3{base.rel + x.rel - v.rel, base.need + x.need - v.need, base.tok + x.tok - v.tok};
}

// Last i in [0, n) with start[i] <= x, for non-decreasing start with start[0] <= x: among equal
// entries the last one, which is the one that owns x.
__device__ __forceinline__ int owner(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) k_kv_tables(const moe_kv_tables_args a) {
  extern __shared__ int sm[];
  const int B = a.B, P = a.page_size, W = a.max_pages;
  int* rel_at = sm;               // [B] pages released before request i
  int* need_at = rel_at + B;      // [B] pages needed before request i
  int* tok_at = need_at + B;      // [B] tokens added before request i
  int* run_at = tok_at + B;       // [B] runs before request i
  int* cur_of = run_at + B;       // [B] clamped current length
  int* kv_of = cur_of + B;        // [B] length after the step; refused requests: -1 - cur
  __shared__ Scan3 red[kTabThreads / 32];

  const int per = (B + kTabThreads - 1) / kTabThreads;   // consecutive requests per thread
  const int i0 = threadIdx.x * per;
  const int shift = __ffs(P) - 1;
  auto pages = [&](int n) { return (n + P - 1) >> shift; };
  int cur[kTabItems], want[kTabItems];
  Scan3 mine = {0, 0, 0};
#pragma unroll
  for (int j = 0; j < kTabItems; ++j) {
    cur[j] = want[j] = 0;
    if (j < per && i0 + j < B) {
      cur[j] = min(max(a.cur_len[i0 + j], 0), W * P);
      want[j] = max(a.new_len[i0 + j], 0);
      if (want[j] <= W * P) {
        const int d = pages(want[j]) - pages(cur[j]);
        mine.rel += max(-d, 0);
        mine.need += max(d, 0);
        mine.tok += max(want[j] - cur[j], 0);
      }
    }
  }
  const int count0 = min(max(*a.free_count, 0), a.num_pages);
  Scan3 all;
  Scan3 at = block_scan3(mine, red, &all);
  const int count1 = count0 + all.rel;
  int refused = 0, granted = 0, runs = 0;
#pragma unroll
  for (int j = 0; j < kTabItems; ++j) {
    const int i = i0 + j;
    if (j < per && i < B) {
      const bool fits = want[j] <= W * P;
      const int d = fits ? pages(want[j]) - pages(cur[j]) : 0;
      const int need = max(d, 0);
      const int add = fits ? max(want[j] - cur[j], 0) : 0;
      const bool ok = fits && (need == 0 || at.need + need <= count1) && (add == 0 || at.tok + add <= a.max_tokens);
      rel_at[i] = at.rel;
      need_at[i] = at.need;
      tok_at[i] = at.tok;
      cur_of[i] = cur[j];
      kv_of[i] = ok ? want[j] : -1 - cur[j];
      run_at[i] = runs;            // within this thread, for now
      at.rel += max(-d, 0);
      at.need += need;
      at.tok += add;
      refused += ok ? 0 : 1;
      granted += ok ? need : 0;
      if (ok && want[j] > cur[j]) runs += ((want[j] - 1) >> shift) - (cur[j] >> shift) + 1;
    }
  }
  Scan3 sums;
  const Scan3 before = block_scan3(Scan3{runs, refused, granted}, red, &sums);
  for (int j = 0; j < per; ++j)
    if (i0 + j < B) run_at[i0 + j] += before.rel;
  __syncthreads();
  const int num_runs = sums.rel, num_granted = sums.tok, total = all.tok;

  // the m-th released page, and entry x of the stack after the releases
  auto released = [&](int m) {
    const int i = owner(rel_at, B, m);
    return a.block_table[(size_t)i * W + pages(kv_of[i]) + m - rel_at[i]];
  };
  auto stack = [&](int x) {
    if (x < 0 || x >= a.num_pages) return -1;
    return x < count0 ? a.free_list[x] : released(x - count0);
  };
  auto entry = [&](int i, int j) {   // block table after the step
    const int kv = kv_of[i] < 0 ? -1 - kv_of[i] : kv_of[i];
    const int held = pages(cur_of[i]);
    if (j >= pages(kv)) return -1;
    if (j < held) return a.block_table[(size_t)i * W + j];
    return stack(count1 - num_granted + need_at[i] + j - held);
  };

  const int tid = blockIdx.x * kTabThreads + threadIdx.x, step = gridDim.x * kTabThreads;
  const int cells = B * W;
  for (int x = tid; x < cells; x += step) {
    const int i = x / W;
    a.out_block_table[x] = entry(i, x - i * W);
  }
  for (int x = tid; x < a.num_pages; x += step)
    a.out_free_list[x] = x >= count0 && x < count1 ? released(x - count0) : a.free_list[x];
  for (int x = tid; x < a.max_tokens; x += step) {
    int slot = -1, pos = 0, req = -1;
    if (x < total) {
      req = owner(tok_at, B, x);
      pos = cur_of[req] + x - tok_at[req];
      if (kv_of[req] >= 0) {
        const int page = entry(req, pos >> shift);
        slot = page < 0 ? -1 : page * P + (pos & (P - 1));
      }
    }
    a.slot[x] = slot;
    a.position[x] = pos;
    a.request[x] = req;
  }
  for (int x = tid; x < a.max_runs; x += step) {
    int tok = 0, len = 0;
    if (x < num_runs) {
      const int i = owner(run_at, B, x);
      const int p0 = ((cur_of[i] >> shift) + x - run_at[i]) << shift;
      const int b = max(p0, cur_of[i]);
      tok = tok_at[i] + b - cur_of[i];
      len = min(p0 + P, kv_of[i]) - b;
    }
    a.run_tok[x] = tok;
    a.run_len[x] = len;
  }
  for (int x = tid; x < B; x += step) {
    a.kv_len[x] = kv_of[x] < 0 ? -1 - kv_of[x] : kv_of[x];
    a.tok_start[x] = tok_at[x];
  }
  if (tid == 0) {
    a.tok_start[B] = total;
    *a.out_free_count = count1 - num_granted;
    a.info[0] = total;
    a.info[1] = num_runs;
    a.info[2] = sums.need;
    a.info[3] = num_granted;
  }
}

cudaError_t launch_kv_tables(const moe_kv_tables_args& a, cudaStream_t s) {
  const size_t smem = (size_t)6 * a.B * sizeof(int);
  static_assert(6 * kMaxRequests * 4 <= 100 * 1024, "two CTAs fit an SM");
  if (smem > 48 * 1024) {
    const cudaError_t err =
        cudaFuncSetAttribute(k_kv_tables, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
  }
  const long long out = (long long)a.B * a.max_pages + a.num_pages + a.max_tokens + a.max_runs;
  const long long want = (out + kTabThreads * kTabPerThread - 1) / (kTabThreads * kTabPerThread);
  const int grid = (int)(want < 1 ? 1 : want > kTabCtas ? kTabCtas : want);
  k_kv_tables<<<grid, kTabThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
