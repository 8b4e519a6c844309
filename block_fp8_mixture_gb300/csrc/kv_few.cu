// Attention over the 8-bit paged cache for few query rows per request: decode and verification.
//
// Every live byte of the cache is read once and costs a handful of operations, so HBM is the bound
// (256 bytes per token and head at D = 128).  The tokens sit on the MMA's M side and the query rows
// (tokens of the request x heads that share the key/value head, padded to 8, 16, 32 or 64) on its N
// side, so that one pass over a 128-token tile serves all rows, and the E4M3 codes go from the cache
// to the tensor cores as they are:
//   S^T[token][row] = K[token][:] . Q[row][:]          A = K tile, K-major
//   O^T[d][row]     = sum_token V[token][d] P[row][token]   A = V tile, MN-major
// What is not 8-bit is split into E4M3 terms on the N side, each with its own column, which keeps the
// accumulation in fp32 and costs no second read of A: a row of Q, scaled by a power of two, into
// two terms (the second x 32: 8 bits, absolute error 2^-15 of the largest value), a row of P, rounded to
// FP16 first, into three (x 1, x 32, x 1024: 11 bits down to 2^-13 of the running maximum, 8 at 2^-17, 4 at
// 2^-21, nothing below 2^-25).
// The page's K scale multiplies the score.  Its V scale goes into the exponent: with f = K scale x softmax
// scale and lv = log2 V scale, p' = 2^(s f + lv - M), where M is the row's running maximum of s f + lv.  Then
// O = sum p' code needs no scale, the row sum is sum p' / V scale, and the terms keep their bits however far
// apart the scales of a tile's pages are.  (p' relative to the tile's largest V scale loses a bit of P for every
// bit of the ratio past 2^14, and a row whose weight lies on the page with the small scale its result.)
//
// The work is dealt out evenly, whatever the lengths: an item (request, head) weighs kItemUnits, what
// its start and end cost, and one unit per 128-token tile; CTA c takes the tiles that lie in the c-th of
// equal shares of the flattened list.  A CTA that holds part of an item leaves its sums, maximum and
// unscaled output in the workspace; the CTA that arrives last adds the parts, in CTA order, so results do
// not depend on timing.  Where an item has many parts the last of every kJoinGroup CTAs adds theirs first
// (128k tokens on one head: 102 us in one step, 20 us in two).
//   warp 0      producer: lane i fetches page i of the tile (TMA), its scales and the tile's bounds
//   warp 1      MMA issuer
//   warps 2..   one warpgroup per 8 or 16 rows: thread = token for the scores, = d for the output
// The maximum that scores are taken relative to moves only when one passes it by 8 x (2^3): then
// all threads of the warpgroup reduce the tile's maximum and rescale, else a vote is all it costs.
//
// 128 requests of 8k to 16k tokens, 64 / 8 heads of 128: 445 to 452 us from box to box, 6.8 TB/s, at the measured
// copy rate (6.77).  32 / 8 heads, one request of 128k: 53 us, 5.0 TB/s; of 4k: 11 us, of which start and join are
// 9.  61 of 6 to 8190 tokens, 40 / 8 heads: 38 us, 4.0 TB/s.  Heads of 64: 5.2 TB/s at best, a tile's chain of
// scores, softmax and product takes longer than its bytes (three CTAs an SM instead of two: registers spill, 102 ->
// 108 us).
#include <algorithm>

#include "kv_plan.cuh"

namespace moe {

constexpr float kPBias = 5.0f;             // log2 of p' at the running maximum
constexpr float kGrow = 3.0f;              // log2 by which a score may pass the maximum: p' stays below 256
constexpr int kBatch = 8;                  // tiles whose pages are looked up together, at most
constexpr int kItemUnits = 3;              // start and end of an item, in tiles
constexpr int kJoinGroup = 16;             // CTAs whose parts are added first where an item has many parts
constexpr int kJoinOnce = 40;              // parts x rows of a warp that are added in one step
constexpr float kTermStep = 32.0f;         // each further E4M3 term is scaled up by this
constexpr float kNoScore = -3e38f;         // running maximum before the first token: finite, so that
                                           // a masked score (-inf) minus it stays -inf

template <int kD, int kNR>
struct FewCfg {
  static constexpr int Rows = kNR < 16 ? kNR : 16;          // of a warpgroup
  static constexpr int WGs = kNR / Rows;
  static constexpr int Threads = 64 + 128 * WGs;
  static constexpr int HalfBytes = kTile * kD;              // K or V of a tile
  static constexpr int StageBytes = 2 * HalfBytes;
  static constexpr int CtasPerSm = kNR <= 16 ? 2 : 1;
  static constexpr int Stages = (kNR <= 16 ? 3 : 5) * (128 / kD);
  static constexpr int QBytes = 2 * kNR * kD;
  static constexpr int PPieces = kNR < 16 ? 2 : 3 * kNR / 16;   // of 16 columns: 8 rows' three terms fill 1.5
  static constexpr int PBytes = PPieces * 16 * kTile;
  static constexpr int SCols = 2 * kNR;                     // per score buffer, two of them
  static constexpr int OCol = 2 * SCols;
  static constexpr int TmemCols = kNR == 8 ? 64 : kNR == 16 ? 128 : kNR == 32 ? 256 : 512;
  static constexpr int LdCols = kNR == 64 || kNR == 8 ? 8 : 16;   // 64 rows: 96 registers a thread
  static constexpr int SlotBytes = 160;
  static constexpr int CtrlBytes = 1024 + Stages * SlotBytes + WGs * 5 * 16 * 4;
  static constexpr int Smem = 1024 + Stages * StageBytes + QBytes + PBytes + CtrlBytes;
  static_assert(OCol + 16 * PPieces <= TmemCols, "tensor memory");
  static_assert(CtasPerSm * (Smem + 1024) <= 228 * 1024, "shared memory");
};

// What the softmax warps need of a tile.
struct FewSlot {
  float kf[kMaxTilePages];     // K scale x sm_scale x log2 e
  float lv[kMaxTilePages];     // log2 V scale
  float iv[kMaxTilePages];     // 1 / V scale
  int token0;                  // first token of the tile
  int lo, hi;                  // tokens that some row sees
  int pos0, rows, q0, head;    // position of query token 0, live rows, row of it in q, key/value head
  int flags;                   // 2: last tile of the segment (the CTA's part of the item), 4: of the CTA
  int part;                    // workspace part that the segment fills, -1: the whole item is here
  int first_cta, parts;        // CTAs that share the item
  int first_part;              // part of the first of them; the others' first segment has part 2 x CTA
  int pad[4];
};
static_assert(sizeof(FewSlot) == 160, "slot");

struct FewParams {
  moe_kv_attention_args a;
  int G;                       // query heads per key/value head
  int page_shift;
  float* parts;                // [2 * ctas][kNR * (kD + 2)]
  int* arrived;                // [ctas][2][4] per CTA that opens a group or an item and 16 rows: parts, groups done
  int* status;
  int ctas;                    // CTAs that share the tiles; with a plan they follow one that lays it out
  PromptPlan plan;
};

// Request b: position of its first query token, query tokens (of more than max_q the first ones), and the
// tiles that hold the tokens its rows see (one, empty, when they see nothing; none: not this kernel's).
struct FewItem {
  int pos0, n, q0, lo, hi, tile0, tiles;
};

template <int kNR>
__device__ __forceinline__ FewItem few_item(const FewParams& p, int b) {
  FewItem it;
  it.q0 = p.a.tok_start[b];
  const int q1 = p.a.tok_start[b + 1], n = q1 - it.q0;
  it.n = min(n, p.a.max_q);
  it.pos0 = min(max(p.a.kv_len[b], 0), p.a.max_pages << p.page_shift) - n;
  it.lo = it.hi = it.tile0 = it.tiles = 0;
  // (comparisons only, so that no pair of entries passes by a difference that wraps round)
  if (it.q0 >= 0 && q1 > it.q0 && q1 <= p.a.T && it.n <= kNR / p.G) {
    it.hi = max(0, it.pos0 + it.n);
    if (p.a.window > 0) it.lo = max(0, it.pos0 - p.a.window + 1);
    it.tile0 = it.lo / kTile;
    it.tiles = max(1, (it.hi + kTile - 1) / kTile - it.tile0);
  }
  return it;
}

// Position in the CTA's tiles.
template <int kNR>
struct FewWalk {
  int b, h, tile;
  FewItem item;
  int left;                    // units from this tile to the CTA's end; <= 0: no tile here
  __device__ __forceinline__ void next(const FewParams& p) {
    if (--left <= 0 || ++tile < item.tiles) return;
    if ((left -= kItemUnits) <= 0) return;
    tile = 0;
    if (++h < p.a.Hkv) return;
    h = 0;
    do {
      item = few_item<kNR>(p, ++b);
    } while (item.tiles == 0 && b < p.a.B - 1);
  }
};

// kN values per lane (8 or 16) -> the reduction over the warp of value r = lane / (32 / kN).
template <bool kMax, int kN>
__device__ __forceinline__ float warp_reduce_rows(float (&v)[kN], int lane) {
  auto both = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int half = kN / 2; half >= 1; half >>= 1) {
    const int d = half * (32 / kN);
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = both(keep, __shfl_xor_sync(~0u, send, d));
    }
  }
  float r = v[0];
#pragma unroll
  for (int d = 16 / kN; d >= 1; d >>= 1) r = both(r, __shfl_xor_sync(~0u, r, d));
  return r;
}

// kN consecutive 32-bit tensor-memory columns of this warp's lanes (8 or 16).
template <int kN>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[kN]) {
  if constexpr (kN == 16) {
    tmem_ld16(taddr, r);
  } else {
    static_assert(kN == 8, "8 or 16 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  }
}

// Two FP16 values -> the E4M3 codes nearest to them, and 32 x what those leave over (exact in FP16:
// the difference has fewer bits than the value).
__device__ __forceinline__ uint32_t take_term(uint32_t& h2) {
  uint16_t code;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(code) : "r"(h2));
  uint32_t back;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(code));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h2) : "r"(back));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h2) : "r"(0x50005000u));
  return code;
}

// P lies token by token (MN-major B): 8 tokens x 16 rows of one term are 128 contiguous bytes, the
// terms' and warpgroups' 16-row pieces follow each other, then the next 8 tokens.  With 8 rows the first
// piece holds two terms, the second one and zeros.
template <int kNR>
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
  constexpr uint32_t kPieces = FewCfg<128, kNR>::PPieces;
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
  d |= (uint64_t)((kPieces * 128) >> 4) << 16;   // between groups of 8 tokens
  d |= (uint64_t)(128 >> 4) << 32;               // between pieces of 16 rows
  d |= (uint64_t)1 << 46;
  return d;
}

// Parts of an item that are added together: n of them, every step-th from i0 on.  Part 0 of the item lies
// at `first`, part i > 0 at rest + 2 i.  The sum goes to out if they are the whole item, else in i0's place.
struct JoinSet {
  int first, rest, i0, step, n;
  bool whole;
};

// kRows rows of an item, from `row` on and below row1.  One warp: the lanes read the parts' maxima and
// sums, then every lane its D / 32 values of all rows, with as many loads under way as registers allow,
// for latency is all there is to it.
constexpr int kJoinLoads = 8;
template <int kD, int kNR, int kRows>
__device__ __forceinline__ void join_rows(const FewParams& p, const JoinSet& set, int row, int row1, int q0,
                                          int head, int lane) {
  constexpr size_t kPart = kNR * (kD + 2);
  constexpr int kV = kD / 32;               // values of a row per lane
  const int n = set.n;
  auto part = [&](int k) {
    const int i = set.i0 + k * set.step;
    return p.parts + (size_t)(i == 0 ? set.first : set.rest + 2 * i) * kPart;
  };
  float m[kRows], l[kRows], acc[kRows][kV];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = kNoScore;
    l[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) acc[r][v] = 0.0f;
  }
  for (int i0 = 0; i0 < n; i0 += 32) {
    // this group of parts: weights relative to the maximum so far
    float w[kRows];
    float2 ml[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      ml[r] = make_float2(kNoScore, 0.0f);
      if (i0 + lane < n && row + r < row1)
        ml[r] = __ldcg(reinterpret_cast<const float2*>(part(i0 + lane) + kNR * kD + 2 * (row + r)));
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float top = fmaxf(m[r], ml[r].x);
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      const float alpha = m[r] == top ? 1.0f : exp2_approx(m[r] - top);
      w[r] = ml[r].x == top ? 1.0f : exp2_approx(ml[r].x - top);
      m[r] = top;
      l[r] = __fmaf_rn(l[r], alpha, ml[r].y * w[r]);
#pragma unroll
      for (int v = 0; v < kV; ++v) acc[r][v] *= alpha;
    }
    const int k1 = min(32, n - i0);
#pragma unroll(kJoinLoads / kRows)
    for (int k = 0; k < k1; ++k) {
      const float* o = part(i0 + k) + lane * kV;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float wk = __shfl_sync(~0u, w[r], k);
        float x[kV];
        const float* at = o + min(row + r, row1 - 1) * kD;
        if (kV == 4) *reinterpret_cast<float4*>(x) = __ldcg(reinterpret_cast<const float4*>(at));
        else *reinterpret_cast<float2*>(x) = __ldcg(reinterpret_cast<const float2*>(at));
#pragma unroll
        for (int v = 0; v < kV; ++v) acc[r][v] = __fmaf_rn(x[v], wk, acc[r][v]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int d = 16; d; d >>= 1) l[r] += __shfl_xor_sync(~0u, l[r], d);
    if (row + r >= row1) break;
    if (!set.whole) {
      float* o = part(0);
#pragma unroll
      for (int v = 0; v < kV; ++v) o[(row + r) * kD + lane * kV + v] = acc[r][v];
      if (lane == 0) *reinterpret_cast<float2*>(o + kNR * kD + 2 * (row + r)) = make_float2(m[r], l[r]);
      continue;
    }
    const float inv = l[r] > 0.0f || l[r] != l[r] ? 1.0f / l[r] : 0.0f;
    const int i = (row + r) / p.G;
    uint32_t* out = reinterpret_cast<uint32_t*>(
        static_cast<uint16_t*>(p.a.out) + (int64_t)(q0 + i) * p.a.out_token_stride +
        (int64_t)(head * p.G + row + r - i * p.G) * p.a.out_head_stride + lane * kV);
    out[0] = pack_bf16x2(acc[r][0] * inv, acc[r][1] * inv);
    if (kV == 4) out[1] = pack_bf16x2(acc[r][kV - 2] * inv, acc[r][kV - 1] * inv);
  }
}

template <int kD, int kNR>
__global__ void __launch_bounds__(FewCfg<kD, kNR>::Threads, FewCfg<kD, kNR>::CtasPerSm)
    k_attn_few(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ FewParams p) {
  using C = FewCfg<kD, kNR>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  uint8_t* ctrl = smem + C::Stages * C::StageBytes + C::QBytes + C::PBytes;
  const uint32_t sQ = sbase + C::Stages * C::StageBytes, sP = sQ + C::QBytes;
  FewSlot* slots = reinterpret_cast<FewSlot*>(ctrl + 1024);
  float* red = reinterpret_cast<float*>(ctrl + 1024 + C::Stages * C::SlotBytes);   // [WGs][5][16]
  const uint32_t bar0 = smem_addr(ctrl);
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto vfull = [&](int s) { return bar0 + 8u * (C::Stages + s); };
  auto ifull = [&](int s) { return bar0 + 8u * (2 * C::Stages + s); };
  auto empty = [&](int s) { return bar0 + 8u * (3 * C::Stages + s); };
  constexpr int kB = 4 * C::Stages;
  auto sfull = [&](int b) { return bar0 + 8u * (kB + b); };
  const uint32_t qfull = bar0 + 8u * (kB + 2), pfull = bar0 + 8u * (kB + 3), ofull = bar0 + 8u * (kB + 4);
  const uint32_t drain = bar0 + 8u * (kB + 5);
  static_assert(8 * (kB + 6) + 16 + 208 <= 1024, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (kB + 6));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* mma_done = reinterpret_cast<volatile int*>(tmem_slot + 2);
  int* scan = reinterpret_cast<int*>(ctrl + 8 * (kB + 6) + 16);   // [warps + 2], an item

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = p.status;

  const int cta = (int)blockIdx.x - (p.plan.list != nullptr ? 1 : 0);
  if (cta < 0) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    prompt_plan(p.a, p.plan, p.G, p.page_shift, reinterpret_cast<int*>(smem));
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::Stages; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(vfull(s), 1);
      mbar_init(ifull(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(sfull(0), 1);
    mbar_init(sfull(1), 1);
    mbar_init(qfull, 4 * C::WGs);
    mbar_init(pfull, 4 * C::WGs);
    mbar_init(ofull, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *mma_done = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), C::TmemCols);

  // ------------------------------------------------------------ the CTA's share of the units
  // an exclusive sum over threads with consecutive requests each
  auto weight = [&](const FewItem& it) { return it.tiles ? (it.tiles + kItemUnits) * p.a.Hkv : 0; };
  grid_dep_wait();
  // With prompts the next kernel's start is the call's own; else it would only be in this one's way (1 x 4k:
  // 11.2 -> 11.6 us).
  if (p.plan.list != nullptr) grid_dep_launch_dependents();
  const int per = (p.a.B + C::Threads - 1) / C::Threads;
  const int rb0 = threadIdx.x * per, rb1 = min(p.a.B, rb0 + per);
  int mine = 0;
  for (int b = rb0; b < rb1; ++b) mine += weight(few_item<kNR>(p, b));
  int pre = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(~0u, pre, d);
    if (lane >= d) pre += t;
  }
  constexpr int kWarps = C::Threads / 32;
  static_assert(4 * (kWarps + 2) + (int)sizeof(FewItem) <= 208, "scan area");
  if (lane == 31) scan[warp] = pre;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  int total = 0;
  pre -= mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) pre += scan[w];
    total += scan[w];
  }
  // (the CTAs that share an item are neighbours: none between them is without units)
  const int share = (total + p.ctas - 1) / p.ctas;
  const int u0 = min(total, cta * share), u1 = min(total, u0 + share);
  if (u0 < u1 && u0 >= pre && u0 < pre + mine) {
    int at = pre;
    for (int b = rb0; b < rb1; ++b) {
      const FewItem it = few_item<kNR>(p, b);
      const int w = weight(it);
      if (u0 < at + w) {
        scan[kWarps] = b;
        scan[kWarps + 1] = u0 - at;
        *reinterpret_cast<FewItem*>(scan + kWarps + 2) = it;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  // the first tile of the share: where the share begins within an item's own units, tile 0 follows
  FewWalk<kNR> cur;
  cur.left = u1 - u0;
  cur.b = cur.h = cur.tile = 0;
  cur.item = FewItem{};
  if (u0 < u1) {
    cur.b = scan[kWarps];
    cur.item = *reinterpret_cast<const FewItem*>(scan + kWarps + 2);
    const int u = scan[kWarps + 1], per_item = cur.item.tiles + kItemUnits;
    cur.h = u / per_item;
    const int at = u - cur.h * per_item - kItemUnits;
    cur.tile = max(at, 0);
    cur.left += min(at, 0);
  }

  int issued = 0;
  if (cur.left > 0) {
    if (warp == 0) {
      // -------------------------------------------------------------------- producer
      // The page table and the scales it leads to are two dependent loads, so they run ahead of the
      // copies by two batches and one.  A batch is the next kBatch tiles of the walk (fewer with small
      // pages): lane = tile of the batch x page of the tile, and the lanes of a tile do all its work.
      const int npg = kTile >> p.page_shift, P = 1 << p.page_shift;
      const int group = lane / npg, pi = lane - group * npg;
      const int batch = min(kBatch, 32 / npg);
      const bool leader = pi == 0;
      int seg = 0;
      struct Ahead {
        FewItem item;
        int b, h, tile, page, seg;       // page: -1 none; seg: segments of the CTA before this one
        int left;                        // units from the tile to the CTA's end
        int live;                        // 0: no such tile, 1: tile, 2: the CTA's last
      };
      // the lane's tile of the next batch, and its page
      auto look = [&]() {
        Ahead a;
        a.live = 0;
        a.page = -1;
        a.seg = a.left = 0;
        for (int k = 0; k < batch && cur.left > 0; ++k) {
          if (k == group) {
            a.item = cur.item;
            a.b = cur.b;
            a.h = cur.h;
            a.tile = cur.tile;
            a.seg = seg;
            a.left = cur.left;
            a.live = 1;
          }
          if (cur.tile == cur.item.tiles - 1) ++seg;
          cur.next(p);
          if (k == group && cur.left <= 0) a.live = 2;
        }
        if (a.live) {
          const int pg = (a.item.tile0 + a.tile) * npg + pi;
          if ((pg << p.page_shift) < a.item.hi && ((pg + 1) << p.page_shift) > a.item.lo)
            a.page = p.a.block_table[(size_t)a.b * p.a.max_pages + pg];
        }
        return a;
      };
      auto scales = [&](const Ahead& a, float& ks, float& vs) {
        ks = vs = 0.0f;
        if (a.page >= 0 && a.page < p.a.num_pages) {
          ks = p.a.k_scale[(size_t)a.page * p.a.Hkv + a.h];
          vs = p.a.v_scale[(size_t)a.page * p.a.Hkv + a.h];
        }
      };
      Ahead now = look(), nxt;
      float ks, vs;
      scales(now, ks, vs);
      bool ok = true, more = true;
      for (int it = 0; ok && more;) {
        const bool begins = it == 0;
        const bool live = now.page >= 0 && now.page < p.a.num_pages;
        const uint32_t pages = __ballot_sync(~0u, live);
        const uint32_t bytes = __popc((pages >> (group * npg)) & ((1u << npg) - 1)) * P * kD;
        float kf = 0.0f, lv = 0.0f, iv = 0.0f;
        for (int k = 0; k < batch; ++k) {
          if (!__any_sync(~0u, group == k && now.live)) break;
          const int s = it % C::Stages;
          const bool mine = group == k;
          bool here = true;
          if (mine && leader) {
            here = bounded_wait(empty(s), ((it / C::Stages) & 1) ^ 1, abort_flag, status);
            if (here) {
              mbar_arrive_expect_tx(kfull(s), bytes);
              mbar_arrive_expect_tx(vfull(s), bytes);
            }
          }
          ok = __all_sync(~0u, here);
          if (!ok) break;
          FewSlot& slot = slots[s];
          if (mine) {
            if (live) {
              const uint32_t dst = sbase + s * C::StageBytes + pi * P * kD;
              tma_load_4d(dst, &tmK, 0, 0, now.h, now.page, kfull(s));
              tma_load_4d(dst + C::HalfBytes, &tmV, 0, 0, now.h, now.page, vfull(s));
            }
          }
          if (k == 0) {
            // the scales are needed only now that the batch's first copies are on their way
            kf = ks * p.a.sm_scale * kLog2e;
            const float v = vs >= 0.0f ? fmaxf(vs, 1e-30f) : vs;
            lv = log2f(v);
            iv = __fdiv_rn(1.0f, v);
          }
          if (mine) {
            slot.kf[pi] = kf;
            slot.lv[pi] = lv;
            slot.iv[pi] = iv;
            if (leader) {
              const bool end = now.tile == now.item.tiles - 1, last = now.live == 2;
              slot.token0 = (now.item.tile0 + now.tile) * kTile;
              slot.lo = now.item.lo;
              slot.hi = now.item.hi;
              slot.pos0 = now.item.pos0;
              slot.rows = now.item.n * p.G;
              slot.q0 = now.item.q0;
              slot.head = now.h;
              slot.flags = (end || last ? 2 : 0) | (last ? 4 : 0);
              if (end || last) {
                // the item's units: its own from `begin`, then its tiles
                const int begin = u1 - now.left - now.tile - kItemUnits;
                const int first = (begin + kItemUnits) / share;
                const int n = (begin + kItemUnits + now.item.tiles - 1) / share - first + 1;
                slot.part = n == 1 ? -1 : 2 * cta + (now.seg > 0 ? 1 : 0);
                slot.first_cta = first;
                slot.parts = n;
                slot.first_part = 2 * first + (first * share < begin ? 1 : 0);
              }
            }
          }
          __syncwarp();
          if (mine && leader) mbar_arrive(ifull(s));
          ++it;
          ++issued;
        }
        more = !__any_sync(~0u, now.live == 2);
        if (begins) nxt = look();
        const Ahead far = look();
        scales(nxt, ks, vs);
        now = nxt;
        nxt = far;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------------- MMA
      {
        constexpr uint32_t kIdescS = make_idesc_e4m3(kTile, 2 * kNR);
        constexpr uint32_t kIdescO = make_idesc_e4m3(kD, 16 * C::PPieces) | (3u << 15);   // both MN-major
        const uint64_t qd = rows_desc<kD>(sQ), pd = p_desc<kNR>(sP);
        int segs = 0;
        auto scores = [&](int it) {
          const int s = it % C::Stages;
          if (!mbar_wait_warp(kfull(s), (it / C::Stages) & 1, abort_flag, status)) return false;
          tc_fence_after_sync();
          const uint64_t kd = rows_desc<kD>(sbase + s * C::StageBytes);
          const uint32_t d = tmem + (it & 1) * C::SCols;
#pragma unroll
          for (int k = 0; k < kD / 32; ++k) mma_f8_warp(d, kd + 2 * k, qd + 2 * k, kIdescS, k > 0);
          mma_commit_warp(sfull(it & 1));
          return true;
        };
        for (int it = 0;; ++it) {
          const int s = it % C::Stages;
          if (it == 0) {
            if (!mbar_wait_warp(qfull, segs & 1, abort_flag, status) || !scores(0)) break;
            ++segs;
          }
          if (!mbar_wait_warp(ifull(s), (it / C::Stages) & 1, abort_flag, status)) break;
          const int flags = *reinterpret_cast<volatile int*>(&slots[s].flags);
          const bool more = !(flags & 4), same = !(flags & 2);
          if (same && !scores(it + 1)) break;
          if (!mbar_wait_warp(pfull, it & 1, abort_flag, status) ||
              !mbar_wait_warp(vfull(s), (it / C::Stages) & 1, abort_flag, status))
            break;
          tc_fence_after_sync();
          const uint32_t sv = sbase + s * C::StageBytes + C::HalfBytes;
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma_f8_warp(tmem + C::OCol, rows_desc<kD>(sv + k * 32 * kD), pd + k * (32 * C::PPieces), kIdescO, k > 0);
          mma_commit_warp(ofull);
          mma_commit_warp(empty(s));
          if (lane == 0) *mma_done = it + 1;
          if (more && !same) {
            if (!mbar_wait_warp(qfull, segs & 1, abort_flag, status) || !scores(it + 1)) break;
            ++segs;
          }
          if (!more) break;
        }
      }
    } else {
      // --------------------------------------------------------------------- softmax
      const int wg = (warp - 2) >> 2, q = warp & 3;
      const int tl = q * 32 + lane;                     // token of the tile
      const int wt = (warp - 2 - 4 * wg) * 32 + lane;   // thread of the warpgroup, for Q
      const bool holds_d = kD == 128 || lane < 16;
      const int d = kD == 128 ? tl : q * 16 + lane;     // output column of this thread
      float* wred = red + wg * 80;                      // [4 warps][16 rows], for reductions
      float* wqs = wred + 64;                           // [16 rows] value of a code of Q
      const int r0 = wg * 16;
      constexpr int kR = C::Rows;
      constexpr uint32_t kAllRows = (1u << kR) - 1;
      constexpr int kRowLanes = 32 / kR;                // lanes that share a row's reduction
      float m[kR];
      f32x2 l[kR / 2], acc[kR / 2];                     // two rows each
      // A wait that runs out only marks the thread: the warpgroup leaves together, at the next vote,
      // so no barrier is left waiting.
      bool pending = false, bad = false, begin = true;
      auto add_output = [&](int it) {                   // O of tile it
        if (!bounded_wait(ofull, it & 1, abort_flag, status)) {
          bad = true;
          return;
        }
        tc_fence_after_sync();
        const f32x2 step = pack2(1.0f / kTermStep, 1.0f / kTermStep);
#pragma unroll
        for (int r0s = 0; r0s < kR; r0s += C::LdCols) {
          uint32_t t[3][C::LdCols];
          const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + C::OCol + r0 + r0s;
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_ldn<C::LdCols>(at + k * kNR, t[k]);
          tmem_ld_wait();
          auto pair = [&](int k, int r) {
            return pack2(__uint_as_float(t[k][2 * r]), __uint_as_float(t[k][2 * r + 1]));
          };
#pragma unroll
          for (int r = 0; r < C::LdCols / 2; ++r)
            acc[r0s / 2 + r] =
                add2(fma2(fma2(pair(2, r), step, pair(1, r)), step, pair(0, r)), acc[r0s / 2 + r]);
        }
        tc_fence_before_sync();
      };
      // Q of the segment that begins with tile `it`: 8 threads a row, D / 8 values each, two E4M3 terms.
      // The scores of the segment before are done: this warpgroup has read them.
      auto load_q = [&](int rows, int q0, int head) {
        constexpr int kV = kD / 8;
        if (wt < 8 * kR) {
          const int r = r0 + (wt >> 3), c = wt & 7;
          float x[kV];
#pragma unroll
          for (int i = 0; i < kV; ++i) x[i] = 0.0f;
          if (r < rows) {
            const int i = r / p.G;
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(p.a.q) + (int64_t)(q0 + i) * p.a.q_token_stride +
                (int64_t)(head * p.G + r - i * p.G) * p.a.q_head_stride + c * kV);
#pragma unroll
            for (int v = 0; v < kV / 8; ++v) {
              const uint4 w = src[v];
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                x[8 * v + 2 * j] = __uint_as_float(u[j] << 16);
                x[8 * v + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
              }
            }
          }
          float amax = 0.0f;
#pragma unroll
          for (int i = 0; i < kV; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
          // amax x mul in [128, 256)
          const int e = amax > 0.0f ? max((int)(__float_as_uint(amax) >> 23) - 127, -100) : 0;
          // (0 where a value is infinite: its code becomes NaN, where a saturated one would make a finite score)
          const float mul = e == 128 ? 0.0f : __uint_as_float((uint32_t)(127 + 7 - e) << 23);
          uint32_t t1[kV / 4], t2[kV / 4];
#pragma unroll
          for (int i = 0; i < kV / 4; ++i) {
            t1[i] = t2[i] = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float a = x[4 * i + 2 * j] * mul, b = x[4 * i + 2 * j + 1] * mul;
              const uint32_t code = cvt_e4m3x2(a, b);
              float fa, fb;
              e4m3x2_to_f32(code, fa, fb);
              t1[i] |= code << (16 * j);
              t2[i] |= cvt_e4m3x2((a - fa) * kTermStep, (b - fb) * kTermStep) << (16 * j);
            }
          }
          uint8_t* qb = smem + C::Stages * C::StageBytes;
#pragma unroll
          for (int i = 0; i < kV / 4; i += 2) {
            *reinterpret_cast<uint2*>(qb + swz<kD>(r, c * kV + 4 * i)) = make_uint2(t1[i], t1[i + 1]);
            *reinterpret_cast<uint2*>(qb + swz<kD>(kNR + r, c * kV + 4 * i)) = make_uint2(t2[i], t2[i + 1]);
          }
          if (c == 0) wqs[wt >> 3] = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
        }
        fence_proxy_async_smem();
        named_barrier_sync(1 + wg, 128);
        if (lane == 0) mbar_arrive(qfull);
      };
      // the segment whose Q comes next; the CTA's first is known before the producer has its pages
      int q_rows = cur.item.n * p.G, q_q0 = cur.item.q0, q_head = cur.h;
      load_q(q_rows, q_q0, q_head);
      for (int it = 0;; ++it) {
        const int s = it % C::Stages;
        if (!bounded_wait(ifull(s), (it / C::Stages) & 1, abort_flag, status)) bad = true;
        const FewSlot& slot = slots[s];
        const int rows = bad ? 0 : slot.rows, pos0 = slot.pos0, q0 = slot.q0, head = slot.head;
        if (begin) {
#pragma unroll
          for (int i = 0; i < kR; ++i) m[i] = kNoScore;
#pragma unroll
          for (int i = 0; i < kR / 2; ++i) l[i] = acc[i] = 0ull;
        }
        // scores of this thread's token
        const int page = tl >> p.page_shift;
        const float kf = slot.kf[page], lv = slot.lv[page], iv = slot.iv[page];
        const int j = slot.token0 + tl;
        const bool edge = slot.token0 < slot.lo || slot.token0 + kTile > slot.hi;
        // rows [from, to) of the warpgroup see the token; rows past the live ones may see anything
        int from = max(j - pos0, 0) * p.G, to = kR + r0;
        if (p.a.window > 0)
          to = min(to, j - pos0 + p.a.window > 0 ? min(j - pos0 + p.a.window, 64) * p.G : 0);
        if (j >= slot.hi || j < slot.lo) to = 0;
        from = min(max(from - r0, 0), kR);
        to = min(max(to - r0, 0), kR);
        const uint32_t seen = to > from ? ((1u << to) - (1u << from)) : 0u;
        if (!bounded_wait(sfull(it & 1), (it >> 1) & 1, abort_flag, status)) bad = true;
        tc_fence_after_sync();
        float sc[kR];
        {
          const f32x2 step = pack2(1.0f / kTermStep, 1.0f / kTermStep), kf2 = pack2(kf, kf), lv2 = pack2(lv, lv);
#pragma unroll
          for (int r0s = 0; r0s < kR; r0s += C::LdCols) {
            uint32_t t[C::LdCols], t2[C::LdCols];
            const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (it & 1) * C::SCols + r0 + r0s;
            tmem_ldn<C::LdCols>(at, t);
            tmem_ldn<C::LdCols>(at + kNR, t2);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < C::LdCols; r += 4) {
              const float4 qs = *reinterpret_cast<const float4*>(wqs + r0s + r);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int x = r + 2 * i;
                const f32x2 v = fma2(pack2(__uint_as_float(t2[x]), __uint_as_float(t2[x + 1])), step,
                                     pack2(__uint_as_float(t[x]), __uint_as_float(t[x + 1])));
                const f32x2 f = mul2(i ? pack2(qs.z, qs.w) : pack2(qs.x, qs.y), kf2);
                unpack2(fma2(v, f, lv2), sc[r0s + x], sc[r0s + x + 1]);
              }
            }
          }
          tc_fence_before_sync();
          if (seen != kAllRows) {
#pragma unroll
            for (int r = 0; r < kR; ++r)
              if (!((seen >> r) & 1)) sc[r] = -INFINITY;
          }
        }
        bool grow = false;
#pragma unroll
        for (int r = 0; r < kR; ++r) grow |= sc[r] > m[r] + (kGrow + kPBias);
        if (vote_any<128>(1 + wg, grow || bad)) {
          if (vote_any<128>(1 + wg, bad)) break;
          // the maximum of some row moved: bring what is outstanding in, then rescale
          if (pending) add_output(it - 1);
          pending = false;
          float v[kR];
#pragma unroll
          for (int r = 0; r < kR; ++r) v[r] = sc[r];
          const float top = warp_reduce_rows<true, kR>(v, lane);
          if (!(lane & (kRowLanes - 1))) wred[q * 16 + lane / kRowLanes] = top;
          named_barrier_sync(1 + wg, 128);
#pragma unroll
          for (int r = 0; r < kR; r += 2) {
            float alpha[2];
#pragma unroll
            for (int i = r; i < r + 2; ++i) {
              const float t = fmaxf(fmaxf(wred[i], wred[16 + i]), fmaxf(wred[32 + i], wred[48 + i]));
              const float mn = fmaxf(m[i], t - kPBias);
              alpha[i - r] = m[i] == mn ? 1.0f : exp2_approx(m[i] - mn);
              m[i] = mn;
            }
            l[r / 2] = mul2(l[r / 2], pack2(alpha[0], alpha[1]));
            acc[r / 2] = mul2(acc[r / 2], pack2(alpha[0], alpha[1]));
          }
        }
        if (pending) add_output(it - 1);
        // probabilities, rounded to FP16 (11 bits, down to 2^-29), then three E4M3 terms each
        uint32_t term[3][kR / 4];
#pragma unroll
        for (int r = 0; r < kR; r += 2) {
          float p0, p1;
          unpack2(add2(pack2(sc[r], sc[r + 1]), pack2(-m[r], -m[r + 1])), p0, p1);
          const f32x2 pr = pack2(exp2_approx(p0), exp2_approx(p1));
          l[r / 2] = fma2(pr, pack2(iv, iv), l[r / 2]);
          unpack2(pr, p0, p1);
          uint32_t h2 = pack_f16x2(p0, p1);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t code = take_term(h2);
            if (r & 2) term[k][r / 4] |= code << 16;
            else term[k][r / 4] = code;
          }
        }
        uint8_t* pt = smem + (sP - sbase) + (tl >> 3) * (C::PPieces * 128) + (tl & 7) * 16;
        if constexpr (kR == 8) {
          *reinterpret_cast<uint4*>(pt) = make_uint4(term[0][0], term[0][1], term[1][0], term[1][1]);
          *reinterpret_cast<uint4*>(pt + 128) = make_uint4(term[2][0], term[2][1], 0, 0);
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4*>(pt + (k * C::WGs + wg) * 128) =
                make_uint4(term[k][0], term[k][1], term[k][kR / 4 - 2], term[k][kR / 4 - 1]);
        }
        if (edge && wg == 0) {
          // V rows that no query row sees may hold anything: 0 x NaN would spread
          if (!bounded_wait(vfull(s), (it / C::Stages) & 1, abort_flag, status)) bad = true;
          if (j < slot.lo || j >= slot.hi) {
            uint4* row = reinterpret_cast<uint4*>(smem + s * C::StageBytes + C::HalfBytes + tl * kD);
#pragma unroll
            for (int i = 0; i < kD / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
          }
        }
        pending = true;
        const int part = slot.part, first_cta = slot.first_cta, parts = slot.parts, first_part = slot.first_part;
        const int flags = slot.flags;
        begin = flags & 2;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
        if (begin) {
          // ------------------------------------------------------- end of the segment
          if (!(flags & 4)) {                  // the next segment's, while the last P V runs
            const int ns = (it + 1) % C::Stages;
            if (!bounded_wait(ifull(ns), ((it + 1) / C::Stages) & 1, abort_flag, status)) bad = true;
            load_q(bad ? 0 : slots[ns].rows, slots[ns].q0, slots[ns].head);
          }
          add_output(it);
          pending = false;
          float lr[kR], ar[kR];
#pragma unroll
          for (int r = 0; r < kR / 2; ++r) {
            unpack2(l[r], lr[2 * r], lr[2 * r + 1]);
            unpack2(acc[r], ar[2 * r], ar[2 * r + 1]);
          }
          const float sum = warp_reduce_rows<false, kR>(lr, lane);
          if (!(lane & (kRowLanes - 1))) wred[q * 16 + lane / kRowLanes] = sum;
          named_barrier_sync(1 + wg, 128);
          // every kR-th lane from r on knows row r's sum and place; the others ask them
          const int mr = lane & (kR - 1), my_row = r0 + mr;
          const float lsum = (wred[mr] + wred[16 + mr]) + (wred[32 + mr] + wred[48 + mr]);
          if (part < 0) {
            const float inv = lsum > 0.0f || lsum != lsum ? 1.0f / lsum : 0.0f;
            const int i = my_row / p.G;
            const long long at = (long long)(q0 + i) * p.a.out_token_stride +
                                 (long long)(head * p.G + my_row - i * p.G) * p.a.out_head_stride;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              if (r0 + r >= rows) break;
              const float f = __shfl_sync(~0u, inv, r);
              const long long o = __shfl_sync(~0u, at, r);
              if (holds_d) static_cast<uint16_t*>(p.a.out)[o + d] = (uint16_t)f32_to_bf16_bits(ar[r] * f);
            }
          } else {
            float* o = p.parts + (size_t)part * (kNR * (kD + 2));
            float mm = 0.0f;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              if (mr == r) mm = m[r];
              if (r0 + r < rows && holds_d) o[(r0 + r) * kD + d] = ar[r];
            }
            if (wt < kR && my_row < rows)
              *reinterpret_cast<float2*>(o + kNR * kD + 2 * my_row) = make_float2(mm, lsum);
          }
          if (part >= 0) {
            // the last of a group of CTAs to get here adds the group's parts, the last of the groups theirs
            const int row1 = min(rows, r0 + kR), jw = wt >> 5;
            JoinSet set;
            set.first = first_part;
            set.rest = 2 * first_cta;
            set.whole = parts <= kJoinGroup || (row1 - r0 + 3) / 4 * parts <= kJoinOnce;
            set.i0 = set.whole ? 0 : (cta - first_cta) & -kJoinGroup;
            set.step = 1;
            set.n = set.whole ? parts : min(kJoinGroup, parts - set.i0);
            int* arrived = p.arrived + 8 * (first_cta + set.i0) + wg;
            while (true) {
              if (set.n > 1) {
                __threadfence();
                named_barrier_sync(1 + wg, 128);
                if (wt == 0) {
                  const int before = atomicAdd(arrived, 1);
                  if (before == set.n - 1) *arrived = 0;
                  __threadfence();
                  wred[0] = before == set.n - 1 ? 1.0f : 0.0f;
                }
                named_barrier_sync(1 + wg, 128);
                if (wred[0] == 0.0f) break;
                if (kNR == 64 || row1 - r0 <= 4) {   // 64 rows: no registers for more at once
                  for (int row = r0 + jw; row < row1; row += 4)
                    join_rows<kD, kNR, 1>(p, set, row, row1, q0, head, lane);
                } else {
                  for (int row = r0 + 2 * jw; row < row1; row += 8)
                    join_rows<kD, kNR, 2>(p, set, row, row1, q0, head, lane);
                }
              }
              if (set.whole) break;
              set.i0 = 0;
              set.step = kJoinGroup;
              set.n = (parts + kJoinGroup - 1) / kJoinGroup;
              set.whole = true;
              arrived = p.arrived + 8 * first_cta + 4 + wg;
            }
          }
          named_barrier_sync(1 + wg, 128);     // the sums have been read
          if (flags & 4) break;
        }
      }
    }
  }

  // ------------------------------------------------------------------------ teardown
  __syncthreads();
  grid_dep_launch_dependents();
  auto drain_wait = [&](uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicCAS(status, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
        return;
      }
    }
  };
  if (warp == 1) {
    mma_commit_warp(drain);
    drain_wait(drain, 0);
  }
  if (warp == 0 && lane == 0 && *abort_flag) {
    for (int i = *mma_done; i < issued; ++i) {
      drain_wait(kfull(i % C::Stages), (i / C::Stages) & 1);
      drain_wait(vfull(i % C::Stages), (i / C::Stages) & 1);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TmemCols);
  }
}

// ------------------------------------------------------------------------------------ launch
// Rows per item of a call: tokens of a request x heads that share a key/value head, 8, 16, 32 or 64.  Rows
// cost softmax time whether they are live or not, so the fewest that hold them win: 64 x 4000 tokens, 4 rows
// live, 8 / 16 / 32 / 64 rows: 89 / 90 / 120 / 235 us; 40 x 4000, 16 live: 42 / 51 / 89 us from 16 on.
// More than 64 rows are the prompt kernel's; up to 64 this one is faster (32 rows, 32 x 4000: 44 against
// 114 us; 64 rows, 32 x 8000: 121 against 198 us), and at 72 and 96 the prompt kernel costs what it does at 64.
int few_rows(int G, int max_q) {
  const long long r = (long long)G * max_q;
  const long long rows = r <= 64 ? r : G;   // prompts: the single tokens among them still come here
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

static int few_ctas(int nr) { return nr <= 16 ? 304 : 152; }   // at most; 152 SMs

// The same for all variants: calls with other row counts may use the workspace in between, and must leave
// the counters at zero.
size_t few_counter_bytes() { return (256 + (size_t)few_ctas(8) * 32 + 255) & ~(size_t)255; }

size_t few_parts_bytes(int D, int nr) { return (size_t)2 * few_ctas(nr) * nr * (D + 2) * 4; }

template <int kD, int kNR>
static cudaError_t launch(const moe_kv_attention_args& a, void* workspace, void* plan, void* parts, cudaStream_t s) {
  using C = FewCfg<kD, kNR>;
  CUtensorMap tmK, tmV;
  if (!cache_map(&tmK, a.k_codes, kD, a.page_size, a.Hkv, a.num_pages, a.page_size, kD) ||
      !cache_map(&tmV, a.v_codes, kD, a.page_size, a.Hkv, a.num_pages, a.page_size, kD))
    return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(k_attn_few<kD, kNR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem);
  if (err != cudaSuccess) return err;
  const int ctas = std::min(few_ctas(kNR), sm_count() * C::CtasPerSm);
  FewParams p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int*>(ws);
  p.arrived = reinterpret_cast<int*>(ws + 256);
  p.parts = static_cast<float*>(parts);
  p.ctas = ctas - (plan != nullptr ? 1 : 0);   // all of the grid at once on the SMs
  p.plan = PromptPlan{};
  if (plan != nullptr) p.plan = prompt_plan_at(plan);
  p.plan.min_n = kNR / p.G;
  static_assert(C::Smem - 1024 >= kPlanSmem, "shared memory");
  return launch_pdl(k_attn_few<kD, kNR>, dim3(ctas), dim3(C::Threads), C::Smem, s, tmK, tmV, p);
}

template <int kD>
static cudaError_t launch_rows(const moe_kv_attention_args& a, int nr, void* workspace, void* plan, void* parts,
                               cudaStream_t s) {
  switch (nr) {
    case 8: return launch<kD, 8>(a, workspace, plan, parts, s);
    case 16: return launch<kD, 16>(a, workspace, plan, parts, s);
    case 32: return launch<kD, 32>(a, workspace, plan, parts, s);
    default: return launch<kD, 64>(a, workspace, plan, parts, s);
  }
}

cudaError_t launch_attn_few(const moe_kv_attention_args& a, int nr, void* workspace, void* plan, void* parts,
                            cudaStream_t s) {
  return a.D == 128 ? launch_rows<128>(a, nr, workspace, plan, parts, s)
                    : launch_rows<64>(a, nr, workspace, plan, parts, s);
}

}  // namespace moe
