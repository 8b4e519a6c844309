// Attention over the 8-bit paged cache for many query rows per request: prompts and chunks.
//
// Two matrix products of 128 x 128 x D per 128-token tile and 128 rows, so the tensor cores are the
// bound; the exponentials, then shared memory's bandwidth, come close behind.  A block is 512 rows of one
// request and key/value head (row = token x heads that share the head + head: any group size fills the
// tiles).  Two CTAs on neighbouring SMs work on it together (cta_group::2): each has two tiles of 128 rows,
// and a product takes one tile of each, so that every K and V tile is fetched, widened and read once for
// 512 rows.  While one pair of tiles is in the softmax the tensor cores work on the other.
//   S = Q K^T   kind::f8f6f4: the K codes as they are; a row of Q, scaled by a power of two, as two
//               E4M3 terms one after the other along the reduction (2 x D at twice the 16-bit rate)
//   O += P V    kind::f16: P in FP16 from tensor memory (it takes the place of S), V codes widened to
//               FP16, which is exact, by a warpgroup that has nothing else to do
// The pages' scales cost nothing per value: with f = K scale x softmax scale and lv = log2 V scale a
// probability is formed as p' = 2^(s f + lv - M), one multiply-add per value, where M is the row's
// running maximum of s f + lv.  O = sum p' code needs no scale, the row sum is sum p' / V scale, one
// multiply-add per 16 values.  M moves only when a row passes it by 2^8, so the rescaling of O is rare;
// p' carries a factor of 2^4, which leaves FP16 its full precision down to 2^-18 of the maximum.
//
//   warp 0        producer: lane i fetches page i of a tile (half the tokens of K, half the values of V)
//                 and its scales
//   warp 1        leader: MMA issuer; peer: tells the leader that its K has landed
//   warps 4..7    V codes -> FP16
//   warps 8..15   softmax: thread = row, one warpgroup per tile of rows
// Work: rounds over the blocks, longest first, and a last one whose tiles are poured over the pairs up to
// a common level (kv_plan.cuh).  Blocks that this cuts along the cache k_prompt_join adds up, in order.
//
// 4096 tokens after 28000, 32 / 8 heads of 128: 1.31 ms in a short burst, 1.54 PFLOP/s, 81% of the measured
// 16-bit rate; 1.34 to 1.36 ms back to back, where the power cap holds the clock.  At 1.42 ms the other layouts
// took: one CTA per block of 256 rows 1.59 ms; V read past shared memory 1.72 ms;
// two threads a row 1.52 ms; an issuing warp per tile of rows 1.85 ms.  A step of 512 rows x 128 tokens takes
// about 3300 cycles, of which the products need 2050: what is left is the chain score -> softmax -> product
// of each tile.  Five prompts of 300 to 4000 tokens: 174 us, 1.04 PFLOP/s, the start and end of each block
// being about 2.5 steps.
#include <algorithm>

#include "kv_plan.cuh"

namespace moe {

constexpr int kPromptThreads = 512;
constexpr float kPromptGrow = 8.0f;           // log2 by which a row may pass its maximum
constexpr float kPromptBias = 4.0f;           // log2 of p' at the maximum
// registers of the four warpgroups, launched with 128 each
constexpr int kRegsIssue = 88, kRegsWiden = 40, kRegsSoftmax = 192;
static_assert(kRegsIssue + kRegsWiden + 2 * kRegsSoftmax <= 512, "register split must fit the launch");

template <int kD>
struct PromptCfg {
  static constexpr int QTerm = 128 * kD;                 // one E4M3 term of a row tile
  static constexpr int QBytes = 4 * QTerm;               // [row tile][term]
  static constexpr int KBytes = kTile / 2 * kD;          // K codes: this CTA's half of the tokens
  static constexpr int VBytes = kTile * kD / 2;          // V codes: this CTA's half of the values
  static constexpr int WBytes = 2 * VBytes;              // the same in FP16
  static constexpr int KStages = 4, VStages = 3, WStages = 3, Slots = 6, Works = 4;
  static constexpr int Tiles = QBytes + KStages * KBytes + VStages * VBytes + WStages * WBytes;
  static constexpr int OutWarp = 32 * 64 * 2;            // 64 BF16 values of a warp's rows on their way out
  static constexpr int Smem = 1024 + Tiles + 8 * OutWarp + 1024 + Slots * 128 + Works * 64 + kCtaRows * 4;
  // A part of a cut block: a row's values as FP32 without the last 8 bits, four in three words, and the
  // row's maximum and sum.  The join adds in FP32; what is left off, 2^-15 of a part's value, is a 128th of
  // the output's own rounding to BF16.  Whole FP32 values would cost a third more traffic, and 42 instead of 32 MB
  // of workspace at heads of 128.  (FP16 with a scale per row is a 2^-11: seen in single values where large parts
  // cancel.)
  static constexpr int PartWords = kCtaRows * (kD * 3 / 4 + 2);
};

// Per 16 tokens of a tile: K scale x softmax scale x log2 e, log2 V scale, 1 / V scale.
struct PromptSlot {
  float kf[8], lv[8], iv[8];
  float pad[8];
};

struct PromptParams {
  moe_kv_attention_args a;
  PromptPlan plan;
  int G, page_shift;
  uint32_t magic;              // ceil(2^32 / G), 0 for G = 1: row / G is a multiply for row < 2^26
  uint32_t* parts;             // [2 * pairs][CTA of the pair][PartWords]
  int* status;
  bool join;                   // k_prompt_join follows
};

__device__ __forceinline__ int token_of(const PromptParams& p, int row) {
  return p.magic ? (int)__umulhi((uint32_t)row, p.magic) : row;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ------------------------------------------------------------------------------ pairs of CTAs
// Two CTAs of a cluster, on neighbouring SMs, run one product of 256 rows: each holds its 128 rows of A
// and of the result and half of B, so that B, which bounds shared memory's bandwidth when one CTA does it
// alone, is read and laid out once for both.  The leader (rank 0) issues; its peer's warps arrive on the
// leader's barriers, and commits arrive on both CTAs'.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on the leader's barrier at this offset.  What the arrival announces is read by the tensor core
// of the arriving thread's own SM, behind the proxy or tcgen05 fence that came before, not by the
// leader's threads, so the arrival needs no cluster-wide release (which costs 1.4x the whole kernel).
__device__ __forceinline__ void mbar_arrive_leader(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void pair_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(KV_ELECT "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}

__device__ __forceinline__ void pair_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(KV_ELECT "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
               "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}

// Arrive on both CTAs' barrier at this offset when the elected lane's products so far are complete.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
          "r"(bar), "h"((uint16_t)3)
      : "memory");
}

template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int kD>
__global__ void __launch_bounds__(kPromptThreads, 1)
    k_attn_prompt(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ PromptParams p) {
  using C = PromptCfg<kD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const uint32_t sQ = sbase, sK = sQ + C::QBytes, sV = sK + C::KStages * C::KBytes,
                 sW = sV + C::VStages * C::VBytes;
  uint8_t* ctrl = smem + C::Tiles + 8 * C::OutWarp;
  PromptSlot* slots = reinterpret_cast<PromptSlot*>(ctrl + 1024);
  int4* works = reinterpret_cast<int4*>(ctrl + 1024 + C::Slots * 128);
  float* qscales = reinterpret_cast<float*>(ctrl + 1024 + C::Slots * 128 + C::Works * 64);   // [row]
  const uint32_t bar0 = smem_addr(ctrl);
  const int rank = (int)cluster_rank();
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto kempty = [&](int s) { return bar0 + 8u * (8 + s); };
  auto vfull = [&](int s) { return bar0 + 8u * (16 + s); };
  auto vempty = [&](int s) { return bar0 + 8u * (24 + s); };
  auto wempty = [&](int s) { return bar0 + 8u * (32 + s); };
  auto ifull = [&](int s) { return bar0 + 8u * (40 + s); };
  auto iempty = [&](int s) { return bar0 + 8u * (48 + s); };
  auto sfull = [&](int w) { return bar0 + 8u * (56 + w); };
  auto ofull = [&](int w) { return bar0 + 8u * (58 + w); };
  // the leader's: the peer's K has landed, V in FP16, Q and P of both CTAs
  auto kpeer = [&](int s) { return bar0 + 8u * (60 + s); };
  auto wfull = [&](int s) { return bar0 + 8u * (68 + s); };
  auto qfull = [&](int w) { return bar0 + 8u * (76 + w); };
  auto pfull = [&](int w, int half) { return bar0 + 8u * (78 + 2 * w + half); };
  const uint32_t drain = bar0 + 8u * 82;
  auto wkfull = [&](int i) { return bar0 + 8u * (83 + i); };     // pieces of work
  auto wkempty = [&](int i) { return bar0 + 8u * (87 + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * 91);
  static_assert(8 * 91 + 16 <= 1024 && C::KStages <= 8 && C::Slots <= 8, "barriers");
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* k_done = reinterpret_cast<volatile int*>(tmem_slot + 2);
  volatile int* v_done = reinterpret_cast<volatile int*>(tmem_slot + 3);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = p.status;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(kempty(s), 1);
      mbar_init(vfull(s), 1);
      mbar_init(vempty(s), 4);
      mbar_init(wempty(s), 1);
      mbar_init(ifull(s), 1);
      mbar_init(iempty(s), 8);
      mbar_init(kpeer(s), 1);
      mbar_init(wfull(s), 8);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(sfull(w), 1);
      mbar_init(ofull(w), 1);
      mbar_init(qfull(w), 8);
      mbar_init(pfull(w, 0), 8);
      mbar_init(pfull(w, 1), 8);
    }
    for (int i = 0; i < C::Works; ++i) {
      mbar_init(wkfull(i), 1);
      mbar_init(wkempty(i), 13);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *k_done = 0;
    *v_done = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) pair_tmem_alloc(smem_addr(tmem_slot), 512);
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();                  // both CTAs' barriers are there
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();

  // The producer looks the pieces of work up, ahead of everybody, and hands them on: the k-th, for a warp
  // of another role; false when there are no more.
  auto take = [&](int k, PromptWork& w) {
    const int i = k % C::Works;
    const bool ok = mbar_wait_warp(wkfull(i), (k / C::Works) & 1, abort_flag, status);
    const int4 a = works[4 * i], b = works[4 * i + 1], c = works[4 * i + 2];
    w = PromptWork{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z};
    __syncwarp();
    if (lane == 0) mbar_arrive(wkempty(i));
    return ok && w.t1 > 0;
  };

  // Tensor memory: S of row tile w (P in its first half) at 128 w, O at 256 + 128 w.
  if (warp < 4) {
    // One idle warp triggers the join's launch, which waits for this kernel's end all the same (in every warp
    // this costs 2% of a chunk).  Where no join follows, the caller's next kernel would only be in the way.
    regs_down<kRegsIssue>();
    if (warp == 3 && p.join) grid_dep_launch_dependents();
    if (warp == 0) {
      // -------------------------------------------------------------------- producer
      const int npg = kTile >> p.page_shift, P = 1 << p.page_shift;
      // K: this CTA's 64 tokens, in boxes of a page or half of one
      const int krows = min(P, kTile / 2), kboxes = kTile / 2 / krows;
      bool ok = true;
      int it = 0;
      PromptWork w;
      const int pair = blockIdx.x / 2;
      PromptWalk walk;
      walk.start(p.plan, pair, lane);
      for (int k = 0; ok; ++k) {
        const bool have = walk.next(p.a, p.plan, p.G, p.page_shift, pair, w);
        if (!have) w.t1 = 0;
        const int wi = k % C::Works;
        ok = mbar_wait_warp(wkempty(wi), ((k / C::Works) & 1) ^ 1, abort_flag, status);
        if (!ok) break;
        if (lane == 0) {
          works[4 * wi] = make_int4(w.b, w.h, w.row0, w.rows);
          works[4 * wi + 1] = make_int4(w.q0, w.pos0, w.lo, w.hi);
          works[4 * wi + 2] = make_int4(w.t0, w.t1, w.part, 0);
          mbar_arrive(wkfull(wi));
        }
        __syncwarp();
        if (!have) break;
        auto entry = [&](int tile) {
          const int pg = tile * npg + lane;
          if (tile >= w.t1 || lane >= npg || (pg << p.page_shift) >= w.hi ||
              ((pg + 1) << p.page_shift) <= w.lo)
            return -1;
          const int e = p.a.block_table[(size_t)w.b * p.a.max_pages + pg];
          return e < p.a.num_pages ? e : -1;
        };
        auto scale = [&](const float* s, int page) {
          return page >= 0 ? s[(size_t)page * p.a.Hkv + w.h] : 1.0f;
        };
        int page = entry(w.t0), page1 = entry(w.t0 + 1);
        float ks = scale(p.a.k_scale, page), vs = scale(p.a.v_scale, page);
        for (int t = w.t0; t < w.t1; ++t, ++it) {
          const int page2 = entry(t + 2);
          const float ks1 = scale(p.a.k_scale, page1), vs1 = scale(p.a.v_scale, page1);
          const int sk = it % C::KStages, sv = it % C::VStages, si = it % C::Slots;
          if (lane == 0)
            ok = bounded_wait(iempty(si), ((it / C::Slots) & 1) ^ 1, abort_flag, status) &&
                 bounded_wait(kempty(sk), ((it / C::KStages) & 1) ^ 1, abort_flag, status);
          ok = __shfl_sync(~0u, (int)ok, 0);
          if (!ok) break;
          // lane i: box i of K
          const int kpage = __shfl_sync(~0u, page, P == kTile ? 0 : (rank * kboxes + lane) & 31);
          const bool klive = lane < kboxes && kpage >= 0;
          const uint32_t kbytes = __popc(__ballot_sync(~0u, klive)) * krows * kD;
          if (lane == 0) mbar_arrive_expect_tx(kfull(sk), kbytes);
          __syncwarp();
          if (klive)
            tma_load_4d(sK + sk * C::KBytes + lane * krows * kD, &tmK, 0, P == kTile ? rank * krows : 0, w.h,
                        kpage, kfull(sk));
          if (lane == 0) *k_done = it + 1;      // copies issued so far
          // scales of the tile's groups of 16 tokens
          const int src = (lane * 16) >> p.page_shift;
          const float gk = __shfl_sync(~0u, ks, src & 31), gv = __shfl_sync(~0u, vs, src & 31);
          if (lane < 8) {
            slots[si].kf[lane] = gk * p.a.sm_scale * kLog2e;
            const float v = gv >= 0.0f ? fmaxf(gv, 1e-30f) : gv;
            // a K scale that is NaN goes in here: the lower bound on f would hide it
            slots[si].lv[lane] = gk == gk ? log2f(v) : gk;
            slots[si].iv[lane] = 1.0f / v;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(ifull(si));
            ok = bounded_wait(vempty(sv), ((it / C::VStages) & 1) ^ 1, abort_flag, status);
          }
          ok = __shfl_sync(~0u, (int)ok, 0);
          if (!ok) break;
          const uint32_t vbytes = __popc(__ballot_sync(~0u, page >= 0)) * P * (kD / 2);
          if (lane == 0) mbar_arrive_expect_tx(vfull(sv), vbytes);
          __syncwarp();
          if (page >= 0)
            tma_load_4d(sV + sv * C::VBytes + lane * P * (kD / 2), &tmV, rank * (kD / 2), 0, w.h, page, vfull(sv));
          if (lane == 0) *v_done = it + 1;
          page = page1;
          page1 = page2;
          ks = ks1;
          vs = vs1;
        }
      }
    } else if (warp == 1 && rank == 1) {
      // ------------------------------------------------- the peer's K has landed: tell the leader
      bool ok = true;
      int it = 0;
      PromptWork w;
      for (int k = 0; ok && take(k, w); ++k) {
        for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
          ok = mbar_wait_warp(kfull(it % C::KStages), (it / C::KStages) & 1, abort_flag, status);
          if (ok && lane == 0) mbar_arrive_leader(kpeer(it % C::KStages));
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------------- MMA
      constexpr uint32_t kIdescS = make_idesc_e4m3(256, kTile);
      // D fp32, A and B FP16, B MN-major, 256 x kD
      constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(kD >> 3) << 17) | (16u << 24);
      // S of row tile w for tile `tile`
      auto scores = [&](int w, int tile) {
        const uint64_t kd = rows_desc<kD>(sK + tile % C::KStages * C::KBytes);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const uint64_t qd = rows_desc<kD>(sQ + (2 * w + term) * C::QTerm);
#pragma unroll
          for (int k = 0; k < kD / 32; ++k)
            pair_mma_f8(tmem + 128 * w, qd + 2 * k, kd + 2 * k, kIdescS, term + k > 0);
        }
        pair_commit(sfull(w));
        if (w == 1) pair_commit(kempty(tile % C::KStages));
      };
      auto k_ready = [&](int tile) {
        const int s = tile % C::KStages, ph = (tile / C::KStages) & 1;
        return mbar_wait_warp(kfull(s), ph, abort_flag, status) && mbar_wait_warp(kpeer(s), ph, abort_flag, status);
      };
      // P arrives in two halves of the tile's tokens: the product of the first runs while the softmax
      // warps form the second
      auto output = [&](int w, int tile, bool first) {
        const uint64_t vd = rows_desc<kD>(sW + tile % C::WStages * C::WBytes);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait_warp(pfull(w, half), tile & 1, abort_flag, status)) return false;
          tc_fence_after_sync();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            pair_mma_f16_ts(tmem + 256 + 128 * w, tmem + 128 * w + 32 * half + 8 * k, vd + (4 * half + k) * kD,
                            kIdescO, !first || half + k > 0);
        }
        pair_commit(ofull(w));
        if (w == 1) pair_commit(wempty(tile % C::WStages));
        return true;
      };
      auto w_ready = [&](int tile) {
        return mbar_wait_warp(wfull(tile % C::WStages), (tile / C::WStages) & 1, abort_flag, status);
      };
      // One stream of tiles over all pieces: the scores of the next tile are issued behind the products of
      // this one.  Where the next tile begins another piece both products come first, for its Q is some way
      // off: the softmax warps bring it in behind their last probabilities.  All that can be is waited for
      // behind products under way, which hide what a wait costs even when it has nothing to wait for.
      PromptWork w;
      int k = 0, it = -1, t = 0;
      bool first = true, end = true, more = take(0, w), ok = more;
      t = w.t0 - 1;
      while (ok) {
        // tile `it` (none yet: -1), then the scores of tile it + 1, which is the first of piece k if `end`
#pragma unroll 1
        for (int r = 0; ok && r < 2; ++r) {
          if (it >= 0) ok = output(r, it, first);
          if (ok && !end) {
            if (r == 0) ok = k_ready(it + 1);
            if (ok) scores(r, it + 1);
          }
        }
        if (!ok) break;
        if (end) {
          if (it >= 0) {
            more = take(++k, w);
            t = w.t0 - 1;
          }
          if (!more || !k_ready(it + 1)) break;
#pragma unroll 1
          for (int r = 0; ok && r < 2; ++r) {
            ok = mbar_wait_warp(qfull(r), k & 1, abort_flag, status);
            tc_fence_after_sync();
            if (ok) scores(r, it + 1);
          }
        }
        ok = ok && w_ready(it + 1);
        first = end;
        ++it;
        ++t;
        end = t + 1 == w.t1;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------------ V codes -> FP16
    regs_down<kRegsWiden>();
    constexpr int kChunks = kD / 32;         // 16 codes each; rows of kD / 2 codes
    constexpr int kRowsAt = 32 / kChunks;    // rows of a warp's load
    const int c = lane % kChunks, rl = lane / kChunks;
    bool ok = true;
    int it = 0;
    PromptWork w;
    for (int k = 0; ok && take(k, w); ++k) {
      for (int t = w.t0; ok && t < w.t1; ++t, ++it) {
        const int sv = it % C::VStages, sw = it % C::WStages;
        ok = bounded_wait(vfull(sv), (it / C::VStages) & 1, abort_flag, status) &&
             bounded_wait(wempty(sw), ((it / C::WStages) & 1) ^ 1, abort_flag, status);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const uint8_t* in = smem + (sV - sbase) + sv * C::VBytes;
        uint8_t* out = smem + (sW - sbase) + sw * C::WBytes;
        const int token0 = t * kTile;
        const bool edge = token0 < w.lo || token0 + kTile > w.hi;
#pragma unroll 4
        for (int i = 0; i < 32 / kRowsAt; ++i) {
          const int r = (warp & 3) * 32 + i * kRowsAt + rl;
          uint4 x = *reinterpret_cast<const uint4*>(in + r * (kD / 2) + 16 * c);
          // rows that no query row sees may hold anything: 0 x NaN would spread
          if (edge && (token0 + r < w.lo || token0 + r >= w.hi)) x = make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * j]) : "h"((uint16_t)u[j]));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * j + 1]) : "h"((uint16_t)(u[j] >> 16)));
          }
          *reinterpret_cast<uint4*>(out + swz<kD>(r, 32 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(out + swz<kD>(r, 32 * c + 16)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_leader(wfull(sw));
          mbar_arrive(vempty(sv));
        }
      }
    }
  } else {
    // ---------------------------------------------------------------------------- softmax
    regs_up<kRegsSoftmax>();
    const int wg = (warp >> 2) - 2, q = warp & 3;
    const int tr = q * 32 + lane;            // row of the row tile
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128 * wg, tO = tmem + lane_base + 256 + 128 * wg;
    float qs = 0.0f;                         // value of a code of the row's Q

    // Q of the warp's rows: each scaled so that its largest value is in [128, 256), two E4M3 terms.  Eight
    // lanes a row, four rows at a time: whole lines at each load, where a row a lane would touch 32.
    auto load_q = [&](const PromptWork& w) {
      constexpr int kV = kD / 8;             // values of a lane
      const int c = lane & 7;
      uint8_t* o = smem + wg * 2 * C::QTerm;
      // four loads under way at a time (all eight at once cost more in code than they save in waiting)
      const int base = w.row0 + kCtaRows * rank + 128 * wg + 32 * q + (lane >> 3);
      uint4 all[4][kV / 8];
#pragma unroll 1
      for (int n0 = 0; n0 < 8; n0 += 4) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int row = min(base + 4 * (n0 + n), w.rows - 1), i = token_of(p, row);
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(p.a.q) + (int64_t)(w.q0 + i) * p.a.q_token_stride +
              (int64_t)(w.h * p.G + row - i * p.G) * p.a.q_head_stride + c * kV);
#pragma unroll
          for (int v = 0; v < kV / 8; ++v) all[n][v] = __ldg(src + v);
        }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int n = n0 + m, r = 32 * q + 4 * n + (lane >> 3);
        uint4 x[kV / 8];
#pragma unroll
        for (int v = 0; v < kV / 8; ++v) x[v] = base + 4 * n < w.rows ? all[m][v] : make_uint4(0, 0, 0, 0);
        float amax = 0.0f;
#pragma unroll
        for (int v = 0; v < kV / 8; ++v) {
          const uint32_t u[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
        const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
        // (0 where a value is infinite: its code becomes NaN, where a saturated one would make a finite score)
        const float mul = e == 128 ? 0.0f : __uint_as_float((uint32_t)(127 + 7 - e) << 23);
        if (c == 0) qscales[128 * wg + r] = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
#pragma unroll
        for (int v = 0; v < kV / 8; ++v) {
          const uint32_t u[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
          uint32_t t1[2], t2[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float a0 = __uint_as_float(u[2 * j] << 16) * mul, a1 = __uint_as_float(u[2 * j] & 0xFFFF0000u) * mul;
            const float a2 = __uint_as_float(u[2 * j + 1] << 16) * mul,
                        a3 = __uint_as_float(u[2 * j + 1] & 0xFFFF0000u) * mul;
            const uint32_t c0 = cvt_e4m3x2(a0, a1), c1 = cvt_e4m3x2(a2, a3);
            float f0, f1, f2, f3;
            e4m3x2_to_f32(c0, f0, f1);
            e4m3x2_to_f32(c1, f2, f3);
            t1[j] = c0 | (c1 << 16);
            t2[j] = cvt_e4m3x2(a0 - f0, a1 - f1) | (cvt_e4m3x2(a2 - f2, a3 - f3) << 16);
          }
          const uint32_t at = swz<kD>(r, c * kV + 8 * v);
          *reinterpret_cast<uint2*>(o + at) = make_uint2(t1[0], t1[1]);
          *reinterpret_cast<uint2*>(o + C::QTerm + at) = make_uint2(t2[0], t2[1]);
        }
      }
      }
      fence_proxy_async_smem();
      __syncwarp();
      qs = qscales[128 * wg + tr];
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(qfull(wg));
    };

    bool ok = true;
    int it = 0;
    PromptWork w = {};
    bool have = false;               // a piece is under way; the first turn only brings in the first Q
    for (int k = -1; ok; ++k) {
      // tokens that this row sees, and those that every / any row of the tile sees
      const int row = w.row0 + kCtaRows * rank + 128 * wg + tr, tok = have ? token_of(p, row) : 0;
      const bool live = have && row < w.rows;
      const int pos = w.pos0 + tok;
      const int see_lo = p.a.window > 0 ? max(0, pos - p.a.window + 1) : 0, see_hi = live ? pos + 1 : 0;
      const int r_first = w.row0 + kCtaRows * rank + 128 * wg, r_last = min(w.rows, r_first + 128) - 1;
      const int all_hi = have ? w.pos0 + token_of(p, r_first) + 1 : 0;
      const int all_lo = have && p.a.window > 0 ? w.pos0 + token_of(p, max(r_last, 0)) - p.a.window + 1 : 0;
      // where the row goes: the workspace for a piece, else the output
      const bool piece = w.part >= 0;
      uint32_t* const part = p.parts + (size_t)(2 * max(w.part, 0) + rank) * C::PartWords + 128 * wg + tr;
      uint16_t* const out = static_cast<uint16_t*>(p.a.out) + (int64_t)(w.q0 + tok) * p.a.out_token_stride +
                            (int64_t)(w.h * p.G + row - tok * p.G) * p.a.out_head_stride;
      const int t0 = have ? w.t0 : 0, t1 = have ? w.t1 : 0;
      float M = -INFINITY, l = 0.0f;
      for (int t = t0; t < t1; ++t, ++it) {
        const int si = it % C::Slots;
        ok = bounded_wait(ifull(si), (it / C::Slots) & 1, abort_flag, status) &&
             bounded_wait(sfull(wg), it & 1, abort_flag, status);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const PromptSlot& slot = slots[si];
        const int token0 = t * kTile;
        const bool edge = token0 + kTile > all_hi || token0 < all_lo;
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
        tmem_ld_wait();
        auto x = [&](int i) { return __uint_as_float(s[i]); };
        // x f + lv is the score plus log2 of the V scale, in log2 units, with f and lv per 16 tokens.  (They
        // are read again for the probabilities: sixteen registers less in between.)  Masked scores are -inf;
        // f is kept above zero so that they stay so.
        if (edge) {
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            const int lo = min(max(see_lo - token0 - c, 0), 32), hi = min(max(see_hi - token0 - c, 0), 32);
            // bits [lo, hi)
            const uint32_t seen = hi > lo ? (0xFFFFFFFFu >> (32 - (hi - lo))) << lo : 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((seen >> i) & 1)) s[c + i] = __float_as_uint(-INFINITY);
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          float m = max3(x(16 * g), x(16 * g + 1), x(16 * g + 2));
          float m2 = max3(x(16 * g + 3), x(16 * g + 4), x(16 * g + 5));
#pragma unroll
          for (int i = 16 * g + 6; i < 16 * g + 14; i += 4) {
            m = max3(m, x(i), x(i + 1));
            m2 = max3(m2, x(i + 2), x(i + 3));
          }
          m = fmaxf(max3(m, x(16 * g + 14), x(16 * g + 15)), m2);
          top = fmaxf(top, __fmaf_rn(m, fmaxf(slot.kf[g] * qs, 1.2e-38f), slot.lv[g]));
        }
        if (__any_sync(~0u, top > M + kPromptGrow)) {
          const float mn = fmaxf(M, top);
          const float alpha = M == mn ? 1.0f : exp2_approx(M - mn);
          if (t > t0) {
            // O so far is relative to the old maximum
            ok = bounded_wait(ofull(wg), (it - 1) & 1, abort_flag, status);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + c, o);
            }
            tmem_st_wait();
          }
          l *= alpha;
          M = mn;
        }
        const volatile PromptSlot* vslot = &slot;
        const float base = kPromptBias - (M == -INFINITY ? 0.0f : M);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int g = 4 * half; g < 4 * half + 4; ++g) {
            const float fg = fmaxf(vslot->kf[g] * qs, 1.2e-38f), ag = vslot->lv[g] + base;
            const f32x2 f2 = pack2(fg, fg), add = pack2(ag, ag);
            f32x2 sum = 0ull;
#pragma unroll
            for (int i = 16 * g; i < 16 * g + 16; i += 2) {
              float p0, p1;
              unpack2(fma2(pack2(x(i), x(i + 1)), f2, add), p0, p1);
              p0 = exp2_approx(p0);
              p1 = exp2_approx(p1);
              sum = add2(sum, pack2(p0, p1));
              s[i / 2] = pack_f16x2(p0, p1);
            }
            float s0, s1;
            unpack2(sum, s0, s1);
            l = __fmaf_rn(s0 + s1, vslot->iv[g], l);
          }
          tmem_st32(tS + 32 * half, s + 32 * half);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (half == 1) mbar_arrive(iempty(si));
            mbar_arrive_leader(pfull(wg, half));
          }
        }
      }
      if (!ok) break;
      // the next piece's Q goes in while the last P V runs
      const bool had = have;
      have = take(k + 1, w);
      if (have) load_q(w);
      if (!had) {
        if (!have) break;
        continue;
      }
      ok = bounded_wait(ofull(wg), (it - 1) & 1, abort_flag, status);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      tc_fence_after_sync();
      if (piece) {
#pragma unroll 1
        for (int c = 0; c < kD; c += 16) {
          uint32_t v[16];
          tmem_ld16(tO + c, v);
          tmem_ld_wait();
          uint32_t* to = part + c * 3 / 4 * kCtaRows;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            // byte 3, 2 and 1 of the fourth value take the others' byte 0
            to[(i * 3 / 4) * kCtaRows] = __byte_perm(v[i], v[i + 3], 0x3217);
            to[(i * 3 / 4 + 1) * kCtaRows] = __byte_perm(v[i + 1], v[i + 3], 0x3216);
            to[(i * 3 / 4 + 2) * kCtaRows] = __byte_perm(v[i + 2], v[i + 3], 0x3215);
          }
        }
        part[kD * 3 / 4 * kCtaRows] = __float_as_uint(M);
        part[(kD * 3 / 4 + 1) * kCtaRows] = __float_as_uint(l);
      } else {
        // 64 values at a time through shared memory, so that the stores cover whole lines of a row
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        uint8_t* stage = smem + C::Tiles + (4 * wg + q) * C::OutWarp;
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += 64) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t v[32];
            tmem_ld32(tO + c0 + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t r[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float a = __uint_as_float(v[8 * j + 2 * h]), b = __uint_as_float(v[8 * j + 2 * h + 1]);
                // a row that saw nothing may have met anything in O
                r[h] = inv != 0.0f ? pack_bf16x2(a * inv, b * inv) : 0u;
              }
              *reinterpret_cast<uint4*>(stage + swz<128>(lane, 2 * c + 16 * j)) = make_uint4(r[0], r[1], r[2], r[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int r4 = 0; r4 < 32; r4 += 4) {
            const int r = r4 + (lane >> 3);
            const unsigned long long to = __shfl_sync(~0u, live ? (unsigned long long)out : 0ull, r);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + swz<128>(r, 16 * (lane & 7)));
            if (to != 0) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(to) + c0 + 8 * (lane & 7)) = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before_sync();
      if (!have) break;
    }
  }

  // ------------------------------------------------------------------------ teardown
  __syncthreads();
  auto drain_wait = [&](uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicCAS(status, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
        return;
      }
    }
  };
  if (warp == 1 && rank == 0) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(drain)
        : "memory");
    drain_wait(drain, 0);
  }
  if (warp == 0 && lane == 0 && *abort_flag) {
    // copies still in flight: the latest use of each stage
    for (int i = max(0, *k_done - C::KStages); i < *k_done; ++i)
      drain_wait(kfull(i % C::KStages), (i / C::KStages) & 1);
    for (int i = max(0, *v_done - C::VStages); i < *v_done; ++i)
      drain_wait(vfull(i % C::VStages), (i / C::VStages) & 1);
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();                  // the leader's products no longer use the peer's memory
  if (warp == 1) {
    tc_fence_after_sync();
    pair_tmem_dealloc(tmem, 512);
  }
}

// Adds the parts of the items that were cut.  blockIdx.x: item of the last round, blockIdx.y:
// 16 values, blockIdx.z: CTA of the pair; thread = row.
template <int kD>
__global__ void __launch_bounds__(kCtaRows) k_prompt_join(const PromptParams p) {
  using C = PromptCfg<kD>;
  grid_dep_wait();
  const PromptTail& tail = *p.plan.tail;
  if (!tail.pour || blockIdx.x >= tail.rest) return;
  const long long item = (long long)tail.rounds * p.plan.pairs + blockIdx.x;
  const int4 e = p.plan.list[item / p.a.Hkv];
  const int h = (int)(item % p.a.Hkv);
  // the parts' places in the order of the pairs: the first one is its pair's last piece
  __shared__ int places[kPromptPairs], count;
  if (threadIdx.x < 32) {
    const int at = tail.start[blockIdx.x] + kItemStart;
    int n = 0;
#pragma unroll
    for (int i = 0; i < (kPromptPairs + 31) / 32; ++i) {
      const int c = 32 * i + threadIdx.x;
      const bool here =
          c < p.plan.pairs && prompt_cut(tail.bound[c] - at, e.z) < prompt_cut(tail.bound[c + 1] - at, e.z);
      const uint32_t mask = __ballot_sync(~0u, here);
      const int k = n + __popc(mask & ((1u << threadIdx.x) - 1));
      if (here) places[k] = 2 * (2 * c + (k == 0 ? 1 : 0)) + blockIdx.z;
      n += __popc(mask);
    }
    if (threadIdx.x == 0) count = n;
  }
  __syncthreads();
  if (count == 1) return;
  PromptWork w;
  prompt_block(p.a, p.G, p.page_shift, e.x, e.y, w);
  const int row = w.row0 + kCtaRows * blockIdx.z + threadIdx.x;
  if (row >= w.rows) return;
  auto part = [&](int i) { return p.parts + (size_t)places[i] * C::PartWords + threadIdx.x; };
  float M = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < count; ++i) M = fmaxf(M, __uint_as_float(part(i)[kD * 3 / 4 * kCtaRows]));
  float l = 0.0f, acc[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
  const int c0 = blockIdx.y * 16;
#pragma unroll 2
  for (int i = 0; i < count; ++i) {
    const uint32_t* o = part(i);
    const float m = __uint_as_float(o[kD * 3 / 4 * kCtaRows]), lp = __uint_as_float(o[(kD * 3 / 4 + 1) * kCtaRows]);
    uint32_t x[12];
#pragma unroll
    for (int j = 0; j < 12; ++j) x[j] = o[(c0 * 3 / 4 + j) * kCtaRows];
    // a part whose tokens this row does not see has an empty sum; one that holds nothing but NaN has no maximum either
    if (m == -INFINITY && lp == lp) continue;
    const float wgt = m == M ? 1.0f : exp2_approx(m - M);
    l = __fmaf_rn(lp, wgt, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* y = x + 3 * j;
      const uint32_t last = ((y[0] & 0xFF) << 24) | ((y[1] & 0xFF) << 16) | ((y[2] & 0xFF) << 8);
#pragma unroll
      for (int k = 0; k < 3; ++k) acc[4 * j + k] = __fmaf_rn(__uint_as_float(y[k] & ~0xFFu), wgt, acc[4 * j + k]);
      acc[4 * j + 3] = __fmaf_rn(__uint_as_float(last), wgt, acc[4 * j + 3]);
    }
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  const int i = row / p.G;
  uint16_t* out = static_cast<uint16_t*>(p.a.out) + (int64_t)(w.q0 + i) * p.a.out_token_stride +
                  (int64_t)(h * p.G + row - i * p.G) * p.a.out_head_stride + c0;
#pragma unroll
  for (int j = 0; j < 16; j += 8) {
    uint4 r;
    r.x = pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
    r.y = pack_bf16x2(acc[j + 2] * inv, acc[j + 3] * inv);
    r.z = pack_bf16x2(acc[j + 4] * inv, acc[j + 5] * inv);
    r.w = pack_bf16x2(acc[j + 6] * inv, acc[j + 7] * inv);
    *reinterpret_cast<uint4*>(out + j) = r;
  }
}

// ------------------------------------------------------------------------------------ launch
bool prompt_fits(int T, int G, int B) {
  return (long long)T * G / kBlockRows + B <= kMaxBlocks;
}

size_t prompt_plan_bytes() { return kPlanBytes; }

size_t prompt_parts_bytes(int D) { return (size_t)2 * kPromptCtas * kCtaRows * (D * 3 / 4 + 2) * 4; }

template <int kD>
static cudaError_t launch_prompt(const moe_kv_attention_args& a, int* status, void* plan, void* parts,
                                 cudaStream_t s) {
  using C = PromptCfg<kD>;
  CUtensorMap tmK, tmV;
  // K: boxes of at most 64 tokens; V: boxes of half a head's values, unswizzled
  if (!cache_map(&tmK, a.k_codes, kD, a.page_size, a.Hkv, a.num_pages, std::min(a.page_size, kTile / 2), kD) ||
      !cache_map(&tmV, a.v_codes, kD, a.page_size, a.Hkv, a.num_pages, a.page_size, kD / 2))
    return cudaErrorInvalidValue;
  cudaError_t err = cudaFuncSetAttribute(k_attn_prompt<kD>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem);
  if (err != cudaSuccess) return err;
  PromptParams p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  p.magic = p.G == 1 ? 0 : (uint32_t)(((1ull << 32) + p.G - 1) / p.G);
  p.plan = prompt_plan_at(plan);
  p.parts = static_cast<uint32_t*>(parts);
  p.status = status;
  const int pairs = p.plan.pairs;
  // nothing is cut where no block can see enough tiles: one launch less (3 x 104 tokens: 15.6 -> 13.8 us)
  long long tiles = ((long long)a.max_pages * a.page_size + kTile - 1) / kTile;
  if (a.window > 0) tiles = std::min(tiles, ((long long)a.window + kBlockRows / p.G + 1) / kTile + 2);
  p.join = tiles >= kCutTiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kPromptThreads);
  cfg.dynamicSmemBytes = C::Smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, k_attn_prompt<kD>, tmK, tmV, p);
  if (err != cudaSuccess) return err;
  if (!p.join) return cudaSuccess;
  return launch_pdl(k_prompt_join<kD>, dim3(pairs, kD / 16, 2), dim3(kCtaRows), 0, s, p);
}

cudaError_t launch_attn_prompt(const moe_kv_attention_args& a, int* status, void* plan, void* parts,
                               cudaStream_t s) {
  return a.D == 128 ? launch_prompt<128>(a, status, plan, parts, s) : launch_prompt<64>(a, status, plan, parts, s);
}

}  // namespace moe
