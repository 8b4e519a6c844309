// What the attention kernels over the paged 8-bit cache share: tiles of 128 tokens, their tensor map and
// shared-memory layouts, and conversions.
#pragma once

#include "kv_internal.h"
#include "moe_device.cuh"

namespace moe {

constexpr int kTile = kTileTokens;         // tokens per tile
constexpr int kMaxTilePages = 8;           // pages of a tile, at page size 16
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void e4m3x2_to_f32(uint32_t codes, float& lo, float& hi) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)codes));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h2));
}

// Pairs of fp32 values in one 64-bit register, worked on by one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The issuing warp stays converged and one elected lane issues: the descriptors then stay in uniform
// registers.  Issued from a branch that only one lane takes, every product costs 110 to 170 cycles of
// moves, more than the 65 that a 128 x 128 one takes to execute.  (elect.sync names the same lane every
// time, so that lane's commits cover its products.)
#define KV_ELECT "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t@e "

// D[tmem] (+)= A[smem] * B[smem]: E4M3, fp32 sums.
__device__ __forceinline__ void mma_f8_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(KV_ELECT "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
               : "memory");
}

// Arrive on `bar` when the elected lane's products so far are complete.
__device__ __forceinline__ void mma_commit_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Bounded wait for the phase of `bar` with the given parity, as mbar_wait, in few instructions: the kernels
// wait in some forty places, and code that outgrows the instruction cache is fetched at every turn.  (A
// try_wait suspends the thread for a while by itself, so the checks between two cost nothing.)
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicCAS(status, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Whether any of the kThreads threads at the barrier says so.
template <int kThreads>
__device__ __forceinline__ bool vote_any(int barrier, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(barrier), "n"(kThreads)
      : "memory");
  return r != 0;
}

// A wait of the whole warp; the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               int* status) {
  return __all_sync(~0u, bounded_wait(bar, parity, abort_flag, status));
}

// Offset of byte x of row r in K-major rows of kRow bytes with the 128- or 64-byte swizzle.
template <int kRow>
__device__ __forceinline__ uint32_t swz(int r, int x) {
  const int key = kRow == 128 ? (r & 7) : ((r >> 1) & 3);
  return (uint32_t)(r * kRow + ((((x >> 4) ^ key) << 4) | (x & 15)));
}

// Descriptor of rows of kRow bytes (128- or 64-byte swizzle), 8-row groups one after another.  For the
// MN-major V tile the 8-row groups follow along the reduction axis at the same offset.
template <int kRow>
__device__ __forceinline__ uint64_t rows_desc(uint32_t saddr) {
  uint64_t d = make_sdesc_sw128(saddr, 8 * kRow);
  if (kRow == 64) d = (d & ~((uint64_t)7 << 61)) | ((uint64_t)4 << 61);
  return d;
}

// The cache's codes as (value, row of the page, head, page); a box is box_rows rows of one page and head
// and box_d of its values, laid out in rows of box_d bytes: with the swizzle of that width when it is a
// whole head, else as they come.
inline bool cache_map(CUtensorMap* m, const void* codes, int D, int P, int Hkv, int pages, int box_rows, int box_d) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)Hkv, (cuuint64_t)pages};
  const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)P * D, (cuuint64_t)Hkv * P * D};
  const cuuint32_t box[4] = {(cuuint32_t)box_d, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_d < D ? CU_TENSOR_MAP_SWIZZLE_NONE
                      : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
