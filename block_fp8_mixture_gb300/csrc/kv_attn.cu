// Attention over the 8-bit paged cache, first form: one warp per (query token, head) walks the visible
// tokens with a running maximum and sum; a lane holds D / 32 values of q and of the output.
#include "kv_internal.h"
#include "moe_device.cuh"

namespace moe {

template <int kD>
__global__ void __launch_bounds__(128) k_attn_simple(const moe_kv_attention_args a, int min_n) {
  constexpr int kV = kD / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(row / a.Hq), h = (int)(row - (long long)t * a.Hq);
  if (t >= a.T || t >= a.tok_start[a.B]) return;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.tok_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int b = lo, n = a.tok_start[b + 1] - a.tok_start[b];
  if (n <= min_n) return;
  const int pos = a.kv_len[b] - n + t - a.tok_start[b];
  const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int hk = h / (a.Hq / a.Hkv);
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_token_stride + h * a.q_head_stride;
  float qv[kV], acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    qv[i] = bf16_bits_to_f32(q[lane * kV + i]);
    acc[i] = 0.0f;
  }
  auto value = [](uint8_t c) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h2));
    return f;
  };
  float m = -INFINITY, l = 0.0f;
  for (int j = first; j <= pos; ++j) {
    const int page = a.block_table[(size_t)b * a.max_pages + j / a.page_size];
    if (page < 0 || page >= a.num_pages) continue;
    const size_t blk = (size_t)page * a.Hkv + hk;
    const size_t at = (blk * a.page_size + j % a.page_size) * kD + lane * kV;
    const uint8_t* kc = static_cast<const uint8_t*>(a.k_codes) + at;
    const uint8_t* vc = static_cast<const uint8_t*>(a.v_codes) + at;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) s = __fmaf_rn(qv[i], value(kc[i]), s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.k_scale[blk] * a.sm_scale;
    const float mn = fmaxf(m, s);
    const float alpha = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = __fmaf_rn(l, alpha, p);
    const float pv = p * a.v_scale[blk];
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = __fmaf_rn(acc[i], alpha, pv * value(vc[i]));
  }
  uint16_t* o =
      static_cast<uint16_t*>(a.out) + t * a.out_token_stride + h * a.out_head_stride + lane * kV;
#pragma unroll
  for (int i = 0; i < kV; ++i) o[i] = (uint16_t)f32_to_bf16_bits(l > 0.0f ? acc[i] / l : 0.0f);
}

cudaError_t launch_attn_simple(const moe_kv_attention_args& a, int min_n, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)a.T * a.Hq + 3) / 4);
  if (grid == 0) return cudaSuccess;
  if (a.D == 128) k_attn_simple<128><<<grid, 128, 0, s>>>(a, min_n);
  else k_attn_simple<64><<<grid, 128, 0, s>>>(a, min_n);
  return cudaGetLastError();
}

}  // namespace moe
