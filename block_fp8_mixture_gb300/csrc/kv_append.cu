// Rotary positions and the write of K and V into the 8-bit paged cache, one launch.
//
// A scale covers one (page, head) block, so the unit of the cache write is a run: the new tokens of
// one request that share a page.  A unit (run, head, K or V) keeps its rotated values in registers
// (16 values of a row per thread, at most 4 rows per thread), reduces their amax, forms the block's
// scale and quantizes, so K and V are read once.  Where the block already holds older tokens under a
// smaller scale, their codes are rescaled in place.  A unit takes page_size * D / 64 threads (a
// quarter of the page's rows at a time), 1 to 8 warps; four warps make a block, more for one unit of
// eight warps, so small pages pack several units into a block.  The remaining blocks rotate Q, 16
// values per thread: a chunk of 8 pairs (HALF: 8 values and the 8 at rot/2 from them), so that every
// cos/sin is loaded once per thread.  Bound by HBM: Q in and out, K and V in at 2 bytes, codes out.
#include "kv_device.cuh"

namespace moe {

struct Pairs {
  float x[16];
};

// 16 BF16 values as two 16-byte loads.
__device__ __forceinline__ Pairs load_pairs(const uint16_t* lo, const uint16_t* hi) {
  const uint4 a = *reinterpret_cast<const uint4*>(lo), b = *reinterpret_cast<const uint4*>(hi);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  Pairs r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.x[2 * i] = __uint_as_float(w[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

// Where chunk c (16 values) of a head lies: values [lo, lo + 8) and [hi, hi + 8), and the first of
// its 8 pairs (-1: not rotated).
struct Chunk16 {
  int lo, hi, pair;
};

__device__ __forceinline__ Chunk16 chunk16(int c, int rot, int layout) {
  const int rc = rot >> 4;
  if (c >= rc) return Chunk16{16 * c, 16 * c + 8, -1};
  if (layout == MOE_ROPE_INTERLEAVED) return Chunk16{16 * c, 16 * c + 8, 8 * c};
  return Chunk16{8 * c, 8 * c + (rot >> 1), 8 * c};
}

// x'_a = x_a cos - x_b sin, x'_b = x_b cos + x_a sin, products and sums rounded separately.
__device__ __forceinline__ void rotate_pair(float& xa, float& xb, float c, float s) {
  const float a = xa, b = xb;
  xa = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  xb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ void rotate(Pairs& v, const float (&cs)[16], int layout) {
  if (layout == MOE_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(v.x[2 * i], v.x[2 * i + 1], cs[2 * i], cs[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(v.x[i], v.x[i + 8], cs[2 * i], cs[2 * i + 1]);
  }
}

__device__ __forceinline__ void load_cs(float (&cs)[16], const float* rope, int pos, int rot, int pair) {
  const float4* p = reinterpret_cast<const float4*>(rope + (size_t)pos * rot + 2 * pair);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = p[i];
    cs[4 * i] = t.x;
    cs[4 * i + 1] = t.y;
    cs[4 * i + 2] = t.z;
    cs[4 * i + 3] = t.w;
  }
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}

// Four E4M3 codes times r, rounded back to E4M3.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  float f[4];
  e4m3x2_to_f32(w, f[0], f[1]);
  e4m3x2_to_f32(w >> 16, f[2], f[3]);
  return codes4(__fmul_rn(f[0], r), __fmul_rn(f[1], r), __fmul_rn(f[2], r), __fmul_rn(f[3], r));
}

// kWPU warps per unit.
template <int kWPU>
__global__ void __launch_bounds__(kWPU == 8 ? 256 : 128)
    k_rope_append(const moe_rope_append_args a, int kv_blocks) {
  constexpr int kThreads = kWPU == 8 ? 256 : 128;
  constexpr int kUnits = kThreads / (32 * kWPU);
  const int chunks = a.D >> 4;                 // threads per row: 4 or 8
  const int cshift = a.D == 128 ? 3 : 2;

  if ((int)blockIdx.x >= kv_blocks) {          // ---------------------------------- Q
    const long long x = (long long)(blockIdx.x - kv_blocks) * kThreads + threadIdx.x;
    const int c = (int)(x & (chunks - 1));
    const long long th = x >> cshift;
    const int t = (int)(th / a.Hq), h = (int)(th - (long long)t * a.Hq);
    if (t >= a.T) return;
    const Chunk16 ch = chunk16(c, a.rot_dim, a.layout);
    const uint16_t* q =
        static_cast<const uint16_t*>(a.q) + t * a.q_token_stride + h * a.q_head_stride;
    uint16_t* o = static_cast<uint16_t*>(a.q_out) + t * a.qo_token_stride + h * a.qo_head_stride;
    Pairs v = load_pairs(q + ch.lo, q + ch.hi);
    if (ch.pair >= 0) {
      float cs[16];
      load_cs(cs, a.rope, min(max(a.position[t], 0), a.max_pos - 1), a.rot_dim, ch.pair);
      rotate(v, cs, a.layout);
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v.x[2 * i], v.x[2 * i + 1]);
    *reinterpret_cast<uint4*>(o + ch.lo) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(o + ch.hi) = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }

  // -------------------------------------------------------------------------------- K, V
  __shared__ float red[kThreads / 32];
  const int warp = threadIdx.x >> 5;
  const int ut = threadIdx.x & (32 * kWPU - 1);          // thread within the unit
  const long long unit = (long long)blockIdx.x * kUnits + warp / kWPU;
  const int hv = (int)(unit % (2 * a.Hkv));              // head and K / V
  const long long run = unit / (2 * a.Hkv);
  // whole units leave together, so the barriers below stay complete
  if (run >= a.max_runs) return;
  const int n = min(a.run_len[run], a.page_size);
  const int tok0 = a.run_tok[run];
  if (n <= 0 || tok0 < 0 || tok0 + n > a.T) return;
  const int slot = a.slot[tok0];
  const int page = slot < 0 ? -1 : slot / a.page_size;
  if (page < 0 || page >= a.num_pages) return;
  const int off = slot - page * a.page_size;
  if (off + n > a.page_size) return;
  const int h = hv >> 1, is_v = hv & 1;
  const int c = ut & (chunks - 1), r0 = ut >> cshift, rows = (32 * kWPU) >> cshift;
  const Chunk16 ch = chunk16(c, is_v ? 0 : a.rot_dim, a.layout);
  const uint16_t* src = is_v ? static_cast<const uint16_t*>(a.v) + h * a.v_head_stride
                             : static_cast<const uint16_t*>(a.k) + h * a.k_head_stride;
  const int64_t ts = is_v ? a.v_token_stride : a.k_token_stride;
  float* scale = (is_v ? a.v_scale : a.k_scale) + (size_t)page * a.Hkv + h;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_codes : a.k_codes) +
                   ((size_t)page * a.Hkv + h) * a.page_size * a.D;
  const float was = *scale;

  Pairs v[4];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i * rows;
    if (r < n) {
      const uint16_t* x = src + (tok0 + r) * ts;
      v[i] = load_pairs(x + ch.lo, x + ch.hi);
      if (ch.pair >= 0) {
        float cs[16];
        load_cs(cs, a.rope, min(max(a.position[tok0 + r], 0), a.max_pos - 1), a.rot_dim, ch.pair);
        rotate(v[i], cs, a.layout);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(v[i].x[j]));
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
  if (kWPU > 1) {
    if ((threadIdx.x & 31) == 0) red[warp] = amax;
    named_barrier_sync(1 + warp / kWPU, 32 * kWPU);
    const int w0 = warp / kWPU * kWPU;
#pragma unroll
    for (int w = 0; w < kWPU; ++w) amax = fmaxf(amax, red[w0 + w]);
  }
  // every thread has read the old scale before the barrier (one warp: before the shuffles)
  float s = group_scale(amax, a.scale_fmt);
  if (off > 0) s = fmaxf(s, was);
  if (ut == 0) *scale = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i * rows;
    if (r < n) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = codes4(__fdiv_rn(v[i].x[4 * j], s), __fdiv_rn(v[i].x[4 * j + 1], s),
                      __fdiv_rn(v[i].x[4 * j + 2], s), __fdiv_rn(v[i].x[4 * j + 3], s));
      uint8_t* o = codes + (size_t)(off + r) * a.D;
      *reinterpret_cast<uint2*>(o + ch.lo) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(o + ch.hi) = make_uint2(w[2], w[3]);
    }
  }
  if (off > 0 && s > was) {
    const float ratio = __fdiv_rn(was, s);
    for (int r = r0; r < off; r += rows) {
      uint4* o = reinterpret_cast<uint4*>(codes + (size_t)r * a.D + 16 * c);
      uint4 w = *o;
      w.x = rescale4(w.x, ratio);
      w.y = rescale4(w.y, ratio);
      w.z = rescale4(w.z, ratio);
      w.w = rescale4(w.w, ratio);
      *o = w;
    }
  }
}

cudaError_t launch_rope_append(const moe_rope_append_args& a, cudaStream_t s) {
  const int wpu = a.page_size * a.D / 64 <= 32 ? 1 : a.page_size * a.D / 64 / 32;
  const int threads = wpu == 8 ? 256 : 128, units = threads / (32 * wpu);
  const long long kv = ((long long)a.max_runs * 2 * a.Hkv + units - 1) / units;
  const long long q = ((long long)a.T * a.Hq * (a.D / 16) + threads - 1) / threads;
  if (kv + q == 0) return cudaSuccess;
  if (kv + q > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(kv + q);
  switch (wpu) {
    case 1: k_rope_append<1><<<grid, threads, 0, s>>>(a, (int)kv); break;
    case 2: k_rope_append<2><<<grid, threads, 0, s>>>(a, (int)kv); break;
    case 4: k_rope_append<4><<<grid, threads, 0, s>>>(a, (int)kv); break;
    default: k_rope_append<8><<<grid, threads, 0, s>>>(a, (int)kv); break;
  }
  return cudaGetLastError();
}

// -------------------------------------------------------------------------- the table of cos and sin
__global__ void k_rope_table(float2* table, int max_pos, int half, double log2_base, int scaling,
                             double factor, double low, double high, double original_len,
                             float magnitude) {
  const long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (x >= (long long)max_pos * half) return;
  const int pos = (int)(x / half), i = (int)(x - (long long)pos * half);
  double f = exp2(-log2_base * i / half);
  if (scaling == MOE_ROPE_SCALE_LINEAR) f = f / factor;
  if (scaling == MOE_ROPE_SCALE_RAMP) {
    const double turns = original_len * f / 6.283185307179586476925;
    const double w = fmin(fmax((turns - low) / (high - low), 0.0), 1.0);
    f = f * (w + (1.0 - w) / factor);
  }
  double sn, cn;
  sincos(pos * f, &sn, &cn);
  table[x] = make_float2((float)(cn * magnitude), (float)(sn * magnitude));
}

cudaError_t launch_rope_table(float* table, int max_pos, int rot, double base, int scaling,
                              double factor, double low, double high, int original_len,
                              float magnitude, cudaStream_t s) {
  const long long n = (long long)max_pos * (rot / 2);
  if (n == 0) return cudaSuccess;
  k_rope_table<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(
      reinterpret_cast<float2*>(table), max_pos, rot / 2, log2(base), scaling, factor, low, high,
      original_len, magnitude);
  return cudaGetLastError();
}

}  // namespace moe
