// Rotary positions and the write of K and V into the 8-bit paged cache, one launch.
//
// A scale covers one (page, head) block, so the unit of the cache write is a run: the new tokens of
// one request that share a page.  A unit (run, head, K or V) loads its rows (16 values of a row per
// thread, up to four rows), rotates them and reduces their amax, forms the block's scale, then rotates
// once more and quantizes: keeping the BF16 rows costs half the registers of keeping rotated ones, and
// the loads' latency, which bounds the kernel, needs the warps.  Where the block already holds older
// tokens under a smaller scale, their codes are rescaled in place.  In a step of single tokens a unit is
// one warp, in prompts the warps that hold a page; four warps or more make a block.  The remaining blocks
// rotate Q, a token each: a thread holds the cos and sin of 8 pairs (HALF: 8 values and the 8 at rot/2
// from them) and applies them to every head it has.
// Prompts of 8331 tokens, 32 + 2 x 8 heads of 128: 40.7 us as a graph (43.0 back to back from Python), 4.7 TB/s,
// 70% of the measured copy rate (rotated rows kept: 53 us; eight rows a thread: 63 us).  32 single tokens: 3.2 us,
// 253: 7.1 us, latency.
#include <algorithm>

#include "kv_device.cuh"

namespace moe {

constexpr int kRows = 4;      // rows of a cache unit that a thread keeps, as BF16

struct Pairs {
  float x[16];
};

// 16 BF16 values as two 16-byte loads, and their values.  Loads come first and values when they are
// needed: a warp issues in order, so a load behind a wait would wait too.
struct Raw16 {
  uint4 lo, hi;
};
__device__ __forceinline__ Raw16 load_raw(const uint16_t* lo, const uint16_t* hi) {
  return Raw16{*reinterpret_cast<const uint4*>(lo), *reinterpret_cast<const uint4*>(hi)};
}
__device__ __forceinline__ Pairs values(const Raw16& w) {
  const uint32_t u[8] = {w.lo.x, w.lo.y, w.lo.z, w.lo.w, w.hi.x, w.hi.y, w.hi.z, w.hi.w};
  Pairs r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.x[2 * i] = __uint_as_float(u[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
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

  // the cache's blocks come first: they wait for chains of loads and finish last
  const bool is_kv = blockIdx.x < (unsigned)kv_blocks;
  if (!is_kv) {                                // ---------------------------------- Q
    // a block takes one token: its cos and sin are loaded once for all heads of a thread
    const int t = blockIdx.x - kv_blocks, c = threadIdx.x & (chunks - 1);
    const Chunk16 ch = chunk16(c, a.rot_dim, a.layout);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_token_stride;
    uint16_t* o = static_cast<uint16_t*>(a.q_out) + t * a.qo_token_stride;
    constexpr int kRound = 2;                  // heads of a thread under way at once
    const int step = kThreads >> cshift;
    float cs[16];
    bool have_cs = false;
    for (int h0 = threadIdx.x >> cshift; h0 < a.Hq; h0 += kRound * step) {
      Raw16 raw[kRound];
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int h = min(h0 + i * step, a.Hq - 1);
        raw[i] = load_raw(q + h * a.q_head_stride + ch.lo, q + h * a.q_head_stride + ch.hi);
      }
      if (!have_cs && ch.pair >= 0)
        load_cs(cs, a.rope, min(max(a.position[t], 0), a.max_pos - 1), a.rot_dim, ch.pair);
      have_cs = true;
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int h = h0 + i * step;
        if (h >= a.Hq) break;
        Pairs v = values(raw[i]);
        if (ch.pair >= 0) rotate(v, cs, a.layout);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(v.x[2 * j], v.x[2 * j + 1]);
        uint16_t* out = o + h * a.qo_head_stride;
        *reinterpret_cast<uint4*>(out + ch.lo) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(out + ch.hi) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    return;
  }

  // -------------------------------------------------------------------------------- K, V
  __shared__ float red[kThreads / 32];
  const int warp = threadIdx.x >> 5;
  const int ut = threadIdx.x & (32 * kWPU - 1);          // thread within the unit
  const unsigned unit = blockIdx.x * kUnits + warp / kWPU;
  const unsigned run = unit / (2 * a.Hkv);
  const int hv = (int)(unit - run * 2 * a.Hkv);          // head and K / V
  // whole units leave together, so the barriers below stay complete
  if (run >= (unsigned)a.max_runs) return;
  const int n = min(a.run_len[run], a.page_size);
  const int tok0 = a.run_tok[run];
  if (n <= 0 || tok0 < 0 || tok0 > a.T - n) return;
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

  auto raw_row = [&](int r) {
    const uint16_t* x = src + (tok0 + r) * ts;
    return load_raw(x + ch.lo, x + ch.hi);
  };
  auto row = [&](const Raw16& raw, int r) {
    Pairs v = values(raw);
    if (ch.pair >= 0) {
      float cs[16];
      load_cs(cs, a.rope, min(max(a.position[tok0 + r], 0), a.max_pos - 1), a.rot_dim, ch.pair);
      rotate(v, cs, a.layout);
    }
    return v;
  };
  Raw16 raw[kRows];
  float amax = 0.0f;
  auto widen = [&](const Pairs& x) {
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x.x[j]));
  };
#pragma unroll
  for (int i = 0; i < kRows; ++i) raw[i] = raw_row(min(r0 + i * rows, n - 1));
  const float was = *scale;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (r0 + i * rows < n) widen(row(raw[i], r0 + i * rows));
  if (kWPU == 1)                               // more warps hold the whole page
    for (int r = r0 + kRows * rows; r < n; r += rows) widen(row(raw_row(r), r));
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
  // x / s rounded once: two corrections of x (1/s) by the exact remainder (Markstein), for finite s.  The remainder
  // is taken with the sign turned, q s - x: so a negative zero stays one.
  const bool finite = s <= 3.4e38f;
  const float inv = finite ? __frcp_rn(s) : 0.0f;
  auto quotient = [&](float x) {
    const float q0 = __fmul_rn(x, inv);
    const float q1 = __fmaf_rn(-__fmaf_rn(q0, s, -x), inv, q0);
    return __fmaf_rn(-__fmaf_rn(q1, s, -x), inv, q1);
  };
  auto write = [&](const Pairs& x, int r) {
    float q[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] = quotient(x.x[j]);
    if (!finite) {
#pragma unroll
      for (int j = 0; j < 16; ++j) q[j] = __fdiv_rn(x.x[j], s);
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = codes4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
    uint8_t* o = codes + (size_t)(off + r) * a.D;
    *reinterpret_cast<uint2*>(o + ch.lo) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(o + ch.hi) = make_uint2(w[2], w[3]);
  };
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (r0 + i * rows < n) write(row(raw[i], r0 + i * rows), r0 + i * rows);
  if (kWPU == 1)
    for (int r = r0 + kRows * rows; r < n; r += rows) write(row(raw_row(r), r), r);
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
  // single tokens: a warp a unit; else the warps that hold a whole page in one go (a run list of
  // max_runs entries means T / max_runs tokens a run at least)
  const int whole = std::max(1, a.page_size * a.D / 2048);
  const int wpu = a.T <= 2 * a.max_runs ? 1 : whole;
  const int threads = std::max(128, 32 * wpu), units = threads / (32 * wpu);
  const long long kv = ((long long)a.max_runs * 2 * a.Hkv + units - 1) / units;
  const long long q = a.Hq > 0 ? a.T : 0;
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
