// Addition to the residual stream, root-mean-square norm and 1x128 quantization in one pass over the rows.
#include "step_device.cuh"

namespace moe {

// y = h w r with r = (mean(h^2) + eps)^-1/2.  A row stays in registers between its one read and its one
// write: 8 values (one 16-byte vector) a thread and step, so that the 16 lanes of a half-warp hold one 1x128 group.
// Squares of BF16 values are exact in fp32; their sum and r are pairs of fp32 words, so that y is the exact
// value rounded once to fp32 (but for some 2^-40), then to BF16.  Rounding in between would put about one value in 10^4 on the
// other side of a BF16 border from a 64-bit evaluation, and a group's scale with its largest value.
// What that takes, some 20 operations a value, is done two values at a time (fp32x2): one at a time, with divisions for the
// codes, 8192 x 7168 with residual and 8-bit form took 172 us.  It takes 85 us, 6.2 TB/s, where a copy runs at 6.7 (without
// the 8-bit form 69 us, 6.8 TB/s).  Few rows are all latency: 1 x 4096 2.3 us, 32 x 4096 with the 8-bit form 2.7 us.
struct NormParams {
  moe_rms_norm_args a;
  float inv_hi, inv_lo;   // 1 / H
  float eps_hi, eps_lo;
};

// The root of s = mean(h^2) + eps needs its square, whose low word has no room from s = 2^100 on (and squares of values above 2^63
// leave fp32's range): such a row is summed again with h * 2^-80, and eps * 2^-160.
constexpr float kSmaller = 8.271806125530277e-25f;    // 2^-80
constexpr float kLargest = 1.2676506002282294e30f;    // 2^100

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 values in one register pair.
struct Two {
  unsigned long long v;
  __device__ __forceinline__ float x() const { return __uint_as_float((uint32_t)v); }
  __device__ __forceinline__ float y() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ Two two(float x, float y) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ Two two(float x) { return two(x, x); }
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// (Not mul.rn.f32x2: where it feeds an addition the two are merged, and the product is not rounded.)
__device__ __forceinline__ Two operator*(Two a, Two b) { return fma(a, b, two(-0.0f)); }
__device__ __forceinline__ Two minus(Two a, Two b) { return fma(b, two(-1.0f), a); }   // a - b
__device__ __forceinline__ Two two_of(uint32_t bf16x2) { return two(lo16(bf16x2), hi16(bf16x2)); }

// Rows off 16 bytes are read and written by whole 16-byte words all the same, shifted into place; values one by one
// are left for the row's two ends, and where a word's other part belongs to another warp's lane.

// The 16 bytes from byte m on of two words.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int m) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t t[7], r[5];
#pragma unroll
  for (int i = 0; i < 7; ++i) t[i] = m & 4 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) r[i] = m & 8 ? t[i + 2] : t[i];
  const int bits = 8 * (m & 3);
  return make_uint4(__funnelshift_r(r[0], r[1], bits), __funnelshift_r(r[1], r[2], bits),
                    __funnelshift_r(r[2], r[3], bits), __funnelshift_r(r[3], r[4], bits));
}

// N vectors of a row of H, j = first + i step: the eight values from 8 j on, zero behind the row's end.  All whole words
// are on their way before the first is used, and before the row's ends are looked at.
template <bool kAligned, int N>
__device__ __forceinline__ void load_vectors(const uint16_t* row, int first, int step, int H, uint4 (&v)[N]) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (kAligned) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = first + i * step;
      v[i] = 8 * j < H ? *reinterpret_cast<const uint4*>(row + 8 * j) : zero;
    }
  } else {
    const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15), off = m / 2, need = m ? 16 : 8;   // bytes into its word
    const uint4* words = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(row) - m);
    const auto whole = [&](int j) { return 8 * j >= off && 8 * j - off + need <= H; };
    uint4 next[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = first + i * step;
      v[i] = whole(j) ? words[j] : zero;
      next[i] = whole(j) && m ? words[j + 1] : zero;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = shifted(v[i], next[i], m);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = first + i * step;
      if (8 * j < H && !whole(j)) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = 8 * j + 2 * u;
          w[u] = (k < H ? row[k] : 0u) | ((k + 1 < H ? row[k + 1] : 0u) << 16);
        }
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// Stores the 16-byte word (codes: the 8 bytes) in which vector j of the row begins: the vector's first values, behind the
// last ones of the vector before it.  The last vector's thread stores what is left behind that word too.
__device__ __forceinline__ void store_word(uint16_t* row, int j, int H, const uint4& v, const uint4& before) {
  const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15), mine = 8 - m / 2, e = 8 * j;
  const bool last = e + 8 >= H;
  if ((m == 0 || j > 0) && !(last && (m != 0 || e + 8 > H))) {
    reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(row) - m)[j] = m == 0 ? v : shifted(before, v, 16 - m);
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w}, b[4] = {before.x, before.y, before.z, before.w};
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (u >= mine && j > 0) row[e - 8 + u] = (uint16_t)(b[u / 2] >> (16 * (u % 2)));
    if ((u < mine || last) && e + u < H) row[e + u] = (uint16_t)(w[u / 2] >> (16 * (u % 2)));
  }
}
__device__ __forceinline__ void store_word(uint8_t* row, int j, int H, const uint2& q, const uint2& ahead) {
  const int m = (int)(reinterpret_cast<uintptr_t>(row) & 7), mine = 8 - m, e = 8 * j;
  const unsigned long long v = q.x | (unsigned long long)q.y << 32, b = ahead.x | (unsigned long long)ahead.y << 32;
  const bool last = e + 8 >= H;
  if ((m == 0 || j > 0) && !(last && (m != 0 || e + 8 > H))) {
    reinterpret_cast<unsigned long long*>(row - m)[j] = m == 0 ? v : b >> (8 * mine) | v << (8 * m);
    return;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (u >= mine && j > 0) row[e - 8 + u] = (uint8_t)(b >> (8 * u));
    if ((u < mine || last) && e + u < H) row[e + u] = (uint8_t)(v >> (8 * u));
  }
}

__device__ __forceinline__ uint4 shuffle(const uint4& v, int from) {
  return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, from), __shfl_sync(0xFFFFFFFFu, v.y, from),
                    __shfl_sync(0xFFFFFFFFu, v.z, from), __shfl_sync(0xFFFFFFFFu, v.w, from));
}
__device__ __forceinline__ uint2 shuffle(const uint2& v, int from) {
  return make_uint2(__shfl_sync(0xFFFFFFFFu, v.x, from), __shfl_sync(0xFFFFFFFFu, v.y, from));
}

// Stores a thread's vectors t + i threads.  The vector before a warp's first is the last of another warp, in `edges`
// (the last lanes' vectors, by i and warp, since before a barrier), or, with a row a warp, lane 31's of the step before.
template <bool kWarpRows, int N, typename V, typename T>
__device__ __forceinline__ void store_words(T* row, int t, int threads, int H, const V (&v)[N], const V* edges) {
  const int lane = t % 32, warp = t / 32;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = t + i * threads;
    V before = shuffle(v[i], max(lane - 1, 0));
    if (kWarpRows) {
      const V last = shuffle(v[i > 0 ? i - 1 : 0], 31);
      if (lane == 0) before = last;
    } else if (lane == 0 && j > 0) {
      before = warp > 0 ? edges[i * 32 + warp - 1] : edges[(i - 1) * 32 + threads / 32 - 1];
    }
    if (8 * j < H) store_word(row, j, H, v[i], before);
  }
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {   // rounded once
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The sum of squares of the thread's values, times `scale`^2.
template <int VPT>
__device__ __forceinline__ Pair sum_squares(const uint4 (&h)[VPT], float scale) {
  Two hi = two(0.0f), lo = two(0.0f);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t w[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      Two v = two_of(w[u]);
      if (scale != 1.0f) v = v * two(scale);
      const Two sq = v * v, s = hi + sq, t = minus(s, hi);
      lo = lo + (minus(hi, minus(s, t)) + minus(sq, t));
      hi = s;
    }
  }
  Pair r = {hi.x(), lo.x()};
  pair_add(r, Pair{hi.y(), lo.y()});
  return r;
}

// Eight values of y: h w r rounded to fp32, then to BF16.  r is the root over `scale`, the power of two that leaves it from 1 to
// 2.  The product of h and w alone may leave fp32's range though y does not; that of the scaled h, which is at most sqrt(H), and w
// leaves it where y does.  A BF16 weight's product with h has 16 bits; with an fp32 one (kWide) h r comes first, as a pair.
// (As a pair for both: 8192 x 7168 8-bit 84.8 -> 86.1 us.)
template <bool kWide>
__device__ __forceinline__ uint4 norm8(const uint4& h, const Two (&w)[4], const Pair& r, float scale) {
  constexpr uint32_t kSigns = 0x80008000u;
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
  uint32_t y[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const Two b = two_of(hw[u]) * two(scale);
    Two v;
    if (kWide) {
      const Two t = b * two(r.hi), low = fma(b, two(r.lo), fma(b, two(r.hi), b * two(-r.hi)));
      v = fma(t, w[u], low * w[u]);
    } else {
      v = fma(b * w[u], two(r.hi), b * two(r.lo) * w[u]);
    }
    // zeros take the product's sign (two-value products lose it)
    const uint32_t w_signs = __byte_perm((uint32_t)w[u].v, (uint32_t)(w[u].v >> 32), 0x7632);
    y[u] = (pack_bf16x2(v.x(), v.y()) & ~kSigns) | ((hw[u] ^ w_signs) & kSigns);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// The scale of a group whose largest magnitude is the BF16 value amax, and what its values are multiplied by: as
// group_scale_numerics's, without its division.  amax / 448 is at most a power of two 2^k where amax's mantissa is at most that of
// 448 = 1.75 * 2^8; else it is rounded by Markstein's step: with z = RN(1 / 448), q + (amax - 448 q) z of q = RN(amax z).
struct GroupScale {
  float scale, times;
  bool product;      // quotients are products
};
__device__ __forceinline__ GroupScale scale_of(float amax, int fmt, int numerics) {
  GroupScale g;
  if (fmt != MOE_SCALE_FP32) {
    constexpr uint32_t kOne = 0x00800000u, kLeast = 110u << 23;       // 2^-17, 1 / (448 * 512) rounded up
    const uint32_t up = ((__float_as_uint(amax) + (kOne / 4 - 1)) & 0xFF800000u);
    const uint32_t bits = max(up, kLeast + 8 * kOne) - 8 * kOne;
    g.scale = __uint_as_float(bits);
    g.times = __uint_as_float(254 * kOne - bits);
    g.product = true;
  } else if (numerics == MOE_NUMERICS_RECIPROCAL) {
    g.scale = group_scale_numerics(amax, fmt, numerics, &g.times);
    g.product = true;
  } else {
    constexpr float kInverse = 1.0f / 448.0f;
    const float q = amax * kInverse;
    g.scale = fmaxf(__fmaf_rn(__fmaf_rn(-q, 448.0f, amax), kInverse, q), kScaleFloor);
    g.times = __frcp_rn(g.scale);
    g.product = false;
  }
  return g;
}

// E4M3 codes of eight BF16 values of a group: as moe_quant_act's, quotients by Markstein's step again.
__device__ __forceinline__ uint2 codes8(const uint4& y, const GroupScale& g) {
  const uint32_t w[4] = {y.x, y.y, y.z, y.w};
  uint32_t c[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const Two v = two_of(w[u]);
    Two q = v * two(g.times);
    if (!g.product) q = fma(fma(q, two(-g.scale), v), two(g.times), q);
    // (a zero's sign is put back: two-value products lose it)
    c[u] = cvt_e4m3x2(q.x(), q.y()) | (__byte_perm(w[u], 0, 0x4431) & 0x8080u);
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// Threads of a block at most: 72 registers a thread let four blocks of 224 with four vectors a thread share an SM (8192 x
// 7168 without the 8-bit form: 69 us, with 84 registers 91 us; 8192 x 7167: 114 us, with 102 registers 157 us).
__host__ __device__ constexpr int most_threads(int vpt) { return vpt <= 2 ? 1024 : vpt == 4 ? 448 : 512; }

// VPT vectors a thread.  kWarpRows: a row a warp, four of them a block; otherwise a row a block of any number of warps.
template <int VPT, bool kWarpRows, bool kAligned, bool kQuant>
__global__ void __launch_bounds__(kWarpRows ? 128 : most_threads(VPT), kWarpRows ? (kAligned ? 7 : 6) : VPT == 4 ? 2 : 1)
k_rms_norm(const __grid_constant__ NormParams p) {
  constexpr int kEdges = kAligned || kWarpRows ? 1 : VPT * 32;      // the last lanes' vectors, for rows off 16 bytes
  __shared__ Pair part[2][32];
  __shared__ uint4 h_edges[kEdges], y_edges[kEdges];
  __shared__ uint2 q_edges[kQuant ? kEdges : 1];
  const moe_rms_norm_args& a = p.a;
  const int threads = kWarpRows ? 32 : blockDim.x, t = kWarpRows ? threadIdx.x % 32 : threadIdx.x;
  const long row = kWarpRows ? (long)blockIdx.x * 4 + threadIdx.x / 32 : (long)blockIdx.x;
  const int H = a.H, nvec = (H + 7) / 8;
  grid_dep_wait();
  grid_dep_launch_dependents();
  int n = a.M_cap;
  if (a.d_num_tokens != nullptr) n = min(max(*a.d_num_tokens, 0), a.M_cap);
  if (row >= n) return;   // all threads of the row, and no barrier joins rows

  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
  uint4 h[VPT];
  load_vectors<kAligned>(x, t, threads, H, h);
  if (a.residual != nullptr) {
    const uint16_t* res = static_cast<const uint16_t*>(a.residual) + row * a.residual_stride;
    uint4 r[VPT];
    load_vectors<kAligned>(res, t, threads, H, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      h[i] = make_uint4(add_bf16x2(h[i].x, r[i].x), add_bf16x2(h[i].y, r[i].y), add_bf16x2(h[i].z, r[i].z),
                        add_bf16x2(h[i].w, r[i].w));
  }

  constexpr bool kExchange = !kAligned && !kWarpRows;
  const bool at_edge = kExchange && t % 32 == 31;
  if (at_edge) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) h_edges[i * 32 + t / 32] = h[i];
  }

  // The sum of squares, twice where it or eps is large.  Code of its own for the second pass only with the tightest bound on
  // registers, where the loop's would spill (8192 x 7167 117.6 -> 114.1 us; 8192 x 7167 8-bit with it 149 -> 154 us).
  constexpr int kPasses = VPT == 4 && !kWarpRows && !kQuant ? 2 : 1;
  float scale = 1.0f;
  Pair sum;
#pragma unroll kPasses
  for (int pass = 0; pass < 2; ++pass) {
    sum = pair_reduce(pass == 0 ? sum_squares(h, 1.0f) : sum_squares(h, kSmaller), 32);
    if (!kWarpRows) {
      const int warps = threads / 32;
      if (t % 32 == 0) part[pass][t / 32] = sum;
      __syncthreads();
      sum = t % 32 < warps ? part[pass][t % 32] : Pair{0.0f, 0.0f};
      sum = pair_reduce(sum, 32);
    }
    if (sum.hi < kLargest && p.eps_hi < kLargest) break;
    if (pass == 0) scale = kSmaller;
  }

  // r: a first value from rsqrtf, then one step of Newton's with the residual 1 - s r^2 in pairs
  Pair s;
  s.hi = sum.hi * p.inv_hi;
  s.lo = __fmaf_rn(sum.hi, p.inv_hi, -s.hi) + (sum.hi * p.inv_lo + sum.lo * p.inv_hi);
  pair_add(s, p.eps_hi * scale * scale);
  s.lo += p.eps_lo * scale * scale;
  Pair r = {rsqrtf(s.hi), 0.0f};
  if (sum.hi < INFINITY) {
    const float q = r.hi * r.hi, q_lo = __fmaf_rn(r.hi, r.hi, -q);
    const float m = s.hi * q, m_lo = __fmaf_rn(s.hi, q, -m) + (s.hi * q_lo + s.lo * q);
    const float d = (1.0f - m) - m_lo;
    const uint32_t bits = __float_as_uint(r.hi), power = bits & 0x7F800000u;
    r.hi = __uint_as_float(bits - power + 0x3F800000u);
    r.lo = r.hi * (d * (0.5f + 0.375f * d));
    scale *= __uint_as_float(power);
  } else {
    scale = 0.0f;   // an infinity: zero but there; a NaN: r is one
  }

  uint16_t* res_out = a.residual_out == nullptr
                          ? nullptr : static_cast<uint16_t*>(a.residual_out) + row * a.residual_out_stride;
  uint16_t* out = a.out == nullptr ? nullptr : static_cast<uint16_t*>(a.out) + row * a.out_stride;
  const bool wide = a.weight_fp32 || a.weight_plus_one;
  if (!kAligned && res_out != nullptr) store_words<kWarpRows>(res_out, t, threads, H, h, h_edges);
  uint4 ys[kAligned ? 1 : VPT];
  uint2 qs[kAligned || !kQuant ? 1 : VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = t + i * threads;
    const bool have = j < nvec;
    asm volatile("" ::: "memory");   // one vector's weights at a time: all of them in registers would cost warps
    if (kAligned && have && res_out != nullptr) *reinterpret_cast<uint4*>(res_out + 8 * j) = h[i];
    Two w[4];
    if (a.weight_fp32) {
      const float* wf = static_cast<const float*>(a.weight) + 8 * j;
      if (kAligned || (8 * j + 8 <= H && reinterpret_cast<uintptr_t>(wf) % 16 == 0)) {
        const float4 w0 = have ? *reinterpret_cast<const float4*>(wf) : make_float4(0, 0, 0, 0);
        const float4 w1 = have ? *reinterpret_cast<const float4*>(wf + 4) : make_float4(0, 0, 0, 0);
        w[0] = two(w0.x, w0.y), w[1] = two(w0.z, w0.w), w[2] = two(w1.x, w1.y), w[3] = two(w1.z, w1.w);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          w[u] = two(8 * j + 2 * u < H ? wf[2 * u] : 0.0f, 8 * j + 2 * u + 1 < H ? wf[2 * u + 1] : 0.0f);
      }
    } else {
      uint4 wb[1];
      load_vectors<kAligned>(static_cast<const uint16_t*>(a.weight), j, 0, H, wb);
      w[0] = two_of(wb[0].x), w[1] = two_of(wb[0].y), w[2] = two_of(wb[0].z), w[3] = two_of(wb[0].w);
    }
    if (a.weight_plus_one) {
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = two(1.0f) + w[u];
    }
    const uint4 y = wide ? norm8<true>(h[i], w, r, scale) : norm8<false>(h[i], w, r, scale);
    if (kAligned && have && out != nullptr) *reinterpret_cast<uint4*>(out + 8 * j) = y;
    if (!kAligned) ys[kAligned ? 0 : i] = y;
    if (kQuant) {
      // the group's largest magnitude (zero behind the row's end)
      constexpr uint32_t kMagnitude = 0x7FFF7FFFu;
      uint32_t most = max_bf16x2(max_bf16x2(y.x & kMagnitude, y.y & kMagnitude),
                                 max_bf16x2(y.z & kMagnitude, y.w & kMagnitude));
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) most = max_bf16x2(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
      const GroupScale g = scale_of(fmaxf(lo16(most), hi16(most)), a.scale_fmt, a.numerics);
      const uint2 q = codes8(y, g);
      if (!kAligned) qs[kAligned ? 0 : i] = q;
      if (have) {
        if (kAligned) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.codes) + row * a.codes_stride + 8 * j) = q;
        if (t % 16 == 0)
          store_scale(a.scales, (size_t)(j / 16) * a.scales_stride + row, g.scale, a.scale_fmt == MOE_SCALE_UE8M0);
      }
    }
  }
  if (!kAligned) {
    if (kExchange) {
      if (at_edge) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          y_edges[i * 32 + t / 32] = ys[kAligned ? 0 : i];
          if (kQuant) q_edges[i * 32 + t / 32] = qs[kAligned ? 0 : i];
        }
      }
      __syncthreads();
    }
    if (out != nullptr) store_words<kWarpRows>(out, t, threads, H, ys, y_edges);
    if (kQuant)
      store_words<kWarpRows>(static_cast<uint8_t*>(a.codes) + row * a.codes_stride, t, threads, H, qs, q_edges);
  }
}

namespace {

template <int VPT, bool kWarpRows>
cudaError_t norm_of(const NormParams& p, bool aligned, int threads, cudaStream_t s) {
  const dim3 grid((unsigned)(kWarpRows ? ((long)p.a.M_cap + 3) / 4 : p.a.M_cap)), block(threads);
  if (p.a.codes != nullptr)
    return aligned ? launch_pdl(k_rms_norm<VPT, kWarpRows, true, true>, grid, block, 0, s, p)
                   : launch_pdl(k_rms_norm<VPT, kWarpRows, false, true>, grid, block, 0, s, p);
  return aligned ? launch_pdl(k_rms_norm<VPT, kWarpRows, true, false>, grid, block, 0, s, p)
                 : launch_pdl(k_rms_norm<VPT, kWarpRows, false, false>, grid, block, 0, s, p);
}

bool rows_on(const void* p, int64_t stride, size_t bytes, size_t size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (stride * size) % bytes == 0);
}

}  // namespace

cudaError_t launch_rms_norm(const moe_rms_norm_args& a, cudaStream_t s) {
  NormParams p;
  p.a = a;
  const double inv = 1.0 / a.H;
  p.inv_hi = (float)inv, p.inv_lo = (float)(inv - (double)p.inv_hi);
  p.eps_hi = (float)a.eps, p.eps_lo = (float)(a.eps - (double)p.eps_hi);
  const bool aligned = a.H % 8 == 0 && rows_on(a.x, a.x_stride, 16, 2) && rows_on(a.residual, a.residual_stride, 16, 2) &&
                       rows_on(a.residual_out, a.residual_out_stride, 16, 2) && rows_on(a.out, a.out_stride, 16, 2) &&
                       rows_on(a.weight, 0, 16, 2) && rows_on(a.codes, a.codes_stride, 8, 1);
  const int nvec = (a.H + 7) / 8;
  // Few rows: a vector a thread, for the shortest chain; many: more vectors a thread, for fewer barriers and whole
  // loads in flight.  8192 x 7168 with 1, 2, 4, 8 vectors a thread: 165, 106, 85, 85 us; 1 x 4096 with 1, 4: 2.2, 3.0 us;
  // 1021 x 1003: 3.8, 5.0 us.
  const long long all = (long long)a.M_cap * nvec, once = 2048ll * sm_count();
  const int want = all <= once ? 1 : all <= 2 * once ? 2 : 4;
  if (nvec <= 32 || (nvec <= 128 && want == 4)) {
    if (nvec <= 32) return norm_of<1, true>(p, aligned, 128, s);
    if (nvec <= 64) return norm_of<2, true>(p, aligned, 128, s);
    return norm_of<4, true>(p, aligned, 128, s);
  }
  const auto threads = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
  if (want <= 1 && threads(1) <= most_threads(1)) return norm_of<1, false>(p, aligned, threads(1), s);
  if (want <= 2 && threads(2) <= most_threads(2)) return norm_of<2, false>(p, aligned, threads(2), s);
  if (threads(4) <= most_threads(4)) return norm_of<4, false>(p, aligned, threads(4), s);
  return norm_of<8, false>(p, aligned, threads(8), s);
}

}  // namespace moe
