// Routing: scores, groups and the top-k choice of experts, one warp a token.
#include "step_device.cuh"

namespace moe {

// The choice is that of exact scores rounded once to fp32.  Scores of fp32 functions are some 2^-20 off, which turns the
// order of two experts round in one token of a few thousand.  So a token's experts are first ranked by fp32 scores; where
// two neighbours of that ranking stand closer than the scores' error (or anything is not a number) the warp evaluates
// the row again with exponentials of some 2^-45 (pairs of fp32 words: 64-bit arithmetic runs at a sixty-fourth of the rate).
//
// What bounds it is the number of operations, half of them on the integer and comparison pipe: about 700 a row of 256 experts
// in groups, 8 chosen (some 250 of them whatever E and k, 130 for groups, 15 for each choice).  16384 such rows 14.1 us (the
// bytes alone: 2.7), 8192 BF16 rows of 128 experts 5.4 us, one row 2.6 us; all scores in 64 bits took 214, 60 and 11 us.
//
// A warp a token.  Its lanes are dealt to the groups (L = 32 / groups a group, rounded down to a power of two) and hold
// consecutive experts, lower ids in higher lanes, so a group's statistics need shuffles among its lanes only.
struct RouteParams {
  moe_route_args a;
  int lanes_log2;  // lanes a group
  int group_size;
  int per_lane;    // experts a lane
  bool quads;      // logits can be loaded four at a time
  bool bias_quads; // and the bias too
};

constexpr int kRouteWarps = 4;
constexpr uint32_t kAllLanes = 0xFFFFFFFFu;

// Order of floats as order of words; 0 for what is never chosen.
__device__ __forceinline__ uint32_t order_of(float key) {
  const uint32_t b = __float_as_uint(key);
  return key > -INFINITY ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_of(uint32_t order) {
  return order == 0 ? -INFINITY : __uint_as_float(order ^ (order & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// ------------------------------------------------------------------------------ scores in pairs
// ln 2 in three words, the first of 16 bits, so that its products with an exponent are exact.
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kLn2a = 0.693145751953125f;
constexpr float kLn2b = (float)(kLn2 - (double)kLn2a);
constexpr float kLn2c = (float)(kLn2 - (double)kLn2a - (double)kLn2b);
constexpr float kSixth = (float)(1.0 / 6.0), kSixthLo = (float)(1.0 / 6.0 - (double)(float)(1.0 / 6.0));

__device__ __forceinline__ Pair pair_mul(const Pair& a, const Pair& b) {
  Pair r;
  r.hi = a.hi * b.hi;
  r.lo = __fmaf_rn(a.hi, b.hi, -r.hi) + (a.hi * b.lo + a.lo * b.hi);
  return r;
}

// exp(x) for x <= 0: x = k ln 2 + 16 m, |m| <= 0.0217; exp(m) - 1 by its power series, whose terms from m^4 on are
// small enough for fp32; then four times (1 + e)^2 = 1 + (2 e + e^2).  The power of two stays apart: a small pair would have
// no room for its low word.
struct Scaled {
  Pair m;      // exp(x - k ln 2), from 0.7 to 1.42, or zero
  int k;       // the value is m 2^k
};
__device__ __forceinline__ Scaled pair_exp(const Pair& x) {
  if (!(x.hi > -200.0f)) return {{0.0f, 0.0f}, 0};
  const float k = rintf(x.hi * 1.44269504f);
  Pair m = {x.hi - k * kLn2a, x.lo};
  const float q = k * kLn2b;
  m.lo -= __fmaf_rn(k, kLn2b, -q) + k * kLn2c;
  pair_add(m, -q);
  m.hi *= 0.0625f, m.lo *= 0.0625f;
  const Pair m2 = pair_mul(m, m), m3 = pair_mul(pair_mul(m2, m), Pair{kSixth, kSixthLo});
  const float y = m.hi;
  const float tail = m2.hi * m2.hi * (1.0f / 24 + y * (1.0f / 120 + y * (1.0f / 720)));
  Pair e = m;
  pair_add(e, Pair{0.5f * m2.hi, 0.5f * m2.lo});
  pair_add(e, m3);
  pair_add(e, tail);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Pair s = pair_mul(e, e);
    e.hi *= 2.0f, e.lo *= 2.0f;
    pair_add(e, s);
  }
  pair_add(e, 1.0f);
  return {e, (int)k};
}

__device__ __forceinline__ float power_of_two(int k) { return __int_as_float((127 + k) << 23); }   // k from -126 on

// The value itself, for a sum of at least one: what a small one loses is far below that sum's low word.
__device__ __forceinline__ Pair value_of(const Scaled& e) {
  const float a = power_of_two(max(e.k, -126));
  return {e.m.hi * a, e.m.lo * a};
}

// (In line, its registers spill in the kernel of two experts a lane.)
__device__ __noinline__ float small_quotient(float q, float rest, int k) {
  return __double2float_rn(((double)q + (double)rest) * __hiloint2double((1023 + k) << 20, 0));
}

// a / b rounded once, for b from 1 to 1024.  Below 2^-126 fp32 keeps fewer bits, so a quotient that may lie there is
// joined and scaled in 64 bits, and the conversion rounds it.
__device__ __forceinline__ float pair_div(const Scaled& a, const Pair& b) {
  const float q = a.m.hi / b.hi;
  const float rest = (__fmaf_rn(-q, b.hi, a.m.hi) + (a.m.lo - q * b.lo)) / b.hi;
  if (a.k > -100) return (q + rest) * power_of_two(a.k);
  return small_quotient(q, rest, a.k);
}

// ------------------------------------------------------------------------------------- the row
// Logits of the lane's experts, -inf past its last.
template <int EPL, bool kBf16>
__device__ __forceinline__ void load_logits(const RouteParams& p, long row, int base, int have, float (&x)[EPL]) {
  const int64_t at = row * p.a.logits_stride + base;
#pragma unroll
  for (int i = 0; i < EPL; ++i) x[i] = -INFINITY;
  if (EPL >= 4 && p.quads) {
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i)
      if (4 * i < have) {
        if (kBf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.a.logits) + at + 4 * i);
          x[4 * i] = __uint_as_float(w.x << 16), x[4 * i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
          x[4 * i + 2] = __uint_as_float(w.y << 16), x[4 * i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.a.logits) + at + 4 * i);
          x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < have)
        x[i] = kBf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p.a.logits)[at + i])
                     : static_cast<const float*>(p.a.logits)[at + i];
  }
}

template <int EPL>
__device__ __forceinline__ void load_bias(const RouteParams& p, int base, int have, float (&b)[EPL]) {
  const float* at = p.a.bias + base;
  if (EPL >= 4 && p.bias_quads) {
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i) {
      const float4 w = 4 * i < have ? *reinterpret_cast<const float4*>(at + 4 * i) : make_float4(0, 0, 0, 0);
      b[4 * i] = w.x, b[4 * i + 1] = w.y, b[4 * i + 2] = w.z, b[4 * i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = i < have ? at[i] : 0.0f;
  }
}

// An expert's word in the fp32 ranking: the order of its key with the low bits given to its place in the lane (lower
// places above), so that one word sorts and names it.  (Those bits of BF16 logits say nothing anyway.)
constexpr uint32_t kNever = 0x007FFFFFu;      // the order of -inf: never chosen
constexpr uint32_t kInfinite = 0xFF800000u;   // of +inf
__device__ __forceinline__ uint32_t word_of(float key, uint32_t places, uint32_t place) {
  const uint32_t b = __float_as_uint(key), o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return (o & ~places) | (places - place);
}
__device__ __forceinline__ float word_key(uint32_t word, uint32_t places) {
  return word <= kNever ? -INFINITY : key_of(word & ~places);
}

__device__ __forceinline__ float max_lanes(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float min_lanes(float v) {
  float r;
  asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The two largest keys of the lane's group, from those of the lane; returns its value.
__device__ __forceinline__ float group_value(const RouteParams& p, float& one, float& two) {
  for (int d = (1 << p.lanes_log2) >> 1; d >= 1; d >>= 1) {
    const float o1 = __shfl_xor_sync(kAllLanes, one, d), o2 = __shfl_xor_sync(kAllLanes, two, d);
    two = fmaxf(fmaxf(two, o2), fminf(one, o1));
    one = fmaxf(one, o1);
  }
  return p.a.group_best == 2 && two > -INFINITY ? one + two : one;
}

// Whether the lane's group is one of the topk_groups of the largest values.  Each of a group's lanes compares with
// its share of the other groups.
__device__ __forceinline__ bool group_stays(const RouteParams& p, float value, int group, int sub) {
  const int lanes = 1 << p.lanes_log2;
  int above = 0;
  for (int g0 = 0; g0 < p.a.num_groups; g0 += lanes) {
    const int g = g0 + sub;
    const float o = __shfl_sync(kAllLanes, value, 31 - ((g << p.lanes_log2) & 31));
    above += g < p.a.num_groups && (o > value || (o == value && g < group));
  }
  for (int d = lanes >> 1; d >= 1; d >>= 1) above += __shfl_xor_sync(kAllLanes, above, d);
  return above < p.a.topk_groups;
}

struct Choice {
  int id;         // lane j: the j-th expert, -1 for none
  float score;
  bool spoilt;
};

// The score of a logit that is a number or -inf.
__device__ __noinline__ float exact_score(float x, bool softmax, float top, Pair total) {
  Pair d = {x, 0.0f};
  if (softmax) {
    if (!(x > -INFINITY)) return 0.0f;
    pair_add(d, -top);
    return pair_div(pair_exp(d), total);
  }
  const Scaled e = pair_exp(Pair{-fabsf(x), 0.0f});
  Pair one = value_of(e);
  pair_add(one, 1.0f);
  return pair_div(x < 0.0f ? e : Scaled{{1.0f, 0.0f}, 0}, one);
}

// The sum of exp(x - top) over the warp's logits, `have` of them a lane, 32 words apart.
__device__ __noinline__ Pair exact_sum(const uint32_t* xs, int have, float top) {
  Pair total = {0.0f, 0.0f};
#pragma unroll 2
  for (int i = 0; i < have; ++i) {
    Pair d = {__uint_as_float(xs[32 * i]), 0.0f};
    if (d.hi > -INFINITY) {
      pair_add(d, -top);
      pair_add(total, value_of(pair_exp(d)));
    }
  }
  return pair_reduce(total, 32);
}

// The row from exact scores (in pairs).  Few rows come here, so the code is short rather than quick: it is fetched
// for one row.  xs, orders: the warp's shared memory, a word for each lane and place.
template <bool kBf16>
__device__ __noinline__ Choice route_exactly(const RouteParams& p, long row, uint32_t* xs, uint32_t* orders) {
  const moe_route_args& a = p.a;
  const int lane = threadIdx.x % 32, place = 31 - lane, group = place >> p.lanes_log2;
  const int sub = place & ((1 << p.lanes_log2) - 1), first = sub * p.per_lane;
  const int base = group * p.group_size + first;
  const int have = group < a.num_groups ? min(p.per_lane, p.group_size - first) : 0;
  const bool softmax = a.scoring == MOE_ROUTE_SOFTMAX;
  const int64_t at = row * a.logits_stride + base;
  xs += lane, orders += lane;
  bool spoilt = false;
  float top = -INFINITY;
  for (int i = 0; i < have; ++i) {
    float x = kBf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[at + i])
                    : static_cast<const float*>(a.logits)[at + i];
    if (isnan(x) || (softmax && x == INFINITY)) {
      spoilt = true;
      x = -INFINITY;
    }
    xs[32 * i] = __float_as_uint(x);
    top = fmaxf(top, x);
  }
  top = max_lanes(top);
  Pair total = {0.0f, 0.0f};
  if (softmax) total = exact_sum(xs, have, top);
  float one = -INFINITY, two = -INFINITY;
#pragma unroll 2
  for (int i = 0; i < have; ++i) {
    const float x = __uint_as_float(xs[32 * i]), s = exact_score(x, softmax, top, total);
    const uint32_t order = x > -INFINITY ? order_of(a.bias != nullptr ? s + a.bias[base + i] : s) : 0u;
    xs[32 * i] = __float_as_uint(s);
    orders[32 * i] = order;
    const float k = key_of(order);
    two = fmaxf(two, fminf(one, k));
    one = fmaxf(one, k);
  }
  const bool stays = a.num_groups == 1 || group_stays(p, group_value(p, one, two), group, sub);

  // the largest keys one by one
  Choice c = {-1, 0.0f, __any_sync(kAllLanes, spoilt) != 0};
  for (int j = 0; j < a.topk; ++j) {
    uint32_t best = 0;
    int best_at = 0;
    for (int i = 0; stays && i < have; ++i) {
      const uint32_t o = orders[32 * i];
      if (o > best) best = o, best_at = i;
    }
    const uint32_t most = __reduce_max_sync(kAllLanes, best);
    if (most == 0) break;
    const int src = 31 - __clz(__ballot_sync(kAllLanes, best == most));   // the lower ids among equals
    const int id = __shfl_sync(kAllLanes, base + best_at, src);
    const float score = __shfl_sync(kAllLanes, __uint_as_float(xs[32 * best_at]), src);
    if (lane == src) orders[32 * best_at] = 0;
    if (lane == j) c.id = id, c.score = score;
  }
  return c;
}

// ----------------------------------------------------------------------- fp32 scores, sorted lanes
// exp(d) within (2^-22 + |d| 2^-22) of its value.
__device__ __forceinline__ float fast_exp(float d) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(d * 1.44269504f));
  return r;
}
// The same within (2^-22 + |d| 2^-24): what the product lost is put back.
__device__ __forceinline__ float exp_of(float d) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(-1e4f));   // an infinity would make the correction a NaN
  const float t = d * kHi, rest = __fmaf_rn(d, kLo, __fmaf_rn(d, kHi, -t));
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(t));
  return __fmaf_rn(r, rest * 0.693147181f, r);
}
__device__ __forceinline__ float fast_rcp(float v) {   // within 2^-23
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float fast_sigmoid(float x) {
  const float e = fast_exp(-fabsf(x));
  return (x < 0.0f ? e : 1.0f) * fast_rcp(1.0f + e);
}

// Descending order by Batcher's odd-even merges.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = max(a, b);
            v[i + j + k] = min(a, b);
          }
}

// kSoftmax: with the scoring known when it is compiled a kernel holds fewer registers and branches (16384 x 256 grouped
// 15.2 -> 14.6 us, 8192 x 128 5.9 -> 5.5 us).  The few rows that fp32 does not decide are settled in place: in functions of
// their own, or begun anew there, 16384 rows take 0.6 to 1 us more, because the last of the few ends later.
template <int EPL, bool kBf16, bool kSoftmax>
__global__ void __launch_bounds__(32 * kRouteWarps) k_route(const __grid_constant__ RouteParams p) {
  constexpr uint32_t kPlace = EPL - 1;
  __shared__ uint32_t lists[kRouteWarps][EPL + 1][32], more[kRouteWarps][EPL][32];
  const moe_route_args& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long row = (long)blockIdx.x * kRouteWarps + warp;
  grid_dep_wait();
  grid_dep_launch_dependents();
  int n = a.M_cap;
  if (a.d_num_tokens != nullptr) n = min(max(*a.d_num_tokens, 0), a.M_cap);
  if (row >= n) return;

  // the last lane holds the lowest ids: the highest of a ballot's bits is found in one step
  const int place = 31 - lane, group = place >> p.lanes_log2, sub = place & ((1 << p.lanes_log2) - 1);
  const int first = sub * p.per_lane, base = group * p.group_size + first;   // id of the lane's first expert
  const int have = group < a.num_groups ? min(p.per_lane, p.group_size - first) : 0;
  float x[EPL];
  load_logits<EPL, kBf16>(p, row, base, have, x);

  // softmax: the largest logit and one over the sum
  float top = 0.0f, inv = 1.0f;
  if (kSoftmax) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) top = fmaxf(top, x[i]);
    top = max_lanes(top);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum[i % 4] += exp_of(x[i] - top);   // zero for -inf
    float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(kAllLanes, total, d);
    inv = fast_rcp(total);
  }
  auto score_of = [&](float v) { return kSoftmax ? exp_of(v - top) * inv : fast_sigmoid(v); };
  // How far off such a score may be, rounding to fp32 included.  Sigmoid: s ((1 - s) (2^-22 + |x| 2^-22) + 3 2^-24)
  // at most, and s (1 - s) (1 + |x|) < 0.55.  Softmax, in units of 2^-24 of the largest score, inv: the sum is off by 4 (its
  // exponentials), 1 (their correction), 7 (the rounded differences d = l - top: |d| each, whose mean under the softmax is
  // at most ln 1024) and 15 (additions); an expert's exponential by (6 + |d|) exp(-|d|) <= 6; reciprocal, product and
  // rounding by 4: 37.
  const float slack = kSoftmax ? 2.4e-6f * inv : 5e-7f;

  // Without a bias scores order as logits do, so logits are ranked.
  uint32_t v[EPL];
  if (a.bias == nullptr) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = word_of(x[i] + 0.0f, kPlace, i);   // a negative zero is zero
  } else {
    float key[EPL];
    if (kSoftmax) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = exp_of(x[i] - top) * inv;
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = fast_rcp(1.0f + fast_exp(-x[i]));   // zero below -88: less than slack
    }
    float b[EPL];
    load_bias<EPL>(p, base, have, b);
    float whole = 0.0f;   // a NaN where a logit is infinite: products are cheaper than comparisons (14.4 -> 14.1 us)
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] += b[i], whole = __fmaf_rn(x[i], 0.0f, whole);
    if (__any_sync(kAllLanes, isnan(whole))) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = x[i] == -INFINITY ? -INFINITY : key[i];
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = word_of(key[i], kPlace, i);
  }
  sort_down(v);
  // what is not a number stands before all numbers or behind all; so does an infinity
  const bool odd = v[0] >= kInfinite || v[EPL - 1] < (kNever & ~kPlace);

  // What the low bits' loss may hide: a share of the key (or logit) as fp32 has it.
  constexpr float kLoss = 1.2e-7f * EPL;      // EPL * 2^-23
  bool unsure = false, undecided = false;
  // For the few rows where fp32 does not decide: exact keys of single experts, and the most that the key of an expert
  // may be whose word is not above another's.
  Pair exact_total = {0.0f, 0.0f};
  auto sum_exactly = [&] {
    if (kSoftmax && !(exact_total.hi > 0.0f)) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) more[warp][i][lane] = __float_as_uint(x[i]);
      exact_total = exact_sum(&more[warp][0][lane], EPL, top);
    }
  };
  auto id_of = [&](uint32_t w) { return base + (int)(~w & kPlace); };   // of one of the lane's own
  auto logit_of = [&](int id) {
    const int64_t at = row * a.logits_stride + id;
    return kBf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[at])
                 : static_cast<const float*>(a.logits)[at];
  };
  auto exact_key = [&](uint32_t w) {      // of one of the lane's own
    const bool is = w > kNever;
    const int id = is ? id_of(w) : 0;
    const float e = exact_score(is ? logit_of(id) : -INFINITY, kSoftmax, top, exact_total);
    return !is ? -INFINITY : a.bias != nullptr ? e + a.bias[id] : e;
  };
  auto bound_of = [&](uint32_t w) {
    if (w <= kNever) return -INFINITY;
    const float k = key_of(w | kPlace);
    return a.bias != nullptr ? k + slack + 1.2e-7f * fabsf(k) : score_of(k) + slack;
  };
  if (a.num_groups > 1) {
    // the two largest keys of the lane, and how far off their sum may be
    float one = word_key(v[0], kPlace), two = EPL > 1 ? word_key(v[EPL > 1 ? 1 : 0], kPlace) : -INFINITY, err;
    if (a.bias == nullptr) {
      // logits so far; what a logit has lost, a share |logit| of it is lost in the score.  The terms fall with the
      // score, so the larger key's stand for both; the softmax's sum is common to all
      const float l = one;
      if (one > -INFINITY) one = score_of(one);
      if (two > -INFINITY) two = score_of(two);
      err = 2.0f * one * (2.5e-7f * (2.5f + fabsf(l - top)) + kLoss * (1.0f + fabsf(l)));
    } else {
      err = 2.0f * slack + (kLoss + 2.4e-7f) * (fabsf(one) + (two > -INFINITY ? fabsf(two) : 0.0f));
    }
    if (!(one > -INFINITY)) err = 0.0f;
    float value = group_value(p, one, two);
    bool stays = group_stays(p, value, group, sub);
    // the values on the two sides of the border
    const float least = min_lanes(stays ? value : INFINITY), next = max_lanes(stays ? -INFINITY : value);
    if (next > -INFINITY && !(least - next > 2.0f * max_lanes(err) + 1e-36f)) {
      // the same from exact keys of each lane's first two; the third must not reach its group's second
      sum_exactly();
      const float k0 = exact_key(v[0]), k1 = EPL > 1 ? exact_key(v[EPL > 1 ? 1 : 0]) : -INFINITY;
      one = fmaxf(k0, k1), two = fminf(k0, k1);
      value = group_value(p, one, two);
      stays = group_stays(p, value, group, sub);
      const float bound = EPL > 2 ? bound_of(v[EPL > 2 ? 2 : 0]) : -INFINITY;
      undecided = bound > -INFINITY && bound >= (a.group_best == 2 ? two : one);
    }
    if (!stays) v[0] = 0;   // (no lane looks past its first word then)
  }

  // The largest words one by one; the lane that has the j-th leaves its expert in found[j].  A lane's sorted list waits in
  // shared memory, where the next word is one load away (in registers the whole list would shift, in every round).  (Words
  // and lanes handed to lane j by shuffles and selections: 16384 x 256 14.6 us instead of 14.4, 8192 x 128 5.5 instead of 5.3.)
  uint32_t* list = &lists[warp][0][lane];
  uint32_t(&found)[32] = lists[warp][0];
  found[lane] = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 1; i < EPL; ++i) list[32 * i] = v[i];
  list[32 * EPL] = 0;
  __syncwarp();
  uint32_t head = v[0];
  auto pop = [&](int j) {
    const uint32_t mine = head & ~kPlace, most = __reduce_max_sync(kAllLanes, mine);
    const int src = 31 - __clz(__ballot_sync(kAllLanes, mine == most));   // the lower ids among equals
    if (lane == src && most > kNever) {
      found[j] = id_of(head);
      list += 32;
      head = *list;
    }
  };
  for (int j = 0; j < a.topk; ++j) pop(j);
  const uint32_t rest = __reduce_max_sync(kAllLanes, head & ~kPlace);     // of all that are left
  __syncwarp();

  // Their scores and keys, and how far off those may be.  Weights come of these scores unless the row is evaluated again: off by
  // 1.1 units of 2^-24 in the mean square; with expf and true divisions in their place by 1.1 too, in the same time.
  int id = (int)found[lane];
  float s = 0.0f, key = -INFINITY, off = 0.0f, logit = -INFINITY, depth = -INFINITY;   // depth: the score is at most its exp
  if (id >= 0) {
    logit = logit_of(id);
    if (kSoftmax) {
      Pair d = {logit, 0.0f};
      pair_add(d, -top);
      s = exp_of(d.hi) * (1.0f + d.lo) * inv;
      depth = d.hi;
    } else {
      const float e = exp_of(-fabsf(logit));
      s = (logit < 0.0f ? e : 1.0f) * fast_rcp(1.0f + e);
      depth = logit;
    }
    key = a.bias != nullptr ? s + a.bias[id] : s;
    // with a bias: 7 units of 2^-24 in the score, what the softmax's sum is off, the key's rounding
    off = 4.2e-7f * s + 1.2e-7f * fabsf(key) + 1e-36f;
    if (kSoftmax) off += slack;
  }
  // Each place against the next, the last one against all that are left, of which their words' upper end is known.
  const float next_key = __shfl_down_sync(kAllLanes, key, 1), next_off = __shfl_down_sync(kAllLanes, off, 1);
  const float next_logit = __shfl_down_sync(kAllLanes, logit, 1);
  if (id >= 0) {
    const bool last = lane == a.topk - 1;
    const float bound = rest <= kNever ? -INFINITY : key_of(rest | kPlace);
    if (a.bias != nullptr) {
      // a score near fp32's smallest numbers weighs as its few bits say: it is evaluated again, unless it is zero for sure
      unsure |= s < 1e-36f && depth > -105.0f;
      unsure |= !(key - (last ? bound : next_key) > off + (last ? off + slack : next_off));
    } else {
      // rounded scores keep the order of logits; they differ where the scores are more than 2^-23 of them apart, and
      // s' = s (1 - s), or s in a softmax whose sum stands.  (BF16 logits are whole in their words.)
      const float other = !last ? next_logit : kBf16 && bound >= 0.0f ? key_of(rest) : bound;
      const float slope = kSoftmax ? 1.0f : fast_rcp(1.0f + fast_exp(logit));   // 1 - s at the upper end: the least
      // equal logits have equal scores; behind the last place only if the next lower logit has another one (BF16: it is
      // |logit| / 256 lower at least; a word does not tell equal FP32 logits)
      const bool equal = logit == other;
      const float gap = !equal ? logit - other : kBf16 ? fabsf(logit) * 0.00390625f : 0.0f;
      unsure |= !(equal && !last) && !(gap * slope > 1.5e-7f && s > 1e-36f);
    }
  }
  bool spoilt = false;
  if (__any_sync(kAllLanes, unsure || undecided || odd)) {
    if (!__any_sync(kAllLanes, odd || undecided)) {
      // exact keys of the experts found and of a few more, ranked anew
      constexpr int kMore = 4;
      __syncwarp();
      for (int j = a.topk; j < a.topk + kMore; ++j) pop(j);
      const float bound = bound_of(__reduce_max_sync(kAllLanes, head & ~kPlace));
      sum_exactly();
      __syncwarp();
      id = (int)found[lane];
      s = exact_score(id >= 0 ? logit_of(id) : -INFINITY, kSoftmax, top, exact_total);
      key = id < 0 ? -INFINITY : a.bias != nullptr ? s + a.bias[id] : s;
      int rank = 0;
      for (int j = 0; j < a.topk + kMore; ++j) {
        const float o = __shfl_sync(kAllLanes, key, j);
        const int o_id = __shfl_sync(kAllLanes, id, j);
        rank += o > key || (o == key && o_id < id);
      }
      // the last one wanted has to stand clear of those that were not looked at
      undecided = id >= 0 && rank == a.topk - 1 && !(key > bound);
      uint32_t(&pass)[32] = more[warp][0];
      uint32_t(&pass_s)[32] = lists[warp][0];
      pass[lane] = 0xFFFFFFFFu;
      pass_s[lane] = 0;
      __syncwarp();
      if (id >= 0) pass[rank] = id, pass_s[rank] = __float_as_uint(s);
      __syncwarp();
      id = (int)pass[lane], s = __uint_as_float(pass_s[lane]);
    }
    if (__any_sync(kAllLanes, odd || undecided)) {
      __syncwarp();
      const Choice c = route_exactly<kBf16>(p, row, lists[warp][0], more[warp][0]);
      id = c.id, s = c.score, spoilt = c.spoilt;
    }
  }
  if (lane >= a.topk) s = 0.0f;
  float total = s;
  for (int d = 8; d >= 1; d >>= 1) total += __shfl_xor_sync(kAllLanes, total, d);
  if (lane < a.topk) {
    float w = s;
    // (an approximate division's bounds end at divisors of 2^-126; sums of small sigmoids lie below)
    if (a.renormalize) w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
    w *= a.scale;
    if (spoilt) w = __int_as_float(0x7FC00000);
    const int64_t at = row * a.topk + lane;
    a.topk_ids[at] = id;
    a.topk_weights[at] = w;
  }
}

namespace {

template <int EPL>
cudaError_t route_of(const RouteParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)(((long)p.a.M_cap + kRouteWarps - 1) / kRouteWarps)), block(32 * kRouteWarps);
  if (p.a.scoring == MOE_ROUTE_SOFTMAX)
    return p.a.logits_bf16 ? launch_pdl(k_route<EPL, true, true>, grid, block, 0, s, p)
                           : launch_pdl(k_route<EPL, false, true>, grid, block, 0, s, p);
  return p.a.logits_bf16 ? launch_pdl(k_route<EPL, true, false>, grid, block, 0, s, p)
                         : launch_pdl(k_route<EPL, false, false>, grid, block, 0, s, p);
}

}  // namespace

cudaError_t launch_route(const moe_route_args& a, cudaStream_t s) {
  RouteParams p;
  p.a = a;
  p.lanes_log2 = 5;
  while ((a.num_groups << p.lanes_log2) > 32) --p.lanes_log2;
  p.group_size = a.E / a.num_groups;
  p.per_lane = (p.group_size + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
  // whole vectors, on fewer lanes where they do not come out even
  const size_t size = a.logits_bf16 ? 2 : 4;
  p.quads = p.per_lane > 2 && p.group_size % 4 == 0 && a.logits_stride % 4 == 0 &&
            reinterpret_cast<uintptr_t>(a.logits) % (4 * size) == 0;
  p.bias_quads = p.quads && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  if (p.quads) p.per_lane = (p.per_lane + 3) / 4 * 4;
  if (p.per_lane <= 1) return route_of<1>(p, s);
  if (p.per_lane <= 2) return route_of<2>(p, s);
  if (p.per_lane <= 4) return route_of<4>(p, s);
  if (p.per_lane <= 8) return route_of<8>(p, s);
  if (p.per_lane <= 16) return route_of<16>(p, s);
  return route_of<32>(p, s);
}

}  // namespace moe
