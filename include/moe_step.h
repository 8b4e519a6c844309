/*
 * moe_step.h -- C ABI of what a decoder step does beside attention (moe_kv.h) and experts (moe_fp8.h):
 * the residual stream's addition and norm in front of either, the routing that chooses the experts, and the
 * verification of drafted tokens after the step, which says how many of them the cache keeps.
 *
 * The conventions are those of moe_fp8.h: tensor arguments are device pointers owned by the caller;
 * nothing is allocated, the host is not synchronised, all work goes to `stream` (so a step can be
 * captured in a CUDA graph); arguments are validated on the host before anything is launched.  No call needs
 * a workspace or keeps anything, so calls on several streams do not meet.
 * d_num_tokens, when not NULL, is a device int32 holding the number of live rows n (clamped to [0, M_cap]);
 * rows from n on are neither read nor written.  NULL means n = M_cap.
 */
#ifndef MOE_STEP_H_
#define MOE_STEP_H_

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------------------- norm of the residual stream
 * Per live row of H values:
 *   h = RN_bf16(x + residual), or x where residual is NULL; h is written to residual_out
 *   y = RN_bf16(RN_fp32(h * w * (mean(h^2) + eps)^-1/2)), w = weight, or RN_fp32(1 + weight) with weight_plus_one
 * Squares, their sum, the root and the products carry some 40 bits up to the one rounding to fp32, so y
 * does not depend on how a row is split over threads.  (Fewer where y is below 2^-100, or h below that share of the root.)
 * Weights are finite; h * w may leave fp32's range where y does not.
 *   out     y itself (NULL: not wanted)
 *   codes, scales: y quantized per 1x128 group exactly as moe_quant_act quantizes such a row, with its formats
 *           and numerics (NULL: not wanted).  The last group is shorter where 128 does not divide H.
 *           scales[g * scales_stride + row], fp32 or, for MOE_SCALE_UE8M0, one byte: column-major, as the
 *           layer's own.
 * residual and residual_out are given together; residual_out may be residual, and out may be x or residual,
 * with the same stride.  Any other overlap of an output with an input or another output is refused
 * (MOE_ERR_INVALID_ARG).
 * Sums of x and residual that leave BF16's range become infinite.  Values of h as large as BF16 holds are
 * normed; a row that holds an infinity is NaN there and zero elsewhere, a row that holds a NaN is NaN.
 * Codes and scales of such rows hold nothing of use.
 * Supported: 1 <= H <= 32768, eps from 1e-20 on, finite; 0 <= M_cap.  Strides in elements, at least H for outputs
 * of more than one row and not negative for inputs; the values of a row are contiguous.  Pointers aligned to
 * their type (rows and strides on 16 bytes, H a multiple of 8, are the quicker). */
typedef struct {
  const void* x;               /* bf16 [M_cap, H] */
  const void* residual;        /* bf16 [M_cap, H] or NULL */
  const void* weight;          /* bf16 or fp32 [H] */
  const int32_t* d_num_tokens; /* device int32 n, or NULL */
  void* residual_out;          /* bf16 [M_cap, H]; NULL without residual */
  void* out;                   /* bf16 [M_cap, H] or NULL */
  void* codes;                 /* E4M3 [M_cap, H] or NULL */
  void* scales;                /* [ceil(H / 128), M_cap] fp32 or uint8; NULL without codes */
  int64_t x_stride, residual_stride, residual_out_stride, out_stride, codes_stride, scales_stride;
  double eps;
  int M_cap, H;
  int weight_fp32;             /* 1: weight is fp32 */
  int weight_plus_one;
  moe_scale_fmt scale_fmt;
  moe_numerics numerics;
} moe_rms_norm_args;

moe_status moe_rms_norm(const moe_rms_norm_args* args, moe_stream_t stream);

/* The experts' input from rows that are quantized already (moe_rms_norm's codes and scales, or any in moe_quant_act's
 * format): moe_place_act stands in moe_quant_act's place behind moe_align and leaves the same workspace;
 * moe_fp8_block_forward_codes is moe_fp8_block_forward with it (args->x is not used).
 * codes: E4M3 [M_cap, H], 16-byte aligned, codes_stride a multiple of 16; scales[g * scales_stride + row], H / 128 of them a
 * row, in the format act_fmt (args->act_scale_fmt).  Strides in elements, not negative. */
moe_status moe_place_act(const void* codes, int64_t codes_stride, const void* scales, int64_t scales_stride,
                         const int32_t* d_num_tokens, int M_cap, int E, int H, int I, int topk, moe_scale_fmt act_fmt,
                         void* workspace, size_t workspace_bytes, moe_stream_t stream);
moe_status moe_fp8_block_forward_codes(const moe_fwd_args* args, const void* codes, int64_t codes_stride,
                                       const void* scales, int64_t scales_stride, void* workspace,
                                       size_t workspace_bytes, moe_stream_t stream);

/* -------------------------------------------------------------------------------------- routing to experts
 * Per live row of E logits l, the topk experts and their weights as moe_fp8_block_forward takes them:
 *   s_e   = RN_fp32(softmax(l)_e) or RN_fp32(1 / (1 + exp(-l_e))), the exact value rounded once
 *   key_e = RN_fp32(s_e + bias_e), or s_e without a bias
 *   With num_groups > 1 the experts fall into that many groups of E / num_groups consecutive ones.  A group's
 *   value is its largest key (group_best 1) or the fp32 sum of its two largest (group_best 2); only experts of
 *   the topk_groups groups of the largest values stay, the lower group first among equals.
 *   topk_ids: the experts of the topk largest keys, in descending order, the lower id first among equals.
 *   topk_weights: s of those (not the key); with renormalize divided by their sum (0 where the sum is 0); times scale.
 * Keys are compared as if they had been computed exactly and rounded as above: the choice is that of a 64-bit
 * evaluation but where that itself stands within 2^-38 of a rounding border.  Weights are within 2^-18 of their value, where
 * the bounds of all that approximates add up; some 2^-24 as a rule, as with every part of them rounded to fp32.
 * An expert whose logit is -inf (a mask), or whose key is -inf or NaN, is never chosen, nor a group without any
 * other.  Places that find no expert get id -1 and weight 0 (the layer drops such pairs).  A NaN logit, and with
 * MOE_ROUTE_SOFTMAX a logit of +inf, is never chosen and makes all the row's weights NaN.
 * Supported: 1 <= E <= 1024, 1 <= topk <= 16, topk <= E / num_groups * topk_groups, num_groups from 1 to 32 that divides
 * E, E / num_groups * (num_groups rounded up to a power of two) <= 1024, 1 <= topk_groups <= num_groups, 0 <= M_cap, M_cap * topk < 2^31.
 * logits_stride in elements, not negative; topk_ids and topk_weights are [M_cap, topk], contiguous. */
typedef enum { MOE_ROUTE_SOFTMAX = 0, MOE_ROUTE_SIGMOID = 1 } moe_route_scoring;

typedef struct {
  const void* logits;          /* fp32 or bf16 [M_cap, E] */
  const float* bias;           /* [E] or NULL */
  const int32_t* d_num_tokens; /* device int32 n, or NULL */
  int32_t* topk_ids;           /* [M_cap, topk] */
  float* topk_weights;         /* [M_cap, topk] */
  int64_t logits_stride;
  int M_cap, E, topk;
  int logits_bf16;             /* 1: logits are BF16 */
  moe_route_scoring scoring;
  int num_groups, topk_groups, group_best;
  int renormalize;
  float scale;                 /* finite */
} moe_route_args;

moe_status moe_route(const moe_route_args* args, moe_stream_t stream);

/* --------------------------------------------------------------------------- verification of drafted tokens
 * A verification step feeds request b the rows [tok_start[b], tok_start[b+1]) of a step (moe_kv_tables): its last
 * token and then its drafted ones.  target row i is the model's distribution of the token that follows row i, and
 * draft row i the distribution that the token fed at row i + 1 was drawn from (draft NULL: drafts were certain,
 * their distribution one at the drafted token).  With n rows, request b has n - 1 drafts.
 *   Draft x at row i is accepted if uniform[i] * draft[i][x] < target[i][x] (compared exactly).  a = the
 *   number of drafts accepted before the first that is not.
 *   The token after them has the distribution r: max(target - draft, 0) of row a where its draft was refused
 *   (fp32 difference; with certain drafts target without the drafted token), target of row n - 1 where all were
 *   accepted; target of row a where nothing is left of r.  It is the first token whose cumulative sum of r
 *   exceeds uniform_next[b] times the sum of r, with sums in pairs of fp32 words, some 45 bits (a place within
 *   2^-32 of the sum beside a border between two tokens may fall to either).
 * Entries that are NaN or not above zero count as zero.  Rows need not sum to exactly one.
 *   accepted[b] = a;  next_token[b] = the token, -1 where r is zero throughout or its sum leaves fp32's range
 *   kept_len[b] = kv_len[b] - n + a + 1: the cached tokens that stay (the length to take the cache back to)
 * A request without rows gets 0, -1, kv_len[b]; so does one whose first row's slot is -1 (slot not NULL: the
 * step's tables refused it).  uniform and uniform_next are in [0, 1); what is not counts as the nearest end
 * (NaN as 0).  A drafted token outside [0, V) is refused and takes nothing from the target.  tok_start is clamped to [0, T].
 * Supported: 1 <= B <= 4096, 1 <= V <= 2^24, 0 <= T; strides in elements, not negative; target and draft of one type.
 * No output may share memory with an input or another output. */
typedef struct {
  const void* target;          /* fp32 or bf16 [T, V] */
  const void* draft;           /* same type [T, V], or NULL */
  const int32_t* tokens;       /* [T] tokens fed at each row */
  const int32_t* tok_start;    /* [B + 1] */
  const int32_t* kv_len;       /* [B] cached tokens, the step's included */
  const int32_t* slot;         /* [T] or NULL */
  const float* uniform;        /* [T] */
  const float* uniform_next;   /* [B] */
  int32_t* accepted;           /* [B] */
  int32_t* next_token;         /* [B] */
  int32_t* kept_len;           /* [B] */
  int64_t target_stride, draft_stride;
  int T, B, V;
  int bf16;                    /* 1: target and draft are BF16 */
} moe_verify_drafts_args;

moe_status moe_verify_drafts(const moe_verify_drafts_args* args, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_STEP_H_ */
