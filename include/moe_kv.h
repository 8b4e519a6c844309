/*
 * moe_kv.h -- C ABI of the attention half of a serving step beside the block-FP8 experts: a paged
 * key/value cache held as E4M3 codes with one scale per block of tokens and head, the tables that
 * address it, the rotary embedding that feeds it and the attention that reads it.
 *
 * The conventions are those of moe_fp8.h: tensor arguments are device pointers owned by the caller;
 * nothing is allocated, the host is not synchronised, all work goes to `stream` (so a step can be
 * captured in a CUDA graph); arguments are validated on the host before anything is launched.
 *
 * The cache.  A page holds `page_size` consecutive tokens of one request for all key/value heads:
 *   k_codes, v_codes  uint8 E4M3 [num_pages, Hkv, page_size, D]   (16-byte aligned)
 *   k_scale, v_scale  fp32       [num_pages, Hkv]                 (a code c stands for c * scale)
 * page_size is 16, 32, 64 or 128; D is 64 or 128; num_pages * page_size < 2^31.
 * Token j of request b is row j % page_size of page block_table[b][j / page_size].
 */
#ifndef MOE_KV_H_
#define MOE_KV_H_

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ block tables and slot maps
 * Takes every request from cur_len[b] cached tokens to new_len[b]: growth appends new_len - cur_len
 * tokens, a smaller new_len gives pages back (0 when the request has finished).  All tables are
 * written to a second set of buffers, so a step in flight on another stream keeps reading the first.
 *
 * With pages(n) = ceil(n / page_size):
 *  - Released pages, table entries [pages(new), pages(cur)), are pushed on the free stack in request
 *    order.  Then requests are granted pages(new) - pages(cur) pages each, in request order, while
 *    the sum of the needs so far fits the stack; once one does not fit, later requests that need
 *    pages are refused too (a request that needs none never is).  The granted pages are the topmost
 *    entries of the stack, handed out in stored order, so growing and giving back restores the stack.
 *  - A request whose new_len exceeds max_pages * page_size is refused and adds no tokens.
 *  - While the added tokens so far fit max_tokens; once a request's do not, it and later requests that
 *    add tokens are refused (their tokens are counted all the same: info[0] above max_tokens shows it).
 *  - kv_len[b] = new_len[b], or cur_len[b] for a refused request.
 *  - The added tokens of all requests are numbered in request order: those of request b are
 *    [tok_start[b], tok_start[b+1]).  Token t: request[t] = b, position[t] = its place in the
 *    request, slot[t] = page * page_size + row, or -1 when the request was refused (nothing is written to the
 *    cache for it, and its rows of the attention's output hold nothing of use).  Entries from the
 *    total up to max_tokens read slot -1, position 0, request -1 (a captured graph can run on them).
 *  - A run is the added tokens of one request that share a page: run r is tokens
 *    [run_tok[r], run_tok[r] + run_len[r]); unused entries are 0, 0.
 *  - info = {added tokens, runs, refused requests, granted pages}.
 * Table entries past pages(kv_len[b]) are -1.  cur_len outside [0, max_pages * page_size] and a
 * negative new_len are clamped.
 * No output may share memory with an input (kv_len is not cur_len): MOE_ERR_INVALID_ARG.
 * Supported: 1 <= B <= 4096, B * max_pages * page_size < 2^31, max_tokens and max_runs below 2^31 - 2^20.
 * max_runs must cover the runs:
 * min(max_tokens, max_tokens / page_size + 2 * B) always does (runs past max_runs are not listed). */
typedef struct {
  const int32_t* cur_len;      /* [B] */
  const int32_t* new_len;      /* [B] */
  const int32_t* block_table;  /* [B, max_pages] */
  const int32_t* free_list;    /* [num_pages], the stack: entries [0, free_count) are free */
  const int32_t* free_count;   /* [1] */
  int32_t* out_block_table;    /* [B, max_pages] */
  int32_t* out_free_list;      /* [num_pages] */
  int32_t* out_free_count;     /* [1] */
  int32_t* kv_len;             /* [B] */
  int32_t* tok_start;          /* [B + 1] */
  int32_t* slot;               /* [max_tokens] */
  int32_t* position;           /* [max_tokens] */
  int32_t* request;            /* [max_tokens] */
  int32_t* run_tok;            /* [max_runs] */
  int32_t* run_len;            /* [max_runs] */
  int32_t* info;               /* [4] */
  int B, max_pages, num_pages, page_size, max_tokens, max_runs;
} moe_kv_tables_args;

moe_status moe_kv_tables(const moe_kv_tables_args* args, moe_stream_t stream);

/* ------------------------------------------------------------------------------ rotary positions
 * Layouts: HALF rotates pairs (i, i + rot/2), INTERLEAVED pairs (2i, 2i + 1), i < rot/2; values from
 * rot_dim on are left as they are. */
typedef enum { MOE_ROPE_HALF = 0, MOE_ROPE_INTERLEAVED = 1 } moe_rope_layout;

/* Frequencies f_i = base^(-2i / rot_dim), scaled for long contexts:
 * NONE    as they are;
 * LINEAR  f_i / factor (positions interpolated);
 * RAMP    f_i * (w + (1 - w) / factor), w = clamp((r_i - low) / (high - low), 0, 1) with
 *         r_i = original_len * f_i / 2 pi, the turns that the pair makes over the original context:
 *         fast pairs keep their frequency, slow ones are interpolated. */
typedef enum { MOE_ROPE_SCALE_NONE = 0, MOE_ROPE_SCALE_LINEAR = 1, MOE_ROPE_SCALE_RAMP = 2 } moe_rope_scale;

/* Writes table fp32 [max_pos, rot_dim / 2, 2]: magnitude * (cos, sin) of position * f_i, evaluated in
 * 64 bits and rounded once (an fp32 angle at position 10^6 would be off by 0.06).
 * rot_dim: a multiple of 16, at most 128; base > 1; factor >= 1; low < high; original_len >= 1. */
moe_status moe_rope_table(float* table, int max_pos, int rot_dim, double base, moe_rope_scale scaling,
                          double factor, double low, double high, int original_len, float magnitude,
                          moe_stream_t stream);

/* ------------------------------------------------------- rotary positions and the cache's write
 * Rotates q and k by each token's position (fp32 products and sums, rounded separately), writes the
 * rotated q as BF16 and appends the rotated k and v to the cache, page by page over the runs of
 * moe_kv_tables.  For each run's page and head, over the new tokens of that page:
 *   s = max(amax / 448, 1 / (448 * 512)), rounded up to a power of two with MOE_SCALE_FP32_POW2;
 *   if the page holds older tokens of the request: s = max(s, the page's scale), and where that
 *   raises the scale the older codes become q8(c * RN(scale / s));
 *   new codes q8(RN(x / s)), q8 = round to nearest even E4M3, saturating (as moe_quant_act).
 * Rows of the page past the new tokens are not touched.  Tokens with slot -1 write nothing.
 * q_out may be q itself.  Strides are in elements, multiples of 8; values of a head are contiguous.
 * position[t] must be below max_pos (it is clamped).  rot_dim 0 (rope NULL): no rotation.
 * Infinite inputs saturate the page's scale; a NaN becomes the NaN code and does not enter amax.
 * max_runs * 2 * Hkv < 2^32 - 8, else MOE_ERR_UNSUPPORTED_SHAPE.
 * scale_fmt: MOE_SCALE_FP32 or MOE_SCALE_FP32_POW2.  Hq may be 0 (q and q_out NULL): cache write only. */
typedef struct {
  const void* q;           /* bf16 [T, Hq, D] */
  const void* k;           /* bf16 [T, Hkv, D] */
  const void* v;           /* bf16 [T, Hkv, D] */
  void* q_out;             /* bf16 [T, Hq, D] */
  const float* rope;       /* [max_pos, rot_dim / 2, 2] */
  const int32_t* position; /* [T] */
  const int32_t* slot;     /* [T] */
  const int32_t* run_tok;  /* [max_runs] */
  const int32_t* run_len;  /* [max_runs] */
  void* k_codes;
  void* v_codes;
  float* k_scale;
  float* v_scale;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
  int64_t qo_token_stride, qo_head_stride;
  int T, Hq, Hkv, D, page_size, num_pages, max_runs;
  int rot_dim, max_pos;
  moe_rope_layout layout;
  moe_scale_fmt scale_fmt;
} moe_rope_append_args;

moe_status moe_rope_append(const moe_rope_append_args* args, moe_stream_t stream);

/* ------------------------------------------------------------------------------------ attention
 * Query token i of request b (row tok_start[b] + i of q, i < n = tok_start[b+1] - tok_start[b]) stands
 * at position p = kv_len[b] - n + i and sees the cached tokens j <= p, and with window > 0 only
 * j > p - window.  out = sum_j softmax_j(sm_scale * q . k_j) v_j per head; head h reads key/value head
 * h / (Hq / Hkv).  A row that sees nothing (kv_len[b] < n, or kv_len[b] = 0) is zero.  Rows of q past
 * tok_start[B] are neither read nor written.
 * Scores, softmax statistics and sums are fp32; out is rounded once to BF16.  On the way into the matrix
 * products a row of q is rounded to 2^-15 of its largest value (2^-17 with many query rows), and a probability
 * times the V scale of its page to 11 bits, down to 2^-13 of the largest of its row; from there the error is
 * absolute, at most 2^-25 of that largest one (2^-29 with many query rows).
 * Scales are not negative; a V scale below 1e-30 counts as 1e-30.
 * A row that sees something and whose q holds an infinity or a NaN is NaN.
 * max_q is an upper bound of the n (requests with more tokens are cut to max_q tokens by the caller's
 * mistake: their later rows are left unwritten).
 * A NaN among the codes and scales of the tokens that a row sees makes the row NaN (a V code: that value of
 * it) and may reach other rows of the same request; codes outside every row's view (stale rows of the last
 * page, other pages) never matter.
 * Supported: 1 <= num_pages, Hq % Hkv == 0, Hq / Hkv <= 64, sm_scale finite and > 0, 1 <= B <= 4096, max_q >= 1.
 * Strides in elements, multiples of 8.
 * Parts of a long request are kept in the workspace on the way: FP32 with few query rows, FP32
 * without the last 8 bits (with whole FP32 statistics) with many: 2^-15, where the rounding of out is 2^-8.
 * MOE_ERR_INVALID_ARG with num_pages 0; MOE_ERR_UNSUPPORTED_SHAPE where the work would pass 32-bit counts:
 * max_pages * page_size > 2^31 - 128, T * (Hq / Hkv) / 512 + B > 65536 with more rows than 64 in a request, or
 * Hkv * (B * max_pages * page_size / 128 + 4 * B) >= 2^31 - 2^20.
 * The workspace (256-byte aligned) starts with the int32 status word that moe_last_device_status
 * reads; the caller zeroes the workspace once after allocating it, and again after a call whose status
 * is MOE_ERR_DEVICE_TIMEOUT (the status stays, and counters may be left half way).  One workspace serves
 * one stream at a time. */
typedef struct {
  const void* q;               /* bf16 [T, Hq, D] */
  const void* k_codes;
  const void* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;  /* [B, max_pages] */
  const int32_t* kv_len;       /* [B] */
  const int32_t* tok_start;    /* [B + 1] */
  void* out;                   /* bf16 [T, Hq, D] */
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
  int T, B, Hq, Hkv, D, page_size, num_pages, max_pages, max_q, window;
  float sm_scale;
} moe_kv_attention_args;

/* Bytes of workspace moe_kv_attention needs for these heads (0 if unsupported). */
size_t moe_kv_attention_workspace_bytes(int Hq, int Hkv, int D, int max_q);

moe_status moe_kv_attention(const moe_kv_attention_args* args, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_KV_H_ */
