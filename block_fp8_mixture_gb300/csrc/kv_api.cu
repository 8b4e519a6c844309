// Host side of the paged cache's C ABI: argument checks, then one launch each.
#include <math.h>

#include <algorithm>

#include "kv_internal.h"

namespace moe {

static bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
static bool good(const void* p, size_t a) { return p != nullptr && aligned_to(p, a); }
static moe_status launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static moe_status check_cache(int Hkv, int D, int page_size, int num_pages) {
  if (Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0) return MOE_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (Hkv > 1024 || (long long)num_pages * page_size > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

static bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

// Whether an output of the tables shares memory with an input.  Every CTA reads the inputs
// for itself while others already write, so what is updated in place would differ from CTA to CTA.
static bool tables_overlap(const moe_kv_tables_args& a) {
  struct Range {
    const int32_t* p;
    long long n;
  };
  const long long B = a.B, cells = B * a.max_pages;
  constexpr int kOut = 11;
  const Range r[] = {{a.out_block_table, cells}, {a.out_free_list, a.num_pages}, {a.out_free_count, 1},
                     {a.kv_len, B}, {a.tok_start, B + 1}, {a.slot, a.max_tokens}, {a.position, a.max_tokens},
                     {a.request, a.max_tokens}, {a.run_tok, a.max_runs}, {a.run_len, a.max_runs}, {a.info, 4},
                     {a.cur_len, B}, {a.new_len, B}, {a.block_table, cells}, {a.free_list, a.num_pages},
                     {a.free_count, 1}};
  constexpr int kAll = sizeof(r) / sizeof(r[0]);
  for (int i = 0; i < kOut; ++i)
    for (int j = kOut; j < kAll; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(r[i].p), y = reinterpret_cast<uintptr_t>(r[j].p);
      if (r[i].n > 0 && r[j].n > 0 && x < y + 4 * r[j].n && y < x + 4 * r[i].n) return true;
    }
  return false;
}

// The workspace: status and counters, the prompts' plan, and parts, which the two kernels need one after the other.
struct AttentionSpace {
  size_t plan, parts, total;
};
static AttentionSpace attention_space(int D, int rows, bool prompts) {
  AttentionSpace w;
  w.plan = few_counter_bytes();
  w.parts = w.plan + (prompts ? prompt_plan_bytes() : 0);
  w.total = w.parts + std::max(few_parts_bytes(D, rows), prompts ? prompt_parts_bytes(D) : (size_t)0);
  return w;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_tables(const moe_kv_tables_args* a, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (a->B <= 0 || a->max_pages <= 0 || a->num_pages < 0 || a->max_tokens < 0 || a->max_runs < 0)
    return MOE_ERR_INVALID_ARG;
  if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->B > kMaxRequests || (long long)a->B * a->max_pages * a->page_size > 0x7FFFFFFFll ||
      (long long)a->num_pages * a->page_size > 0x7FFFFFFFll)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  // a stride of the grid past the end stays within 32 bits
  if (a->max_tokens > kMaxList || a->max_runs > kMaxList) return MOE_ERR_UNSUPPORTED_SHAPE;
  const void* need[] = {a->cur_len, a->new_len, a->block_table, a->free_count, a->out_block_table,
                        a->out_free_count, a->kv_len, a->tok_start, a->info};
  for (const void* p : need)
    if (!good(p, 4)) return MOE_ERR_INVALID_ARG;
  if (a->num_pages > 0 && (!good(a->free_list, 4) || !good(a->out_free_list, 4)))
    return MOE_ERR_INVALID_ARG;
  if (a->max_tokens > 0 && (!good(a->slot, 4) || !good(a->position, 4) || !good(a->request, 4)))
    return MOE_ERR_INVALID_ARG;
  if (a->max_runs > 0 && (!good(a->run_tok, 4) || !good(a->run_len, 4))) return MOE_ERR_INVALID_ARG;
  if (tables_overlap(*a)) return MOE_ERR_INVALID_ARG;
  return launched(launch_kv_tables(*a, (cudaStream_t)stream));
}

moe_status moe_rope_table(float* table, int max_pos, int rot_dim, double base, moe_rope_scale scaling,
                          double factor, double low, double high, int original_len, float magnitude,
                          moe_stream_t stream) {
  if (max_pos < 0 || rot_dim <= 0 || !(base > 1.0) || !isfinite(base) || !isfinite(magnitude))
    return MOE_ERR_INVALID_ARG;
  if (rot_dim % 16 || rot_dim > 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (scaling < MOE_ROPE_SCALE_NONE || scaling > MOE_ROPE_SCALE_RAMP) return MOE_ERR_INVALID_ARG;
  if (scaling != MOE_ROPE_SCALE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return MOE_ERR_INVALID_ARG;
  if (scaling == MOE_ROPE_SCALE_RAMP && (!(low < high) || !isfinite(low) || !isfinite(high) || original_len < 1))
    return MOE_ERR_INVALID_ARG;
  if (max_pos > 0 && !good(table, 16)) return MOE_ERR_INVALID_ARG;
  return launched(launch_rope_table(table, max_pos, rot_dim, base, scaling, factor, low, high,
                                    original_len, magnitude, (cudaStream_t)stream));
}

moe_status moe_rope_append(const moe_rope_append_args* a, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (a->T < 0 || a->Hq < 0 || a->max_runs < 0 || a->rot_dim < 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_cache(a->Hkv, a->D, a->page_size, a->num_pages);
  if (st != MOE_OK) return st;
  if (a->rot_dim % 16 || a->rot_dim > a->D || a->Hq > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
  // the units of the cache's write (run, head, K or V) and the last block's spare ones are counted in 32 bits
  if ((long long)a->max_runs * 2 * a->Hkv > 0xFFFFFFFFll - 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->layout < MOE_ROPE_HALF || a->layout > MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
  if (a->scale_fmt != MOE_SCALE_FP32 && a->scale_fmt != MOE_SCALE_FP32_POW2) return MOE_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_OK;
  if (a->rot_dim > 0 && (!good(a->rope, 16) || a->max_pos <= 0)) return MOE_ERR_INVALID_ARG;
  if (!good(a->position, 4) || !good(a->slot, 4)) return MOE_ERR_INVALID_ARG;
  if (a->max_runs > 0) {
    if (!good(a->run_tok, 4) || !good(a->run_len, 4) || !good(a->k, 16) || !good(a->v, 16) ||
        !good(a->k_codes, 16) || !good(a->v_codes, 16) || !good(a->k_scale, 4) || !good(a->v_scale, 4))
      return MOE_ERR_INVALID_ARG;
    if (!stride_ok(a->k_token_stride) || !stride_ok(a->k_head_stride) || !stride_ok(a->v_token_stride) ||
        !stride_ok(a->v_head_stride))
      return MOE_ERR_INVALID_ARG;
  }
  if (a->Hq > 0) {
    if (!good(a->q, 16) || !good(a->q_out, 16)) return MOE_ERR_INVALID_ARG;
    if (!stride_ok(a->q_token_stride) || !stride_ok(a->q_head_stride) || !stride_ok(a->qo_token_stride) ||
        !stride_ok(a->qo_head_stride))
      return MOE_ERR_INVALID_ARG;
  }
  return launched(launch_rope_append(*a, (cudaStream_t)stream));
}

size_t moe_kv_attention_workspace_bytes(int Hq, int Hkv, int D, int max_q) {
  if (Hq <= 0 || max_q <= 0 || check_cache(Hkv, D, 16, 0) != MOE_OK) return 0;
  if (Hq % Hkv || Hq / Hkv > kMaxGroup) return 0;
  const int G = Hq / Hkv, rows = few_rows(G, max_q);
  return attention_space(D, rows, (long long)G * max_q > rows).total;
}

moe_status moe_kv_attention(const moe_kv_attention_args* a, void* workspace, size_t workspace_bytes,
                            moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (a->T < 0 || a->B <= 0 || a->Hq <= 0 || a->max_pages <= 0 || a->max_q <= 0 || a->window < 0)
    return MOE_ERR_INVALID_ARG;
  const moe_status st = check_cache(a->Hkv, a->D, a->page_size, a->num_pages);
  if (st != MOE_OK) return st;
  if (a->Hq % a->Hkv || a->Hq / a->Hkv > kMaxGroup || a->B > kMaxRequests ||
      (long long)a->max_pages * a->page_size > 0x80000000ll - kTileTokens)   // tiles end within 32 bits
    return MOE_ERR_UNSUPPORTED_SHAPE;
  // shares of the few-row kernel's tiles are counted in 32 bits
  if (((long long)a->B * a->max_pages * a->page_size / kTileTokens + 4ll * a->B) * a->Hkv > 0x7FFFFFFFll - (1 << 20))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!(a->sm_scale > 0.0f) || !isfinite(a->sm_scale)) return MOE_ERR_INVALID_ARG;
  if (!good(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_kv_attention_workspace_bytes(a->Hq, a->Hkv, a->D, a->max_q))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (a->T == 0) return MOE_OK;
  if (!good(a->q, 16) || !good(a->out, 16) || !good(a->k_codes, 16) || !good(a->v_codes, 16) ||
      !good(a->k_scale, 4) || !good(a->v_scale, 4) || !good(a->block_table, 4) || !good(a->kv_len, 4) ||
      !good(a->tok_start, 4))
    return MOE_ERR_INVALID_ARG;
  if (!stride_ok(a->q_token_stride) || !stride_ok(a->q_head_stride) || !stride_ok(a->out_token_stride) ||
      !stride_ok(a->out_head_stride))
    return MOE_ERR_INVALID_ARG;
  if (a->num_pages == 0) return MOE_ERR_INVALID_ARG;
  moe_kv_attention_args c = *a;
  c.window = std::min(a->window, 1 << 30);               // positions + window stay within 32 bits
  const int G = a->Hq / a->Hkv, rows = few_rows(G, a->max_q);
  const bool prompts = (long long)G * a->max_q > rows;   // some request may have more rows than that
  if (prompts && !prompt_fits(a->T, G, a->B)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const AttentionSpace w = attention_space(a->D, rows, prompts);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* plan = prompts ? ws + w.plan : nullptr;
  cudaError_t err = launch_attn_few(c, rows, workspace, plan, ws + w.parts, (cudaStream_t)stream);
  if (err == cudaSuccess && prompts)
    err = launch_attn_prompt(c, static_cast<int*>(workspace), plan, ws + w.parts, (cudaStream_t)stream);
  return launched(err);
}

}  // extern "C"
