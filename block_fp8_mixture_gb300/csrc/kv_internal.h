// Internal declarations of the paged 8-bit cache: limits, kernel parameter blocks and launchers.
#pragma once

#include "../../include/moe_kv.h"
#include "moe_internal.h"

namespace moe {

constexpr int kMaxRequests = 4096;
constexpr int kMaxList = 0x7FFFFFFF - (1 << 20);   // entries of a step's token or run list
constexpr int kMaxGroup = 64;          // query heads per key/value head
constexpr int kTileTokens = 128;       // cached tokens that the attention kernels take at a time

cudaError_t launch_kv_tables(const moe_kv_tables_args& a, cudaStream_t s);
cudaError_t launch_rope_table(float* table, int max_pos, int rot, double base, int scaling,
                              double factor, double low, double high, int original_len,
                              float magnitude, cudaStream_t s);
cudaError_t launch_rope_append(const moe_rope_append_args& a, cudaStream_t s);
// Requests with few query rows, n <= few_rows / (Hq / Hkv) tokens.  plan (nullptr: the call has no
// longer requests) receives the blocks of the others.
int few_rows(int G, int max_q);
size_t few_counter_bytes();
size_t few_parts_bytes(int D, int rows);
cudaError_t launch_attn_few(const moe_kv_attention_args& a, int rows, void* workspace, void* plan, void* parts,
                            cudaStream_t s);
// The others, right after launch_attn_few on the same stream, whose parts are no longer needed then.
bool prompt_fits(int T, int G, int B);
size_t prompt_plan_bytes();
size_t prompt_parts_bytes(int D);
cudaError_t launch_attn_prompt(const moe_kv_attention_args& a, int* status, void* plan, void* parts, cudaStream_t s);

}  // namespace moe
