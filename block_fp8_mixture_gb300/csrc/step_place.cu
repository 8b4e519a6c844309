// Rows that are quantized already, placed for the experts.
#include "step_device.cuh"

namespace moe {

// Each token's codes and scales go to the workspace rows of its live pairs: what k_quant_act does behind its
// quantization.  A thread moves 16 codes; the eight of a group share its scale.  Bound by HBM: H + 4 H / 128 bytes a token read,
// topk times as many written: 4096 x 7168 for 8 experts each 47 us, 5.8 TB/s (quantizing the BF16 rows 54 us).
constexpr int kPlaceThreads = 256;
constexpr int kPlaceBytes = 16;

__global__ void __launch_bounds__(kPlaceThreads) k_place_act(PlaceParams p) {
  const int vectors = p.H / kPlaceBytes;
  const long at = (long)blockIdx.x * kPlaceThreads + threadIdx.x;
  const long t = at / vectors;
  const int v = (int)(at % vectors), g = v / (kGroup / kPlaceBytes);
  grid_dep_wait();
  grid_dep_launch_dependents();
  int n = p.M_cap;
  if (p.d_num_tokens != nullptr) n = min(max(*p.d_num_tokens, 0), p.M_cap);
  if (t >= n) return;
  const uint4 codes = *reinterpret_cast<const uint4*>(p.codes + t * p.codes_stride + v * kPlaceBytes);
  const bool first = v % (kGroup / kPlaceBytes) == 0;
  const int64_t scale = g * p.scales_stride + t;
  const float s32 = first && !p.ue8m0 ? static_cast<const float*>(p.scales)[scale] : 0.0f;
  const uint8_t s8 = first && p.ue8m0 ? static_cast<const uint8_t*>(p.scales)[scale] : 0;
  for (int j = 0; j < p.topk; ++j) {
    const int row = p.pair_row[t * p.topk + j];
    if (row < 0) continue;
    *reinterpret_cast<uint4*>(p.a_q + (size_t)row * p.H + v * kPlaceBytes) = codes;
    if (!first) continue;
    const size_t to = (size_t)g * p.R_cap + row;
    if (p.ue8m0)
      static_cast<uint8_t*>(p.a_s)[to] = s8;
    else
      static_cast<float*>(p.a_s)[to] = s32;
  }
}

cudaError_t launch_place(const PlaceParams& p, cudaStream_t s) {
  const long threads = (long)p.M_cap * (p.H / kPlaceBytes), blocks = (threads + kPlaceThreads - 1) / kPlaceThreads;
  if (blocks == 0) return cudaSuccess;
  return launch_pdl(k_place_act, dim3((unsigned)blocks), dim3(kPlaceThreads), 0, s, p);
}

}  // namespace moe
