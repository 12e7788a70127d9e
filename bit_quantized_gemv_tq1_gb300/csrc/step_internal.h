// step_internal.h -- host-side launchers of a decoder step's remaining
// operators (norm, expert layer, sampling) and the structures they hand to
// their kernels.  Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv_internal.h"

namespace tq1 {

struct NormArgs {
  const float* x;      // [t][k]
  const void* delta;   // [t][k] of delta_type, or nullptr
  const float* gamma;  // [k], or nullptr: ones
  float* x_out;        // [t][k], or nullptr
  uint32_t* q8;        // [t][k/32] blocks of nine words, or nullptr
  void* y;             // [t][k] of y_type, or nullptr
  float eps;
  int delta_type, y_type;
  int k;
};
int launch_rms_norm(const NormArgs& a, int64_t t, unsigned* status, cudaStream_t s);

struct MoeLayerArgs {
  const uint8_t *gate, *up, *down;  // [n_experts] matrices, back to back
  const uint8_t* q8;                // [t][k/32] Q8_1
  const float* logits;              // [t][n_experts]
  const float* res;                 // [t][k], or nullptr
  void* out;                        // [t][k] of out_type
  int32_t* ids;                     // [t][top_k], or nullptr
  float* weights;                   // [t][top_k], or nullptr
  int n_experts, k, f, t, top_k;
  int renormalize, out_type;
  float scale;
};
// Whether the kernels have room for such rows in shared memory.
bool moe_layer_serves(int fmt, int64_t n_experts, int64_t k, int64_t f, int64_t pairs);
size_t moe_layer_workspace_bytes(int64_t k, int64_t f, int64_t t, int64_t top_k);
int launch_moe_layer(const MoeLayerArgs& a, int fmt, void* ws, unsigned* status, cudaStream_t s);

struct SampleArgs {
  const void* logits;  // [t][v] of type, rows ld elements apart
  int64_t ld;
  const float* temperature;  // [t] each, or nullptr
  const int32_t* top_k;
  const float *top_p, *min_p;
  const float* u;
  int32_t* ids;
  float* probs;  // [t], or nullptr
  int type, v;
};
int launch_sample(const SampleArgs& a, int64_t t, unsigned* status, cudaStream_t s);

}  // namespace tq1
