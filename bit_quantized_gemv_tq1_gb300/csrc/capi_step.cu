// capi_step.cu -- the extern "C" entry points of the operators that complete
// a decoder's step (norm, expert layer, sampling; declared in include/tq1.h):
// host-side argument checks and launches.
#include <cmath>

#include "../../include/tq1.h"
#include "step_internal.h"
#include "tq1_device.cuh"
#include "tq1_internal.h"

using namespace tq1;

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 24;
constexpr int64_t kMaxNormK = int64_t{1} << 20;
constexpr int64_t kMaxVocabulary = int64_t{1} << 19;  // weights of 45 bits add up in 64
constexpr int64_t kMaxMoeK = int64_t{1} << 16;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 32;
constexpr int64_t kMaxPairs = 4096;

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool is_type(int d) { return d == TQ1_F32 || d == TQ1_F16 || d == TQ1_BF16; }

int moe(const void* gate, const void* up, const void* down, int64_t n_experts, const void* q8, const float* logits,
        const float* res, void* out, int out_dtype, int32_t* ids, float* weights, int64_t k, int64_t f, int64_t t,
        int64_t top_k, int renormalize, float scale, void* ws, size_t ws_bytes, void* stream, int fmt) {
  if (t < 0 || k <= 0 || f <= 0 || k % kQK != 0 || f % kQK != 0 || n_experts <= 0 || top_k <= 0 || top_k > n_experts ||
      !std::isfinite(scale))
    return TQ1_ERR_SHAPE;
  if (!is_type(out_dtype) || k > kMaxMoeK || f > kMaxMoeK || n_experts > kMaxExperts || top_k > kMaxTopK || t > kMaxPairs ||
      t * top_k > kMaxPairs || !moe_layer_serves(fmt, n_experts, k, f, t * top_k))
    return TQ1_ERR_UNSUPPORTED;
  if (t == 0) return TQ1_OK;
  if (!gate || !up || !down || !q8 || !logits || !out || !ws) return TQ1_ERR_NULL;
  if (off16(gate) || off16(up) || off16(down) || off16(q8) || off4(logits) || off16(res) || off16(out) || off4(ids) ||
      off4(weights) || off16(ws))
    return TQ1_ERR_ALIGN;
  if (ws_bytes < moe_layer_workspace_bytes(k, f, t, top_k)) return TQ1_ERR_WORKSPACE;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  const MoeLayerArgs a = {static_cast<const uint8_t*>(gate),
                          static_cast<const uint8_t*>(up),
                          static_cast<const uint8_t*>(down),
                          static_cast<const uint8_t*>(q8),
                          logits,
                          res,
                          out,
                          ids,
                          weights,
                          static_cast<int>(n_experts),
                          static_cast<int>(k),
                          static_cast<int>(f),
                          static_cast<int>(t),
                          static_cast<int>(top_k),
                          renormalize != 0,
                          out_dtype,
                          scale};
  return launch_moe_layer(a, fmt, ws, st, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int tq1_rms_norm(const float* x, const void* delta, int delta_dtype, const float* gamma, float eps, float* x_out, void* q8,
                 void* y, int y_dtype, int64_t t, int64_t k, void* stream) {
  if (t < 0 || k <= 0 || k % kQK8 != 0 || !(eps >= 0) || !std::isfinite(eps)) return TQ1_ERR_SHAPE;
  if ((delta && !is_type(delta_dtype)) || (y && !is_type(y_dtype)) || t > kMaxRows || k > kMaxNormK) return TQ1_ERR_UNSUPPORTED;
  if (t == 0) return TQ1_OK;
  if (!x || (!q8 && !y)) return TQ1_ERR_NULL;
  if (off16(x) || off16(delta) || off16(gamma) || off16(x_out) || off16(q8) || off16(y)) return TQ1_ERR_ALIGN;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  const NormArgs a = {x, delta, gamma, x_out, static_cast<uint32_t*>(q8), y, eps, delta_dtype, y_dtype, static_cast<int>(k)};
  return launch_rms_norm(a, t, st, static_cast<cudaStream_t>(stream));
}

size_t tq1_moe_workspace_size(int64_t n_experts, int64_t k, int64_t f, int64_t t, int64_t top_k) {
  if (t < 0 || k <= 0 || f <= 0 || k % kQK != 0 || f % kQK != 0 || n_experts <= 0 || top_k <= 0 || top_k > n_experts ||
      k > kMaxMoeK || f > kMaxMoeK || n_experts > kMaxExperts || top_k > kMaxTopK || t > kMaxPairs || t * top_k > kMaxPairs)
    return 0;
  if (!moe_layer_serves(kFmtTq1, n_experts, k, f, t * top_k) && !moe_layer_serves(kFmtTq2, n_experts, k, f, t * top_k)) return 0;
  return moe_layer_workspace_bytes(k, f, t, top_k);
}

int tq1_moe(const void* gate, const void* up, const void* down, int64_t n_experts, const void* q8, const float* logits,
            const float* res, void* out, int out_dtype, int32_t* ids, float* weights, int64_t k, int64_t f, int64_t t,
            int64_t top_k, int renormalize, float scale, void* ws, size_t ws_bytes, void* stream) {
  return moe(gate, up, down, n_experts, q8, logits, res, out, out_dtype, ids, weights, k, f, t, top_k, renormalize, scale, ws,
             ws_bytes, stream, kFmtTq1);
}

int tq2_moe(const void* gate, const void* up, const void* down, int64_t n_experts, const void* q8, const float* logits,
            const float* res, void* out, int out_dtype, int32_t* ids, float* weights, int64_t k, int64_t f, int64_t t,
            int64_t top_k, int renormalize, float scale, void* ws, size_t ws_bytes, void* stream) {
  return moe(gate, up, down, n_experts, q8, logits, res, out, out_dtype, ids, weights, k, f, t, top_k, renormalize, scale, ws,
             ws_bytes, stream, kFmtTq2);
}

int tq1_sample(const void* logits, int dtype, int64_t ld, int64_t t, int64_t v, const float* temperature, const int32_t* top_k,
               const float* top_p, const float* min_p, const float* u, int32_t* ids, float* probs, void* stream) {
  if (t < 0 || v <= 0 || ld < v) return TQ1_ERR_SHAPE;
  if (!is_type(dtype) || v > kMaxVocabulary || t > (int64_t{1} << 20) || ld > (int64_t{1} << 40)) return TQ1_ERR_UNSUPPORTED;
  if (t == 0) return TQ1_OK;
  if (!logits || !u || !ids) return TQ1_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == TQ1_F32 ? 3u : 1u)) != 0 || off4(temperature) || off4(top_k) ||
      off4(top_p) || off4(min_p) || off4(u) || off4(ids) || off4(probs))
    return TQ1_ERR_ALIGN;
  unsigned* st = status_word();
  if (!st) return TQ1_ERR_CUDA;
  const SampleArgs a = {logits, ld, temperature, top_k, top_p, min_p, u, ids, probs, dtype, static_cast<int>(v)};
  return launch_sample(a, t, st, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
