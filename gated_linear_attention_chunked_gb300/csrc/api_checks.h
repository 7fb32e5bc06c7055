// api_checks.h -- argument checks shared by the C ABI's translation units of the operators around the
// mixer.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "gla.h"
#include "kernels.h"

namespace gla {
namespace api {

constexpr long long kMaxInt = (1ll << 31) - 1;

template <class... P>
bool aligned16(P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 15u) == 0;
}
template <class... P>
bool aligned4(P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline bool valid_dtype(gla_dtype t) { return t == GLA_BF16 || t == GLA_FP16 || t == GLA_FP32; }

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

inline gla_status done(cudaError_t e) { return e == cudaSuccess ? GLA_OK : GLA_ERR_CUDA; }

// Sizes and types of the windowed attention; the tensors' element counts stay below 2^40.
inline gla_status check_window(gla_dtype in, gla_dtype out, int window, int sink, int H, int KV,
                               int dk, int dv) {
  if (H <= 0 || KV <= 0 || H % KV != 0 || window <= 0 || sink < 0) return GLA_ERR_INVALID_ARG;
  if (dk != kDK || dv != kDV || (in != GLA_BF16 && in != GLA_FP16) || (out != in && out != GLA_FP32))
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}
// Slots of a page and of the whole pool.
inline gla_status check_window_pool(int n_pages, int pool_layers, int layer, int window, int sink,
                                    int KV) {
  if (n_pages <= 0 || pool_layers <= 0 || layer < 0 || layer >= pool_layers)
    return GLA_ERR_INVALID_ARG;
  if (window > (1 << 30) - sink || KV > (1 << 16) ||
      (long long)n_pages * pool_layers > (1ll << 40) / ((long long)(window + sink) * KV))
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}
inline gla_status check_window_active(int n_active, int H, int window, int sink) {
  if (n_active < 0) return GLA_ERR_INVALID_ARG;
  // CTAs: at most 64 parts of each (sequence, head)
  if (window > (1 << 30) - sink || (long long)n_active * H > kMaxInt / 64)
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

}  // namespace api
}  // namespace gla
