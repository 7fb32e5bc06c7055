// layer_norm.h -- launch interface of the layer norm (layer_norm.cu).
#pragma once
#include "gla.h"
#include "kernels.h"

namespace gla {

constexpr int kLayerNormMaxD = 16384;

struct LayerNormArgs {
  const void* x;                 // [n,D] x_type
  const float* weight = nullptr; // [D] or null (ones)
  const float* bias = nullptr;   // [D] or null (zeros)
  float* mean = nullptr;         // [n]: written forward (may be null), read backward
  float* rstd = nullptr;
  void* y = nullptr;             // forward: [n,D] out_type
  const void* dy = nullptr;      // backward: [n,D] out_type, as dx
  void* dx = nullptr;
  float* dw = nullptr;           // [D] or null
  float* db = nullptr;
  float* part = nullptr;         // partial sums of dw, db
  gla_dtype x_type, out_type;    // out_type: x_type or GLA_FP32
  float eps = 0.f;
  long long n;
  int D;
};
size_t layer_norm_bwd_workspace_bytes(long long n, int D, int n_sm);
cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, int n_sm, DevCtl ctl,
                                  cudaStream_t stream);
cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, int n_sm, DevCtl ctl,
                                  cudaStream_t stream);

}  // namespace gla
