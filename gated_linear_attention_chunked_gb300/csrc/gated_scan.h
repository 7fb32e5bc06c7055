// gated_scan.h -- launch interface of the gated scan (gated_scan.cu).
#pragma once
#include "gla.h"
#include "kernels.h"

namespace gla {

struct ScanArgs {
  const void* x;  // [B,T,D]
  const void* g;  // [B,T,D], same type
  const float* init = nullptr;  // [B,D] or null (zeros)
  const int* lens = nullptr;    // [B] or null (all T)
  float* y = nullptr;           // [B,T,D]: written forward, read backward
  float* fin = nullptr;         // [B,D] or null
  const float* dy = nullptr;    // backward only, as are the rest
  const float* dfin = nullptr;
  float* dx = nullptr;
  float* dg = nullptr;
  float* dinit = nullptr;
  int B, T, D;
};
cudaError_t launch_scan(const ScanArgs& a, gla_dtype t, bool backward, int n_sm, DevCtl ctl,
                        cudaStream_t stream);

struct ScanDecodeArgs {
  float* state;               // [rows,D], or the pool [n_pages,pool_layers,D] with a page table
  const int* page = nullptr;  // [rows / L] or null
  int n_pages = 0, pool_layers = 1, layer0 = 0, L = 1;
  const void* x;              // [rows,D]
  const void* g;
  float* y;                   // [rows,D]
  long long rows;
  int D;
};
cudaError_t launch_scan_decode(const ScanDecodeArgs& a, gla_dtype t, DevCtl ctl,
                               cudaStream_t stream);

}  // namespace gla
