// rotary.h -- launch interface of the rotary positions (rotary.cu).
#pragma once
#include "gla.h"
#include "kernels.h"

namespace gla {

struct RotaryTensor {
  const void* x = nullptr;  // [B,T,heads,D], channels adjacent
  long long stride[3];      // elements from sequence to sequence, token to token, head to head
  void* y = nullptr;        // [B,T,heads,D] contiguous; may be x where x is contiguous too
  int heads = 0;
};
struct RotaryArgs {
  RotaryTensor q, k;        // k.heads == 0: no keys
  const unsigned long long* turns;  // [R / 2]
  const int* pos;           // [B,T] or null: a token's index in its sequence
  float scale;
  bool interleaved, inverse;
  int B, T, D, R;
  gla_dtype in_type, out_type;  // out_type: in_type or GLA_FP32
};
cudaError_t launch_rotary(const RotaryArgs& a, int n_sm, cudaStream_t stream);

}  // namespace gla
