// window_attn.h -- launch interface of the windowed attention (window_fwd.cu, window_bwd.cu,
// window_decode.cu).
#pragma once
#include "gla.h"
#include "kernels.h"

namespace gla {

struct WindowArgs {
  const void* q;  // [B,T,H,96] 16-bit
  const void* k;  // [B,T,KV,96]
  const void* v;  // [B,T,KV,192]
  const int* lens = nullptr;  // [B] or null (all T)
  int B, T, H, KV, window, sink;
  gla_dtype in_type, out_type;  // out_type (o, dq, dk, dv): in_type or GLA_FP32
  void* o = nullptr;            // [B,T,H,192]
  float* lse = nullptr;         // [B,H,T]
  // gradient
  long long o_stride[3];        // elements from sequence to sequence, token to token, head to head
  const void* dO = nullptr;     // [B,T,H,192] in_type
  void* dq = nullptr;
  void* dk = nullptr;
  void* dv = nullptr;
  void* workspace = nullptr;
};
cudaError_t launch_window_fwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream);
size_t window_bwd_workspace_bytes(int B, int T, int H, int KV, int window, int sink);
cudaError_t launch_window_bwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream);

// Caches: [n_pages, pool_layers, sink + window slots, KV, 96 | 192], one page per sequence.
struct WindowCache {
  void* k;
  void* v;
  const int* page;  // [n]
  int n, n_pages, pool_layers, layer, KV, window, sink;
  gla_dtype type;
};
struct WindowDecodeArgs {
  WindowCache c;
  const int* pos;   // [n] position of the token
  const void* q;    // [n,H,96]
  const void* k;    // [n,KV,96]
  const void* v;    // [n,KV,192]
  void* o;          // [n,H,192]
  gla_dtype out_type;
  int H;
  void* workspace;
};
// For the parts of what is cut (window_decode.cu); 0: nothing is.
size_t window_decode_workspace_bytes(int n, int KV, int H, int slots, int n_sm);
cudaError_t launch_window_decode(const WindowDecodeArgs& a, int n_sm, DevCtl ctl,
                                 cudaStream_t stream);
// The last tokens of prompts into their pages: k, v [n,T,KV,d], lens [n] or null.
cudaError_t launch_window_fill(const WindowCache& c, const void* k, const void* v,
                               const int* lens, int T, DevCtl ctl, cudaStream_t stream);

}  // namespace gla
