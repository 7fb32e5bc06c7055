// api_layer.cu -- the C ABI of the operators around the mixer (include/gla.h): gated scan, layer
// norm and windowed attention.  Argument checks, then the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_checks.h"
#include "gated_scan.h"
#include "gla.h"
#include "kernels.h"
#include "layer_norm.h"
#include "window_attn.h"

namespace {

using namespace gla::api;

gla_status check_scan_sizes(int B, int T, int D, gla_dtype t) {
  if (B <= 0 || T <= 0 || D <= 0) return GLA_ERR_INVALID_ARG;
  if (!valid_dtype(t)) return GLA_ERR_UNSUPPORTED;
  // the grid: one CTA per sequence and 32 channels, times a cluster of at most 8
  if (T > kMaxInt - 4096 || (long long)B * ((D + 31ll) / 32) > kMaxInt / 8 ||
      (long long)B * T > (1ll << 40) / D)
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

gla_status check_window_batch(int B, int T, int H) {
  if (B <= 0 || T <= 0) return GLA_ERR_INVALID_ARG;
  if (T > (1 << 30) || (long long)B * T > (1ll << 32) / H ||
      (long long)B * ((T + 63ll) / 64) > kMaxInt / 4 / H)
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}
}  // namespace

extern "C" {

gla_status gla_gated_scan_fwd(const void* x, const void* g, gla_dtype in_dtype,
                              const float* init_state, const int* lens, float* y,
                              float* final_state, int B, int T, int D, cudaStream_t stream) {
  gla_status st = check_scan_sizes(B, T, D, in_dtype);
  if (st != GLA_OK) return st;
  if (!x || !g || !y) return GLA_ERR_INVALID_ARG;
  if (!aligned16(x, g, init_state, y, final_state) || !aligned4(lens)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::ScanArgs a;
  a.x = x; a.g = g; a.init = init_state; a.lens = lens; a.y = y; a.fin = final_state;
  a.B = B; a.T = T; a.D = D;
  return done(gla::launch_scan(a, in_dtype, false, sm_count(), ctl, stream));
}

gla_status gla_gated_scan_bwd(const void* x, const void* g, gla_dtype in_dtype, const float* y,
                              const float* dy, const float* init_state,
                              const float* d_final_state, const int* lens, float* dx, float* dg,
                              float* d_init_state, int B, int T, int D, cudaStream_t stream) {
  gla_status st = check_scan_sizes(B, T, D, in_dtype);
  if (st != GLA_OK) return st;
  if (!x || !g || !y || !dy || !dx || !dg) return GLA_ERR_INVALID_ARG;
  if (!aligned16(x, g, y, dy, init_state, d_final_state, dx, dg, d_init_state) || !aligned4(lens))
    return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::ScanArgs a;
  a.x = x; a.g = g; a.init = init_state; a.lens = lens; a.y = const_cast<float*>(y);
  a.dy = dy; a.dfin = d_final_state; a.dx = dx; a.dg = dg; a.dinit = d_init_state;
  a.B = B; a.T = T; a.D = D;
  return done(gla::launch_scan(a, in_dtype, true, sm_count(), ctl, stream));
}

gla_status gla_gated_scan_decode_step(float* state, const void* x, const void* g,
                                      gla_dtype in_dtype, float* y, long long N, int D,
                                      cudaStream_t stream) {
  if (N < 0 || D <= 0) return GLA_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype)) return GLA_ERR_UNSUPPORTED;
  if (N == 0) return GLA_OK;
  if (!state || !x || !g || !y) return GLA_ERR_INVALID_ARG;
  if (!aligned16(state, x, g, y)) return GLA_ERR_ALIGNMENT;
  if (N > (1ll << 38) / D) return GLA_ERR_UNSUPPORTED;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::ScanDecodeArgs a;
  a.state = state; a.x = x; a.g = g; a.y = y; a.rows = N; a.D = D;
  return done(gla::launch_scan_decode(a, in_dtype, ctl, stream));
}

gla_status gla_gated_scan_decode_step_paged(float* pool, const int* page, int n_active,
                                            int n_pages, int pool_layers, int layer0,
                                            const void* x, const void* g, gla_dtype in_dtype,
                                            float* y, int L, int D, cudaStream_t stream) {
  if (n_active < 0 || n_pages <= 0 || pool_layers <= 0 || L <= 0 || D <= 0 || layer0 < 0 ||
      L > pool_layers - layer0)
    return GLA_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype)) return GLA_ERR_UNSUPPORTED;
  if (n_active == 0) return GLA_OK;
  if (!pool || !page || !x || !g || !y) return GLA_ERR_INVALID_ARG;
  if (!aligned16(pool, x, g, y) || !aligned4(page)) return GLA_ERR_ALIGNMENT;
  if ((long long)n_active * L > (1ll << 38) / D ||
      (long long)n_pages * pool_layers > (1ll << 40) / D)
    return GLA_ERR_UNSUPPORTED;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::ScanDecodeArgs a;
  a.state = pool; a.page = page; a.n_pages = n_pages; a.pool_layers = pool_layers;
  a.layer0 = layer0; a.L = L; a.x = x; a.g = g; a.y = y;
  a.rows = (long long)n_active * L; a.D = D;
  return done(gla::launch_scan_decode(a, in_dtype, ctl, stream));
}

static gla_status check_layer_norm(gla_dtype x_dtype, gla_dtype out_dtype, long long n, int D) {
  if (n < 0 || D <= 0) return GLA_ERR_INVALID_ARG;
  if (!valid_dtype(x_dtype) || !(out_dtype == x_dtype || out_dtype == GLA_FP32) ||
      D > gla::kLayerNormMaxD || n > (1ll << 40) / D)
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

gla_status gla_layer_norm_fwd(const void* x, gla_dtype x_dtype, const float* weight,
                              const float* bias, float eps, void* y, gla_dtype y_dtype,
                              float* mean, float* rstd, long long n_tokens, int D,
                              cudaStream_t stream) {
  gla_status st = check_layer_norm(x_dtype, y_dtype, n_tokens, D);
  if (st != GLA_OK) return st;
  if (!(eps >= 0.f) || !(eps < 1e30f)) return GLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return GLA_OK;
  if (!x || !y) return GLA_ERR_INVALID_ARG;
  if (!aligned16(x, weight, bias, y, mean, rstd)) return GLA_ERR_ALIGNMENT;
  gla::LayerNormArgs a;
  a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
  a.x_type = x_dtype; a.out_type = y_dtype; a.eps = eps; a.n = n_tokens; a.D = D;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  return done(gla::launch_layer_norm_fwd(a, sm_count(), ctl, stream));
}

size_t gla_layer_norm_bwd_workspace_size(long long n_tokens, int D) {
  if (n_tokens <= 0 || D <= 0 || D > gla::kLayerNormMaxD) return 0;
  return gla::layer_norm_bwd_workspace_bytes(n_tokens, D, sm_count());
}

gla_status gla_layer_norm_bwd(const void* dy, gla_dtype dy_dtype, const void* x,
                              gla_dtype x_dtype, const float* weight, const float* mean,
                              const float* rstd, void* dx, float* d_weight, float* d_bias,
                              void* workspace, size_t workspace_bytes, long long n_tokens, int D,
                              cudaStream_t stream) {
  gla_status st = check_layer_norm(x_dtype, dy_dtype, n_tokens, D);
  if (st != GLA_OK) return st;
  if (n_tokens > 0 && (!dy || !x || !mean || !rstd || !dx)) return GLA_ERR_INVALID_ARG;
  if (!aligned16(dy, x, weight, mean, rstd, dx, d_weight, d_bias)) return GLA_ERR_ALIGNMENT;
  const size_t need = gla_layer_norm_bwd_workspace_size(n_tokens, D);
  if (n_tokens > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  if (!aligned256(workspace)) return GLA_ERR_ALIGNMENT;
  gla::LayerNormArgs a;
  a.dy = dy; a.x = x; a.weight = weight; a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd); a.dx = dx; a.dw = d_weight; a.db = d_bias;
  a.part = static_cast<float*>(workspace);
  a.x_type = x_dtype; a.out_type = dy_dtype; a.n = n_tokens; a.D = D;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  return done(gla::launch_layer_norm_bwd(a, sm_count(), ctl, stream));
}

gla_status gla_window_attn_fwd(const void* q, const void* k, const void* v, gla_dtype in_dtype,
                               const int* lens, int window, int sink, void* o,
                               gla_dtype out_dtype, float* lse, int B, int T, int H, int KV,
                               int dk, int dv, cudaStream_t stream) {
  gla_status st = check_window(in_dtype, out_dtype, window, sink, H, KV, dk, dv);
  if (st != GLA_OK || (st = check_window_batch(B, T, H)) != GLA_OK) return st;
  if (!q || !k || !v || !o) return GLA_ERR_INVALID_ARG;
  if (!aligned16(q, k, v, o) || !aligned4(lens, lse)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::WindowArgs a;
  a.q = q; a.k = k; a.v = v; a.lens = lens; a.B = B; a.T = T; a.H = H; a.KV = KV;
  a.window = std::min(window, T); a.sink = std::min(sink, T);
  a.in_type = in_dtype; a.out_type = out_dtype; a.o = o; a.lse = lse;
  return done(gla::launch_window_fwd(a, sm_count(), ctl, stream));
}

size_t gla_window_attn_bwd_workspace_size(int B, int T, int H, int KV, int window, int sink) {
  if (check_window(GLA_BF16, GLA_BF16, window, sink, H, KV, gla::kDK, gla::kDV) != GLA_OK ||
      check_window_batch(B, T, H) != GLA_OK)
    return 0;
  return gla::window_bwd_workspace_bytes(B, T, H, KV, std::min(window, T), std::min(sink, T));
}

gla_status gla_window_attn_bwd(const void* q, const void* k, const void* v, gla_dtype in_dtype,
                               const int* lens, int window, int sink, const void* o,
                               const long long* o_strides, gla_dtype out_dtype, const float* lse,
                               const void* dO, void* dq, void* dk, void* dv, void* workspace,
                               size_t workspace_bytes, int B, int T, int H, int KV, int dk_,
                               int dv_, cudaStream_t stream) {
  gla_status st = check_window(in_dtype, out_dtype, window, sink, H, KV, dk_, dv_);
  if (st != GLA_OK || (st = check_window_batch(B, T, H)) != GLA_OK) return st;
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return GLA_ERR_INVALID_ARG;
  if (!aligned16(q, k, v, o, dO, dq, dk, dv) || !aligned4(lens, lse)) return GLA_ERR_ALIGNMENT;
  gla::WindowArgs a;
  a.o_stride[0] = (long long)T * H * gla::kDV;
  a.o_stride[1] = (long long)H * gla::kDV;
  a.o_stride[2] = gla::kDV;
  for (int i = 0; o_strides && i < 3; ++i) {
    if (o_strides[i] < 0) return GLA_ERR_INVALID_ARG;
    if (o_strides[i] % (out_dtype == GLA_FP32 ? 4 : 8)) return GLA_ERR_ALIGNMENT;
    a.o_stride[i] = o_strides[i];
  }
  const size_t need = gla_window_attn_bwd_workspace_size(B, T, H, KV, window, sink);
  if (!workspace || workspace_bytes < need) return GLA_ERR_WORKSPACE;
  if (!aligned256(workspace)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  a.q = q; a.k = k; a.v = v; a.lens = lens; a.B = B; a.T = T; a.H = H; a.KV = KV;
  a.window = std::min(window, T); a.sink = std::min(sink, T);
  a.in_type = in_dtype; a.out_type = out_dtype; a.o = const_cast<void*>(o);
  a.lse = const_cast<float*>(lse); a.dO = dO; a.dq = dq; a.dk = dk; a.dv = dv;
  a.workspace = workspace;
  return done(gla::launch_window_bwd(a, sm_count(), ctl, stream));
}

gla_status gla_window_cache_fill(const void* k, const void* v, gla_dtype cache_dtype,
                                 const int* lens, void* pool_k, void* pool_v, const int* page,
                                 int n_pages, int pool_layers, int layer, int window, int sink,
                                 int B, int T, int KV, int dk, int dv, cudaStream_t stream) {
  gla_status st = check_window(cache_dtype, cache_dtype, window, sink, KV, KV, dk, dv);
  if (st != GLA_OK || (st = check_window_batch(B, T, KV)) != GLA_OK ||
      (st = check_window_pool(n_pages, pool_layers, layer, window, sink, KV)) != GLA_OK)
    return st;
  if (!k || !v || !pool_k || !pool_v || !page) return GLA_ERR_INVALID_ARG;
  if (!aligned16(k, v, pool_k, pool_v) || !aligned4(lens, page)) return GLA_ERR_ALIGNMENT;
  if ((long long)B * (window + sink) > 8 * kMaxInt) return GLA_ERR_UNSUPPORTED;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::WindowCache c{pool_k, pool_v, page, B, n_pages, pool_layers, layer, KV, window, sink,
                     cache_dtype};
  return done(gla::launch_window_fill(c, k, v, lens, T, ctl, stream));
}

size_t gla_window_attn_decode_workspace_size(int n_active, int H, int KV, int window, int sink) {
  if (check_window(GLA_BF16, GLA_BF16, window, sink, H, KV, gla::kDK, gla::kDV) != GLA_OK ||
      check_window_active(n_active, H, window, sink) != GLA_OK)
    return 0;
  return gla::window_decode_workspace_bytes(n_active, KV, H, window + sink, sm_count());
}

gla_status gla_window_attn_decode_step(void* pool_k, void* pool_v, gla_dtype cache_dtype,
                                       const int* page, const int* pos, int n_active, int n_pages,
                                       int pool_layers, int layer, int window, int sink,
                                       const void* q, const void* k, const void* v, void* o,
                                       gla_dtype out_dtype, void* workspace,
                                       size_t workspace_bytes, int H, int KV, int dk, int dv,
                                       cudaStream_t stream) {
  gla_status st = check_window(cache_dtype, out_dtype, window, sink, H, KV, dk, dv);
  if (st != GLA_OK || (st = check_window_active(n_active, H, window, sink)) != GLA_OK ||
      (st = check_window_pool(n_pages, pool_layers, layer, window, sink, KV)) != GLA_OK)
    return st;
  if (n_active == 0) return GLA_OK;
  if (!pool_k || !pool_v || !page || !pos || !q || !k || !v || !o) return GLA_ERR_INVALID_ARG;
  if (!aligned16(pool_k, pool_v, q, k, v, o) || !aligned4(page, pos)) return GLA_ERR_ALIGNMENT;
  const size_t need = gla_window_attn_decode_workspace_size(n_active, H, KV, window, sink);
  if (need && (!workspace || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  if (need && !aligned256(workspace)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::WindowDecodeArgs a;
  a.c = {pool_k, pool_v, page, n_active, n_pages, pool_layers, layer, KV, window, sink,
         cache_dtype};
  a.pos = pos; a.q = q; a.k = k; a.v = v; a.o = o; a.out_type = out_dtype; a.H = H;
  a.workspace = workspace;
  return done(gla::launch_window_decode(a, sm_count(), ctl, stream));
}

}  // extern "C"
