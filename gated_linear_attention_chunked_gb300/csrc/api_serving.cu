// api_serving.cu -- the C ABI of serving with the windowed attention (include/gla.h): rotary
// positions, packed tokens into pages of 16 and 8 bits, chunks of tokens and single ones over them.
// Argument checks, then the launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "rotary.h"
#include "window_serve.h"

namespace {

using namespace gla::api;

size_t size_of(gla_dtype t) { return t == GLA_FP32 ? 4 : 2; }

gla_status check_packed(int n, int n_tokens, int H) {
  if (n < 0 || n_tokens < 0) return GLA_ERR_INVALID_ARG;
  // (sequences and tokens are counted together as tiles of rows)
  if (n_tokens > (1 << 30) || (long long)n + n_tokens > kMaxInt / 64 / H) return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

}  // namespace

extern "C" {

gla_status gla_rotary_turns(int R, double base, gla_rotary_scaling scaling, double factor,
                            double context, double low, double high, unsigned long long* turns) {
  if (R < 2 || R % 2 || !turns || !(base > 1) || !std::isfinite(base)) return GLA_ERR_INVALID_ARG;
  if (scaling != GLA_ROTARY_PLAIN && scaling != GLA_ROTARY_LINEAR && scaling != GLA_ROTARY_BASE &&
      scaling != GLA_ROTARY_PARTS)
    return GLA_ERR_UNSUPPORTED;
  if (scaling != GLA_ROTARY_PLAIN && (!(factor >= 1) || !std::isfinite(factor)))
    return GLA_ERR_INVALID_ARG;
  if (scaling == GLA_ROTARY_PARTS &&
      (!(context > 0) || !(low >= 0) || !(high > low) || !std::isfinite(context + high)))
    return GLA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  if (scaling == GLA_ROTARY_BASE && R > 2) base *= std::pow(factor, (double)R / (R - 2));
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R) / two_pi;  // turns per position
    if (scaling == GLA_ROTARY_LINEAR) f /= factor;
    if (scaling == GLA_ROTARY_PARTS) {
      const double keep = std::min(std::max((context * f - low) / (high - low), 0.0), 1.0);
      f = f * keep + f / factor * (1 - keep);
    }
    turns[i] = (unsigned long long)std::nearbyint(std::ldexp(f, 64));
  }
  return GLA_OK;
}

gla_status gla_rotary(const void* q, const long long* q_strides, void* q_out, int H, const void* k,
                      const long long* k_strides, void* k_out, int KV, gla_dtype in_dtype,
                      gla_dtype out_dtype, const unsigned long long* turns, const int* pos,
                      float scale, int interleaved, int inverse, int B, int T, int D, int R,
                      cudaStream_t stream) {
  if (H <= 0 || KV < 0 || B < 0 || T < 0 || D <= 0 || R < 2 || R % 2 || R > D ||
      !std::isfinite(scale))
    return GLA_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype) || (out_dtype != in_dtype && out_dtype != GLA_FP32))
    return GLA_ERR_UNSUPPORTED;
  if (D > 4096 || H > 32767 || KV > 32767 || (long long)B * T > (1ll << 40) / ((H + KV) * (long long)D) ||
      (long long)B * T > kMaxInt / ((D + 1) / 2) * 64)
    return GLA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return GLA_OK;
  if (!q || !q_out || !turns || (KV && (!k || !k_out))) return GLA_ERR_INVALID_ARG;
  const uintptr_t odd = size_of(in_dtype) - 1;
  if (((reinterpret_cast<uintptr_t>(q) | (KV ? reinterpret_cast<uintptr_t>(k) : 0)) & odd) ||
      !aligned16(q_out) || (KV && !aligned16(k_out)) || !aligned4(pos) ||
      (reinterpret_cast<uintptr_t>(turns) & 7u))
    return GLA_ERR_ALIGNMENT;
  gla::RotaryArgs a;
  a.q.x = q; a.q.y = q_out; a.q.heads = H;
  a.k.x = k; a.k.y = k_out; a.k.heads = KV;
  for (int j = 0; j < 2; ++j) {
    gla::RotaryTensor& r = j ? a.k : a.q;
    const long long* given = j ? k_strides : q_strides;
    r.stride[0] = (long long)T * r.heads * D;
    r.stride[1] = (long long)r.heads * D;
    r.stride[2] = D;
    if (!given || !r.heads) continue;
    // in place only where both lie alike
    if (r.x == r.y) return GLA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
      if (given[i] < 0) return GLA_ERR_INVALID_ARG;
      r.stride[i] = given[i];
    }
  }
  if ((q == q_out || (KV && k == k_out)) && in_dtype != out_dtype) return GLA_ERR_INVALID_ARG;
  a.turns = turns; a.pos = pos; a.scale = scale; a.interleaved = interleaved != 0;
  a.inverse = inverse != 0; a.B = B; a.T = T; a.D = D; a.R = R;
  a.in_type = in_dtype; a.out_type = out_dtype;
  return done(gla::launch_rotary(a, sm_count(), stream));
}

gla_status gla_window_cache_append(const void* k, const void* v, gla_dtype in_dtype,
                                   const int* pos, const int* start, const int* count,
                                   void* pool_k, void* pool_v, signed char* pool_e,
                                   const int* page, int n, int n_tokens, int n_pages,
                                   int pool_layers, int layer, int window, int sink, int KV,
                                   int dk, int dv, cudaStream_t stream) {
  gla_status st = check_window(in_dtype, in_dtype, window, sink, KV, KV, dk, dv);
  if (st != GLA_OK || (st = check_packed(n, n_tokens, KV)) != GLA_OK ||
      (st = check_window_pool(n_pages, pool_layers, layer, window, sink, KV)) != GLA_OK)
    return st;
  if (n == 0 || n_tokens == 0) return GLA_OK;
  if (!k || !v || !pos || !start || !pool_k || !pool_v || !page) return GLA_ERR_INVALID_ARG;
  if (!aligned16(k, v, pool_k, pool_v, pool_e) || !aligned4(pos, start, count, page))
    return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::AppendArgs a;
  a.cache = {{pool_k, pool_v, page, n, n_pages, pool_layers, layer, KV, window, sink, in_dtype}, pool_e};
  a.tok = {pos, start, n_tokens};
  a.count = count; a.k = k; a.v = v;
  return done(gla::launch_window_append(a, ctl, stream));
}

gla_status gla_window_cache8_read(const void* pool_k, const void* pool_v,
                                  const signed char* pool_e, const int* page, int n, int n_pages,
                                  int pool_layers, int layer, int window, int sink, void* k,
                                  void* v, gla_dtype out_dtype, int KV, int dk, int dv,
                                  cudaStream_t stream) {
  gla_status st = check_window(out_dtype, out_dtype, window, sink, KV, KV, dk, dv);
  if (st != GLA_OK ||
      (st = check_window_pool(n_pages, pool_layers, layer, window, sink, KV)) != GLA_OK)
    return st;
  if (n < 0) return GLA_ERR_INVALID_ARG;
  // the grid: 18 pieces of a row, 256 a CTA
  if ((long long)n * (window + sink) > kMaxInt * 8 / KV) return GLA_ERR_UNSUPPORTED;
  if (n == 0) return GLA_OK;
  if (!pool_k || !pool_v || !pool_e || !page || !k || !v) return GLA_ERR_INVALID_ARG;
  if (!aligned16(pool_k, pool_v, pool_e, k, v) || !aligned4(page)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  const gla::ServeCache c{{const_cast<void*>(pool_k), const_cast<void*>(pool_v), page, n, n_pages,
                           pool_layers, layer, KV, window, sink, out_dtype},
                          const_cast<signed char*>(pool_e)};
  return done(gla::launch_window_read8(c, k, v, nullptr, nullptr, ctl, stream));
}

size_t gla_window_attn8_decode_workspace_size(int n_active, int H, int KV, int window, int sink) {
  if (check_window(GLA_BF16, GLA_BF16, window, sink, H, KV, gla::kDK, gla::kDV) != GLA_OK ||
      check_window_active(n_active, H, window, sink) != GLA_OK)
    return 0;
  return gla::window_decode8_workspace_bytes(n_active, KV, H, window + sink, sm_count());
}

gla_status gla_window_attn8_decode_step(void* pool_k, void* pool_v, signed char* pool_e,
                                        const int* page, const int* pos, int n_active,
                                        int n_pages, int pool_layers, int layer, int window,
                                        int sink, const void* q, const void* k, const void* v,
                                        gla_dtype in_dtype, void* o, gla_dtype out_dtype,
                                        void* workspace, size_t workspace_bytes, int H, int KV,
                                        int dk, int dv, cudaStream_t stream) {
  gla_status st = check_window(in_dtype, out_dtype, window, sink, H, KV, dk, dv);
  if (st != GLA_OK || (st = check_window_active(n_active, H, window, sink)) != GLA_OK ||
      (st = check_window_pool(n_pages, pool_layers, layer, window, sink, KV)) != GLA_OK)
    return st;
  // (a page's bytes of a layer stay below 2^40, the largest step of a tensor map)
  if ((window + (long long)sink) * KV > kMaxInt) return GLA_ERR_UNSUPPORTED;
  if (n_active == 0) return GLA_OK;
  if (!pool_k || !pool_v || !pool_e || !page || !pos || !q || !k || !v || !o)
    return GLA_ERR_INVALID_ARG;
  if (!aligned16(pool_k, pool_v, pool_e, q, k, v, o) || !aligned4(page, pos))
    return GLA_ERR_ALIGNMENT;
  const size_t need = gla_window_attn8_decode_workspace_size(n_active, H, KV, window, sink);
  if (need && (!workspace || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  if (need && !aligned256(workspace)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::Decode8Args a;
  a.cache = {{pool_k, pool_v, page, n_active, n_pages, pool_layers, layer, KV, window, sink, in_dtype},
             pool_e};
  a.pos = pos; a.q = q; a.k = k; a.v = v; a.o = o; a.out_type = out_dtype; a.H = H;
  a.workspace = workspace;
  return done(gla::launch_window_decode8(a, sm_count(), ctl, stream));
}

static gla_status check_chunk(int n, int n_tokens, int H, int KV, int window, int sink) {
  gla_status st = check_packed(n, n_tokens, H);
  if (st != GLA_OK) return st;
  // (a page's bytes of a layer stay below 2^40, the largest step of a tensor map)
  if (window > (1 << 30) - sink || H / KV > gla::kChunkMostHeads ||
      (window + (long long)sink) * KV > kMaxInt)
    return GLA_ERR_UNSUPPORTED;
  return GLA_OK;
}

static size_t chunk_bytes(int n, int n_tokens, int H, int KV, int window, int sink, bool codes) {
  return n == 0 || n_tokens == 0
             ? 0
             : gla::window_chunk_workspace_bytes(n, n_tokens, KV, H, window, sink, codes, sm_count());
}

static size_t checked_chunk_bytes(int n, int n_tokens, int H, int KV, int window, int sink, bool codes) {
  if (check_window(GLA_BF16, GLA_BF16, window, sink, H, KV, gla::kDK, gla::kDV) != GLA_OK ||
      check_chunk(n, n_tokens, H, KV, window, sink) != GLA_OK)
    return 0;
  return chunk_bytes(n, n_tokens, H, KV, window, sink, codes);
}
size_t gla_window_attn_chunk16_workspace_size(int n, int n_tokens, int H, int KV, int window,
                                              int sink) {
  return checked_chunk_bytes(n, n_tokens, H, KV, window, sink, false);
}
size_t gla_window_attn_chunk8_workspace_size(int n, int n_tokens, int H, int KV, int window,
                                             int sink) {
  return checked_chunk_bytes(n, n_tokens, H, KV, window, sink, true);
}
size_t gla_window_attn_chunk_workspace_size(int n, int n_tokens, int H, int KV, int window,
                                            int sink) {
  return std::max(checked_chunk_bytes(n, n_tokens, H, KV, window, sink, false),
                  checked_chunk_bytes(n, n_tokens, H, KV, window, sink, true));
}

gla_status gla_window_attn_chunk(const void* pool_k, const void* pool_v,
                                 const signed char* pool_e, const int* page, const int* pos,
                                 const int* start, int n, int n_tokens, int n_pages,
                                 int pool_layers, int layer, int window, int sink, const void* q,
                                 const void* k, const void* v, gla_dtype in_dtype, void* o,
                                 gla_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                 int H, int KV, int dk, int dv, cudaStream_t stream) {
  gla_status st = check_window(in_dtype, out_dtype, window, sink, H, KV, dk, dv);
  if (st != GLA_OK || (st = check_chunk(n, n_tokens, H, KV, window, sink)) != GLA_OK ||
      (st = check_window_pool(n_pages, pool_layers, layer, window, sink, KV)) != GLA_OK)
    return st;
  if (n == 0 || n_tokens == 0) return GLA_OK;
  if (!pool_k || !pool_v || !page || !pos || !start || !q || !k || !v || !o)
    return GLA_ERR_INVALID_ARG;
  if (!aligned16(pool_k, pool_v, pool_e, q, k, v, o) || !aligned4(page, pos, start))
    return GLA_ERR_ALIGNMENT;
  const size_t need = chunk_bytes(n, n_tokens, H, KV, window, sink, pool_e != nullptr);
  if (need && (!workspace || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
  if (need && !aligned256(workspace)) return GLA_ERR_ALIGNMENT;
  gla::DevCtl ctl;
  if (gla::current_device_ctl(&ctl) != cudaSuccess) return GLA_ERR_CUDA;
  gla::ChunkArgs a;
  a.cache = {{const_cast<void*>(pool_k), const_cast<void*>(pool_v), page, n, n_pages, pool_layers,
              layer, KV, window, sink, in_dtype},
             const_cast<signed char*>(pool_e)};
  a.tok = {pos, start, n_tokens};
  a.q = q; a.k = k; a.v = v; a.o = o; a.out_type = out_dtype; a.H = H; a.workspace = workspace;
  return done(gla::launch_window_chunk(a, sm_count(), ctl, stream));
}

}  // extern "C"
