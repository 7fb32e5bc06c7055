// window_chunk.cu -- the windowed attention (window_fwd.cu) of new tokens over the pages of their
// sequences: token t of a sequence, t = pos + i, sees its page's tokens below pos and the call's own
// from pos to t, of these the last `window` and the first `sink`.
//
// Rows are (token, query head of a key head): a tile of 64 has 64 / G tokens with all their G heads, so
// that a key is read once for them.  Four warps of 16 rows each; keys and values come in tiles of 32, in
// the order of their positions.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "window_packed.cuh"

namespace gla {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS, ROWS = 64, BK = 32;

template <class T, class TO, bool CODES>
__global__ void __launch_bounds__(THREADS)
window_chunk_kernel(ChunkArgs a, int per, DevCtl ctl) {
  __shared__ __align__(128) uint8_t sq[ROWS * kDK * 2], sk[BK * kDK * 2], sv[BK * kDV * 2];
  __shared__ int found[2];
  const WindowCache& c = a.cache.c;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int KV = c.KV, G = a.H / KV, kv = blockIdx.x % KV;
  if (tid == 0) {
    int left = blockIdx.x / KV, b = 0;  // the tile among all sequences'
    for (; b < c.n; ++b) {
      const Sequence s = sequence(c, a.tok, b, ctl);
      const int tiles = (s.tokens + per - 1) / per;
      if (left < tiles) break;
      left -= tiles;
    }
    found[0] = b;
    found[1] = left;
  }
  __syncthreads();
  const int b = found[0];
  if (b >= c.n) return;
  const Sequence s = sequence(c, a.tok, b, ctl);
  const int i0 = found[1] * per, i1 = min(i0 + per, s.tokens);  // its new tokens
  const int rows = (i1 - i0) * G, slots = c.window + c.sink;
  const long long page = (long long)s.page * c.pool_layers + c.layer;

  const T* q = static_cast<const T*>(a.q) + ((long long)(s.first + i0) * a.H + kv * G) * kDK;
  for (int x = tid; x < ROWS * kCK; x += THREADS) {
    const int r = x / kCK, ch = x % kCK;
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) y = __ldg(reinterpret_cast<const uint4*>(q + ((long long)(r / G) * a.H + r % G) * kDK) + ch);
    *reinterpret_cast<uint4*>(sq + tile_off<kCK>(r, ch)) = y;
  }
  __syncthreads();
  uint32_t qf[kDK / 16][4];
#pragma unroll
  for (int j = 0; j < kDK / 16; ++j) load_a<kCK>(qf[j], smem_u32(sq), 16 * w, 2 * j);

  const int g = lane >> 2, t2 = (lane & 3) * 2;
  long long p[2];  // positions of this thread's rows
#pragma unroll
  for (int r = 0; r < 2; ++r) p[r] = (long long)s.pos + i0 + (16 * w + g + 8 * r) / G;
  float acc[kDV / 8][4];
#pragma unroll
  for (int j = 0; j < kDV / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  // the tokens that some row sees: sinks, then from the first row's window on
  const long long first = max((long long)s.pos + i0 - c.window + 1, 0ll), end = (long long)s.pos + i1;
  const int far = (int)min((long long)c.sink, first);
  const long long keys = far + end - first;
  for (long long j0 = 0; j0 < keys; j0 += BK) {
    __syncthreads();
    for (int x = tid; x < BK * (kCK + kCV); x += THREADS) {
      const int r = x / (kCK + kCV), ch = x % (kCK + kCV);
      const long long j = j0 + r, t = j < far ? j : first + j - far;
      const bool key = ch < kCK;
      uint4 y = make_uint4(0u, 0u, 0u, 0u);
      if (j < keys) {
        if (t >= s.pos) {
          const long long row = (s.first + t - s.pos) * KV + kv;
          y = key ? __ldg(static_cast<const uint4*>(a.k) + row * kCK + ch)
                  : __ldg(static_cast<const uint4*>(a.v) + row * kCV + ch - kCK);
        } else {
          const int slot = slot_at(t, c.window, c.sink);
          const long long row = (page * slots + slot) * KV + kv;
          if constexpr (CODES) {
            const uint2 o = key ? __ldg(static_cast<const uint2*>(c.k) + row * kCK + ch)
                                : __ldg(static_cast<const uint2*>(c.v) + row * kCV + ch - kCK);
            const float sc = scale_of(a.cache.exps[((page * KV + kv) * slots + slot) * 2 + !key]);
            whole_of<T, false>(o.x, y.x, y.y);
            whole_of<T, false>(o.y, y.z, y.w);
            y = make_uint4(scaled<T>(y.x, sc), scaled<T>(y.y, sc), scaled<T>(y.z, sc), scaled<T>(y.w, sc));
          } else {
            y = key ? __ldg(static_cast<const uint4*>(c.k) + row * kCK + ch)
                    : __ldg(static_cast<const uint4*>(c.v) + row * kCV + ch - kCK);
          }
        }
      }
      *reinterpret_cast<uint4*>(key ? sk + tile_off<kCK>(r, ch) : sv + tile_off<kCV>(r, ch - kCK)) = y;
    }
    __syncthreads();
    float z[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j) z[e][j] = 0.f;
#pragma unroll
    for (int j = 0; j < kDK / 16; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t bf[4];
        load_b<kCK>(bf, smem_u32(sk), 16 * h, 2 * j);
        mma16816<T>(z[2 * h], qf[j], bf[0], bf[1]);
        mma16816<T>(z[2 * h + 1], qf[j], bf[2], bf[3]);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long k = j0 + 8 * e + t2 + (j & 1), t = k < far ? k : first + k - far, at = p[j >> 1];
        if (k >= keys || t > at || (at - t >= c.window && t >= c.sink)) z[e][j] = -INFINITY;
      }
    uint32_t pf[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(z[e][2 * r], z[e][2 * r + 1]));
      top = fmaxf(m[r], quad_max(top));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = ex2((m[r] - base) * kLog2e);
      m[r] = top;
      l[r] *= keep;
#pragma unroll
      for (int j = 0; j < kDV / 8; ++j) {
        acc[j][2 * r] *= keep;
        acc[j][2 * r + 1] *= keep;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p0 = ex2((z[e][2 * r] - base) * kLog2e), p1 = ex2((z[e][2 * r + 1] - base) * kLog2e);
        l[r] += p0 + p1;
        pf[e >> 1][2 * (e & 1) + r] = pack2<T>(p0, p1);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kDV / 8; j += 2) {
        uint32_t bf[4];
        load_bt<kCV>(bf, smem_u32(sv), 16 * h, j);
        mma16816<T>(acc[j], pf[h], bf[0], bf[1]);
        mma16816<T>(acc[j + 1], pf[h], bf[2], bf[3]);
      }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = 16 * w + g + 8 * r;
    const float inv = 1.f / quad_sum(l[r]);
    if (row >= rows) continue;
    TO* o = static_cast<TO*>(a.o) + ((long long)(s.first + i0 + row / G) * a.H + kv * G + row % G) * kDV;
#pragma unroll
    for (int j = 0; j < kDV / 8; ++j)
      store2(o + 8 * j + t2, acc[j][2 * r] * inv, acc[j][2 * r + 1] * inv);
  }
}

template <class T, class TO>
cudaError_t run(const ChunkArgs& a, DevCtl ctl, cudaStream_t stream) {
  const WindowCache& c = a.cache.c;
  const int G = a.H / c.KV, per = std::max(ROWS / G, 1);
  const long long tiles = (long long)a.tok.n_tokens / per + c.n;
  if (a.cache.exps)
    window_chunk_kernel<T, TO, true><<<(unsigned)(tiles * c.KV), THREADS, 0, stream>>>(a, per, ctl);
  else
    window_chunk_kernel<T, TO, false><<<(unsigned)(tiles * c.KV), THREADS, 0, stream>>>(a, per, ctl);
  return cudaGetLastError();
}

}  // namespace

size_t window_chunk_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_window_chunk(const ChunkArgs& a, int, DevCtl ctl, cudaStream_t stream) {
  const bool wide = a.out_type == GLA_FP32;
  if (a.cache.c.type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, ctl, stream);
  return wide ? run<__half, float>(a, ctl, stream) : run<__half, __half>(a, ctl, stream);
}

}  // namespace gla
