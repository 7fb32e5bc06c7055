// window_fwd.cu -- causal softmax attention over the last `window` tokens and the first `sink`
// ones, 96 key and 192 value channels per head, H query heads on KV key heads:
//
//   z_ts = q_t . k_s,   lse_t = ln sum_s exp(z_ts),   o_t = sum_s exp(z_ts - lse_t) v_s
//
// over the s <= t with t - s < window or s < sink.  One pass over the keys with the running
// maximum m and sum l of each row: a tile of scores rescales what was summed by exp(m - m').
#include <cuda_runtime.h>

#include <cmath>

#include "window_common.cuh"

namespace gla {
namespace {

constexpr int BM = 64, BN = 64, THREADS = 128;
constexpr int K_BYTES = BN * kDK * 2, V_BYTES = BN * kDV * 2, STAGE = K_BYTES + V_BYTES;
constexpr int SMEM = 2 * STAGE;

template <class T, class TO>
__global__ void __launch_bounds__(THREADS)
window_fwd_kernel(WindowArgs a, DevCtl ctl) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int tiles = (a.T + BM - 1) / BM;
  const int h = blockIdx.x % a.H;
  const long long bt = blockIdx.x / a.H;
  const int b = (int)(bt / tiles), q0 = (int)(bt % tiles) * BM;
  const int len = window_length(a.lens, b, a.T, ctl);
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  TO* o = static_cast<TO*>(a.o) + ((long long)b * a.T * a.H + h) * kDV;
  float* lse = a.lse ? a.lse + ((long long)b * a.H + h) * a.T : nullptr;
  const int r0 = q0 + w * 16 + g;  // this thread's rows: r0, r0 + 8

  float acc[kDV / 8][4];
#pragma unroll
  for (int n = 0; n < kDV / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  if (q0 < len) {
    const T* q = static_cast<const T*>(a.q) + ((long long)b * a.T * a.H + h) * kDK;
    const int kv = h / (a.H / a.KV);
    const T* k = static_cast<const T*>(a.k) + ((long long)b * a.T * a.KV + kv) * kDK;
    const T* v = static_cast<const T*>(a.v) + ((long long)b * a.T * a.KV + kv) * kDV;
    const KeyTiles kt(q0, min(q0 + BM, len), BN, a.window, a.sink);

    copy_rows<kCK>(sm, q, (long long)a.H * kDK, q0, BM, len, tid, THREADS);
    copy_commit();
    copy_wait<0>();
    __syncthreads();
    uint32_t qf[kDK / 16][4];
#pragma unroll
    for (int c = 0; c < kDK / 16; ++c) load_a<kCK>(qf[c], sm, w * 16, 2 * c);
    __syncthreads();

    auto fetch = [&](int i) {
      const uint32_t s = sm + (i & 1) * STAGE;
      const int s0 = kt.tile(i) * BN;
      copy_rows<kCK>(s, k, (long long)a.KV * kDK, s0, BN, len, tid, THREADS);
      copy_rows<kCV>(s + K_BYTES, v, (long long)a.KV * kDV, s0, BN, len, tid, THREADS);
      copy_commit();
    };
    fetch(0);
    for (int i = 0; i < kt.n; ++i) {
      if (i + 1 < kt.n) {
        fetch(i + 1);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      __syncthreads();
      const uint32_t ks = sm + (i & 1) * STAGE, vs = ks + K_BYTES;
      const int s0 = kt.tile(i) * BN;
      float z[BN / 8][4];
#pragma unroll
      for (int n = 0; n < BN / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = 0.f;
#pragma unroll
      for (int c = 0; c < kDK / 16; ++c)
#pragma unroll
        for (int n = 0; n < BN / 8; n += 2) {
          uint32_t bf[4];
          load_b<kCK>(bf, ks, n * 8, 2 * c);
          mma16816<T>(z[n], qf[c], bf[0], bf[1]);
          mma16816<T>(z[n + 1], qf[c], bf[2], bf[3]);
        }
      // every query of the tile sees every key of it?
      const bool whole = s0 + BN - 1 <= q0 && s0 + BN <= len &&
                         (q0 + BM - 1 - s0 < a.window || s0 + BN <= a.sink);
      if (!whole)
#pragma unroll
        for (int n = 0; n < BN / 8; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = r0 + (j >> 1) * 8, s = s0 + n * 8 + t2 + (j & 1);
            if (s >= len || !window_sees(t, s, a.window, a.sink)) z[n][j] = -INFINITY;
          }
      float sub[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float top = m[r];
#pragma unroll
        for (int n = 0; n < BN / 8; ++n) top = fmaxf(top, fmaxf(z[n][2 * r], z[n][2 * r + 1]));
        top = quad_max(top);
        const float base = top == -INFINITY ? 0.f : top;  // nothing seen so far
        const float keep = ex2((m[r] - base) * kLog2e);
        m[r] = top;
        sub[r] = base * kLog2e;
        l[r] *= keep;
#pragma unroll
        for (int n = 0; n < kDV / 8; ++n) {
          acc[n][2 * r] *= keep;
          acc[n][2 * r + 1] *= keep;
        }
      }
#pragma unroll
      for (int n = 0; n < BN / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[n][j] = ex2(fmaf(z[n][j], kLog2e, -sub[j >> 1]));
          l[j >> 1] += z[n][j];
        }
#pragma unroll
      for (int c = 0; c < BN / 16; ++c) {
        const uint32_t pf[4] = {pack2<T>(z[2 * c][0], z[2 * c][1]),
                                pack2<T>(z[2 * c][2], z[2 * c][3]),
                                pack2<T>(z[2 * c + 1][0], z[2 * c + 1][1]),
                                pack2<T>(z[2 * c + 1][2], z[2 * c + 1][3])};
#pragma unroll
        for (int n = 0; n < kDV / 8; n += 2) {
          uint32_t bf[4];
          load_bt<kCV>(bf, vs, c * 16, n);
          mma16816<T>(acc[n], pf, bf[0], bf[1]);
          mma16816<T>(acc[n + 1], pf, bf[2], bf[3]);
        }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int t = r0 + 8 * r;
    const float sum = quad_sum(l[r]);
    if (t >= a.T) continue;
    const bool live = t < len;  // a live query sees itself: sum > 0
    const float inv = live ? 1.f / sum : 0.f;
#pragma unroll
    for (int n = 0; n < kDV / 8; ++n)
      store2(o + (long long)t * a.H * kDV + n * 8 + t2, live ? acc[n][2 * r] * inv : 0.f,
             live ? acc[n][2 * r + 1] * inv : 0.f);
    if (lse && (lane & 3) == 0) lse[t] = live ? m[r] + logf(sum) : -INFINITY;
  }
}

template <class T, class TO>
cudaError_t run(const WindowArgs& a, DevCtl ctl, cudaStream_t stream) {
  auto k = window_fwd_kernel<T, TO>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long grid = (long long)a.B * a.H * ((a.T + BM - 1) / BM);
  k<<<(unsigned)grid, THREADS, SMEM, stream>>>(a, ctl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  (void)n_sm;
  const bool wide = a.out_type == GLA_FP32;
  if (a.in_type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, ctl, stream);
  return wide ? run<__half, float>(a, ctl, stream) : run<__half, __half>(a, ctl, stream);
}

}  // namespace gla
