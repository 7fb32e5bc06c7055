// layer_norm.cu -- layer norm over the D channels of each token, and its gradient.
//
//   m = mean_c x_c,  r = 1 / sqrt(mean_c (x_c - m)^2 + eps),  n_c = (x_c - m) r
//   y_c = n_c w_c + b_c
// and for the scalar loss sum(y . dy), with d_c = dy_c w_c:
//   dx_c = r (d_c - mean(d) - n_c mean(d n)),   dw_c = sum_tokens dy_c n_c,  db_c = sum_tokens dy_c
//
// Bound by HBM: each element is read once and written once (forward x -> y, backward x, dy ->
// dx), with ~10 and ~20 instructions.  A CTA of D / (V NV) threads takes whole rows: thread t
// holds NV accesses of V consecutive channels (16 bytes of the input where D allows) and keeps
// the weights of its channels, and the sums of their gradients, in registers over all the rows
// of a persistent grid; R rows are in flight per iteration, so that their loads overlap and one
// barrier serves all of them.  The mean and the sum of squares about it are taken per warp (the
// squares about the warp's own mean, so nothing cancels) and the warps' are joined by
//   m = sum(k_i m_i) / D,   q = sum(q_i + k_i (m_i - m)^2).
// dw and db: every CTA leaves its sums in the workspace, and a second kernel adds them up in the
// order of the CTAs, so results repeat bit for bit.  All arithmetic is fp32, with one rounding
// to the output's type.
#include <cuda_runtime.h>

#include <algorithm>

#include "elem.cuh"
#include "layer_norm.h"

namespace gla {
namespace {

constexpr int MAX_WARPS = 32;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Channels [0, D) that warp w holds (accesses i of V channels at (t + threads i) V).
template <int V, int NV>
__device__ __forceinline__ int warp_count(int w, int threads, int D) {
  int k = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    k += min(max(D - (threads * i + 32 * w) * V, 0), 32 * V);
  return k;
}

template <class TX, class TY, int V, int NV, int R, int MAX_T>
__global__ void __launch_bounds__(MAX_T)
layer_norm_fwd_kernel(const TX* __restrict__ x, const float* __restrict__ weight,
                      const float* __restrict__ bias, TY* __restrict__ y,
                      float* __restrict__ mean, float* __restrict__ rstd, long long n, int D,
                      float eps) {
  __shared__ float2 stat[2][R][MAX_WARPS];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, warps = blockDim.x >> 5;
  float wv[NV * V], bv[NV * V];
  bool live[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + blockDim.x * i) * V;
    live[i] = c < D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      wv[i * V + j] = live[i] && weight ? __ldg(weight + c + j) : 1.f;
      bv[i * V + j] = live[i] && bias ? __ldg(bias + c + j) : 0.f;
    }
  }
  const float count = (float)warp_count<V, NV>(w, blockDim.x, D);
  const float lane_count = lane < warps ? (float)warp_count<V, NV>(lane, blockDim.x, D) : 0.f;
  const float inv_count = count > 0.f ? 1.f / count : 0.f, inv_D = 1.f / D;
  int buf = 0;
  for (long long row0 = (long long)blockIdx.x * R; row0 < n;
       row0 += (long long)gridDim.x * R, buf ^= 1) {
    Pack<TX, V> in[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (live[i] && row0 + r < n)
          in[r][i].load(x + (row0 + r) * D + (t + blockDim.x * i) * V);
        else
          in[r][i].fill(0.f);
      }
    float m[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) m[r] += in[r][i].get(j);
      m[r] = warp_sum(m[r]) * inv_count;
      q[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live[i])
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float c = in[r][i].get(j) - m[r];
            q[r] = fmaf(c, c, q[r]);
          }
      q[r] = warp_sum(q[r]);
    }
    if (warps > 1) {
      if (lane == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) stat[buf][r][w] = make_float2(m[r], q[r]);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) {  // lane k joins warp k's
        const float2 s = lane < warps ? stat[buf][r][lane] : make_float2(0.f, 0.f);
        m[r] = warp_sum(lane_count * s.x) * inv_D;
        const float d = s.x - m[r];
        q[r] = warp_sum(fmaf(lane_count * d, d, s.y));
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= n) break;
      const float rs = 1.f / sqrtf(q[r] * inv_D + eps);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live[i]) {
          Pack<TY, V> out;
#pragma unroll
          for (int j = 0; j < V; ++j)
            out.set(j, fmaf((in[r][i].get(j) - m[r]) * rs, wv[i * V + j], bv[i * V + j]));
          out.store(y + (row0 + r) * D + (t + blockDim.x * i) * V);
        }
      if (t == 0) {
        if (mean) mean[row0 + r] = m[r];
        if (rstd) rstd[row0 + r] = rs;
      }
    }
  }
}

template <class TX, class TY, int V, int NV, int R, int MAX_T>
__global__ void __launch_bounds__(MAX_T)
layer_norm_bwd_kernel(const TY* __restrict__ dy, const TX* __restrict__ x,
                      const float* __restrict__ weight, const float* __restrict__ mean,
                      const float* __restrict__ rstd, TY* __restrict__ dx,
                      float* __restrict__ part, long long n, int D) {
  griddep_launch_dependents();  // the reduction launched next waits for this whole grid
  __shared__ float2 stat[2][R][MAX_WARPS];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, warps = blockDim.x >> 5;
  float wv[NV * V], dw[NV * V], db[NV * V];
  bool live[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + blockDim.x * i) * V;
    live[i] = c < D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      wv[i * V + j] = live[i] && weight ? __ldg(weight + c + j) : 1.f;
      dw[i * V + j] = db[i * V + j] = 0.f;
    }
  }
  const float inv_D = 1.f / D;
  int buf = 0;
  for (long long row0 = (long long)blockIdx.x * R; row0 < n;
       row0 += (long long)gridDim.x * R, buf ^= 1) {
    Pack<TX, V> in[R][NV];
    Pack<TY, V> gr[R][NV];
    float m[R], rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool ok = row0 + r < n;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long long at = (row0 + r) * D + (t + blockDim.x * i) * V;
        if (live[i] && ok) {
          in[r][i].load(x + at);
          gr[r][i].load(dy + at);
        } else {
          in[r][i].fill(0.f);
          gr[r][i].fill(0.f);
        }
      }
      m[r] = ok ? __ldg(mean + row0 + r) : 0.f;
      rs[r] = ok ? __ldg(rstd + row0 + r) : 0.f;
    }
    float s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s1[r] = s2[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float g = gr[r][i].get(j), nx = (in[r][i].get(j) - m[r]) * rs[r];
          const float d = g * wv[i * V + j];
          s1[r] += d;
          s2[r] = fmaf(d, nx, s2[r]);
          dw[i * V + j] = fmaf(g, nx, dw[i * V + j]);
          db[i * V + j] += g;
        }
      s1[r] = warp_sum(s1[r]);
      s2[r] = warp_sum(s2[r]);
    }
    if (warps > 1) {
      if (lane == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) stat[buf][r][w] = make_float2(s1[r], s2[r]);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 s = lane < warps ? stat[buf][r][lane] : make_float2(0.f, 0.f);
        s1[r] = warp_sum(s.x);
        s2[r] = warp_sum(s.y);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= n) break;
      const float c1 = s1[r] * inv_D, c2 = s2[r] * inv_D;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live[i]) {
          Pack<TY, V> out;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float nx = (in[r][i].get(j) - m[r]) * rs[r];
            out.set(j, rs[r] * (gr[r][i].get(j) * wv[i * V + j] - c1 - nx * c2));
          }
          out.store(dx + (row0 + r) * D + (t + blockDim.x * i) * V);
        }
    }
  }
  float* p = part + (long long)blockIdx.x * 2 * D;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live[i])
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (t + blockDim.x * i) * V + j;
        p[c] = dw[i * V + j];
        p[D + c] = db[i * V + j];
      }
}

// dw (columns 0..D-1 of a part) and db (D..2D-1): 8 warps take every eighth part of 32 columns,
// then join in order.
__global__ void __launch_bounds__(256)
layer_norm_sum_kernel(const float* __restrict__ part, int parts, int D, float* __restrict__ dw,
                      float* __restrict__ db) {
  __shared__ float acc[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();
  float s = 0.f;
  if (c < 2 * D)
    for (int k = w; k < parts; k += 8) s += part[(long long)k * 2 * D + c];
  acc[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < 2 * D) {
    s = acc[0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k) s += acc[k][lane];
    if (c < D) {
      if (dw) dw[c] = s;
    } else if (db) {
      db[c - D] = s;
    }
  }
}

// Threads of a CTA and channels per thread: V channels per access (the widest that keeps every
// row's accesses aligned), NV accesses, so that 512 threads cover D up to 8192; above that 1024
// threads do, with the registers of a thread halved.
struct Shape {
  int V, NV, threads;
};
Shape shape_of(int D, gla_dtype x_type) {
  Shape s;
  const int wide = x_type == GLA_FP32 ? 4 : 8;
  s.V = D % wide == 0 ? wide : 1;
  const int units = D / s.V;
  if (s.V == 8) s.NV = units <= 512 ? 1 : 2;
  else if (s.V == 4) s.NV = units <= 256 ? 1 : units <= 1024 ? 2 : 4;
  else s.NV = units <= 256 ? 1 : units <= 2048 ? 4 : 16;
  const int per = s.V * s.NV;
  s.threads = ((D + per - 1) / per + 31) / 32 * 32;
  return s;
}

template <class F>
cudaError_t with_shape(const Shape& s, F f) {
  if (s.V == 8) return s.NV == 1 ? f.template go<8, 1>() : f.template go<8, 2>();
  if (s.V == 4)
    return s.NV == 1 ? f.template go<4, 1>() : s.NV == 2 ? f.template go<4, 2>()
                                                         : f.template go<4, 4>();
  return s.NV == 1 ? f.template go<1, 1>() : s.NV == 4 ? f.template go<1, 4>()
                                                       : f.template go<1, 16>();
}

// CTAs that fill the device: as many as an SM holds (registers), at most one per R rows.
template <class K>
int persistent_grid(K kernel, int threads, long long n, int R, int n_sm) {
  int per = 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess)
    per = 1;
  return (int)std::min<long long>((n + R - 1) / R, (long long)n_sm * std::max(per, 1));
}

template <class TX, class TY>
struct Fwd {
  const LayerNormArgs& a;
  int threads, n_sm;
  cudaStream_t stream;
  template <int V, int NV>
  cudaError_t go() const {
    // wide types only exist at their own vector width
    if constexpr (V > 1 && V * sizeof(TX) != 16) {
      return cudaErrorInvalidValue;
    } else {
      constexpr int R = V * NV > 8 ? 1 : V * NV == 8 ? 2 : 4;
      if constexpr (V * NV == 16)
        if (threads > 512) return run<V, NV, 1, 1024>();
      // a row per CTA until they fill the device, then R rows in flight
      if (a.n <= 2ll * n_sm) return run<V, NV, 1, 512>();
      return run<V, NV, R, 512>();
    }
  }
  template <int V, int NV, int R, int MAX_T>
  cudaError_t run() const {
    auto k = layer_norm_fwd_kernel<TX, TY, V, NV, R, MAX_T>;
    const int grid = persistent_grid(k, threads, a.n, R, n_sm);
    k<<<grid, threads, 0, stream>>>((const TX*)a.x, a.weight, a.bias, (TY*)a.y, a.mean, a.rstd,
                                    a.n, a.D, a.eps);
    return cudaGetLastError();
  }
};

// Parts of dw and db: the backward's CTAs, at most this many per SM.
int bwd_ctas_per_sm(int threads) { return std::max(1, std::min(16, 1024 / threads)); }
int bwd_grid(long long n, int threads, int R, int n_sm) {
  return (int)std::min<long long>((n + R - 1) / R, (long long)n_sm * bwd_ctas_per_sm(threads));
}

template <class TX, class TY>
struct Bwd {
  const LayerNormArgs& a;
  int threads, n_sm;
  cudaStream_t stream;
  template <int V, int NV>
  cudaError_t go() const {
    if constexpr (V > 1 && V * sizeof(TX) != 16) {
      return cudaErrorInvalidValue;
    } else {
      if constexpr (V * NV == 16)
        if (threads > 512) return run<V, NV, 1, 1024>();
      return run<V, NV, (V * NV > 8 ? 1 : 2), 512>();
    }
  }
  template <int V, int NV, int R, int MAX_T>
  cudaError_t run() const {
    auto k = layer_norm_bwd_kernel<TX, TY, V, NV, R, MAX_T>;
    const int grid = bwd_grid(a.n, threads, R, n_sm);
    k<<<grid, threads, 0, stream>>>((const TY*)a.dy, (const TX*)a.x, a.weight, a.mean, a.rstd,
                                      (TY*)a.dx, a.part, a.n, a.D);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.dw && !a.db)) return e;
    PdlLaunch l(dim3((2 * a.D + 31) / 32), dim3(256), 0, stream, true);
    return cudaLaunchKernelEx(&l.cfg, layer_norm_sum_kernel, (const float*)a.part, grid, a.D,
                                a.dw, a.db);
  }
};

template <template <class, class> class Op>
cudaError_t dispatch(const LayerNormArgs& a, int n_sm, cudaStream_t stream) {
  const Shape s = shape_of(a.D, a.x_type);
  const bool wide = a.out_type == GLA_FP32;
  if (a.x_type == GLA_FP32)
    return with_shape(s, Op<float, float>{a, s.threads, n_sm, stream});
  if (a.x_type == GLA_BF16)
    return wide ? with_shape(s, Op<__nv_bfloat16, float>{a, s.threads, n_sm, stream})
                : with_shape(s, Op<__nv_bfloat16, __nv_bfloat16>{a, s.threads, n_sm, stream});
  return wide ? with_shape(s, Op<__half, float>{a, s.threads, n_sm, stream})
              : with_shape(s, Op<__half, __half>{a, s.threads, n_sm, stream});
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(long long n, int D, int n_sm) {
  // the widest grid over the input types
  int grid = 0;
  for (gla_dtype t : {GLA_BF16, GLA_FP32})
    grid = std::max(grid, bwd_grid(n, shape_of(D, t).threads, 1, n_sm));
  return (size_t)grid * 2 * D * sizeof(float);
}

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, int n_sm, cudaStream_t stream) {
  return dispatch<Fwd>(a, n_sm, stream);
}
cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, int n_sm, cudaStream_t stream) {
  if (a.n == 0) {  // no token: the weights' gradients are zero
    if (!a.dw && !a.db) return cudaSuccess;
    layer_norm_sum_kernel<<<(2 * a.D + 31) / 32, 256, 0, stream>>>(nullptr, 0, a.D, a.dw, a.db);
    return cudaGetLastError();
  }
  return dispatch<Bwd>(a, n_sm, stream);
}

}  // namespace gla
