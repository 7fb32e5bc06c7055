// gated_scan.cu -- a linear recurrence whose forget gate depends on the data, per channel:
//
//   f_t = sigmoid(g_t),   h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t
//
// and its gradient: with the adjoint G_t = dL/dh_t = dy_t + f_{t+1} G_{t+1},
//   dx_t = (1 - f_t) G_t,   dg_t = f_t (1 - f_t) (h_{t-1} - x_t) G_t,   dh_0 = f_1 G_1.
//
// Both directions are a scan of pairs (a, b): the map c -> a c + b of a token, composed as
// (a2, b2) o (a1, b1) = (a2 a1, a2 b1 + b2).  The forward's pair is (f, (1 - f) x); the
// gradient runs from the last token with c_t = f_t G_t, i.e. the pair (f, f dy).  1 - f is
// sigmoid(-g), taken from the same exponential, so neither loses digits where it is small; all
// arithmetic and the carried state are fp32.
//
// Bound by HBM: a token and channel cost 8 bytes forward (bf16 x, g in, fp32 y out) and 20
// backward (x, g, y, dy in, dx, dg out), against ~20 and ~30 instructions.  The split keeps
// one pass over memory: a CTA owns one sequence and a slab of channels (32 lanes x VEC
// channels: whole 128-byte lines of 16-bit inputs) and walks the tokens in tiles, each of its
// WARPS warps holding S consecutive tokens of the tile in registers.  A warp composes its
// tokens' pairs, the warps' pairs meet in shared memory, and each thread then runs its tokens
// from the state entering them.  Where sequences x slabs leave SMs idle, a cluster of up to 8
// CTAs takes consecutive tiles of the same slab and exchanges its CTAs' pairs through
// distributed shared memory, one cluster barrier per round; no flag in global memory, no
// workspace, and the order of composition is fixed by the sizes, so results repeat bit for bit.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>

#include "elem.cuh"
#include "gated_scan.h"

namespace gla {
namespace {
namespace cg = cooperative_groups;

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int FWD_S = 8, BWD_S = 4;  // tokens per warp and round

// sigmoid(g) and sigmoid(-g) from e = exp(-|g|); g = +inf gives exactly (1, 0), -inf (0, 1).
__device__ __forceinline__ void gates(float g, float& f, float& u) {
  const float e = __expf(-fabsf(g));
  const float r = __fdividef(1.f, 1.f + e), s = e * r;
  f = g >= 0.f ? r : s;
  u = g >= 0.f ? s : r;
}

template <int VEC>
struct alignas(8 * VEC) Pair {
  float a[VEC], b[VEC];
};

template <int VEC, int CL>
struct Exchange {
  Pair<VEC> warp[2][WARPS][32];
  Pair<VEC> cta[CL > 1 ? 2 : 1][CL > 1 ? CL : 1][32];
};

// The state entering this warp's tokens, from the round's pair of every warp (and CTA of the
// cluster) and the state `carry` entering the round, which becomes the one leaving it.
template <int VEC, int CL>
__device__ __forceinline__ void enter(Exchange<VEC, CL>& ex, int buf, const Pair<VEC>& own,
                                      float (&carry)[VEC], float (&in)[VEC]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  ex.warp[buf][w][lane] = own;
  __syncthreads();
  if constexpr (CL > 1) {
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    if (w < CL) {  // warp w hands the CTA's pair to CTA w of the cluster
      Pair<VEC> p = ex.warp[buf][0][lane];
#pragma unroll
      for (int k = 1; k < WARPS; ++k) {
        const Pair<VEC> n = ex.warp[buf][k][lane];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          p.b[j] = fmaf(n.a[j], p.b[j], n.b[j]);
          p.a[j] *= n.a[j];
        }
      }
      *cl.map_shared_rank(&ex.cta[buf][rank][lane], w) = p;
    }
    cl.sync();
#pragma unroll
    for (int k = 0; k < CL; ++k) {
      const Pair<VEC> p = ex.cta[buf][k][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (k == rank) in[j] = carry[j];
        carry[j] = fmaf(p.a[j], carry[j], p.b[j]);
      }
    }
#pragma unroll
    for (int k = 0; k < WARPS - 1; ++k)
      if (k < w) {
        const Pair<VEC> p = ex.warp[buf][k][lane];
#pragma unroll
        for (int j = 0; j < VEC; ++j) in[j] = fmaf(p.a[j], in[j], p.b[j]);
      }
  } else {
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const Pair<VEC> p = ex.warp[buf][k][lane];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (k == w) in[j] = carry[j];
        carry[j] = fmaf(p.a[j], carry[j], p.b[j]);
      }
    }
  }
}

// Tokens of sequence b: lens[b], or all T.  A length outside [0, T] is an error; it is recorded
// and read as the nearer end.
__device__ __forceinline__ int length_of(const int* lens, int b, int T, const DevCtl& ctl) {
  if (!lens) return T;
  const int n = __ldg(lens + b);
  if (n < 0 || n > T) {
    if (threadIdx.x == 0) record_error(ctl, DEV_RANGE);
    return n < 0 ? 0 : T;
  }
  return n;
}

template <class T, int VEC, int CL>
__global__ void __launch_bounds__(THREADS, 3)
scan_fwd_kernel(const T* __restrict__ x, const T* __restrict__ g, const float* __restrict__ init,
                const int* __restrict__ lens, float* __restrict__ y, float* __restrict__ fin,
                int T_, int D, int slabs, DevCtl ctl) {
  constexpr int S = FWD_S, TILE = WARPS * S;
  __shared__ Exchange<VEC, CL> ex;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int rank = CL > 1 ? blockIdx.x % CL : 0, unit = blockIdx.x / CL;
  const int b = unit / slabs, ch = (unit % slabs) * 32 * VEC + lane * VEC;
  const bool live = ch < D;
  const int len = length_of(lens, b, T_, ctl);
  const long long base = (long long)b * T_ * D + ch;

  float carry[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) carry[j] = live && init ? init[(long long)b * D + ch + j] : 0.f;

  Pack<T, VEC> xr[S], gr[S];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int t = t0 + i;
      if (live && t < len) {
        xr[i].load(x + base + (long long)t * D);
        gr[i].load(g + base + (long long)t * D);
      } else {  // past the sequence: the identity (f = 1, 1 - f = 0)
        xr[i].fill(0.f);
        gr[i].fill(INFINITY);
      }
    }
  };
  const int step = TILE * CL;
  int t0 = rank * TILE + w * S;
  fetch(t0);
  for (int at = 0, buf = 0; at < T_; at += step, t0 += step, buf ^= 1) {
    float f[S][VEC], a[S][VEC];
    Pair<VEC> own;
#pragma unroll
    for (int j = 0; j < VEC; ++j) { own.a[j] = 1.f; own.b[j] = 0.f; }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float u;
        gates(gr[i].get(j), f[i][j], u);
        a[i][j] = u * xr[i].get(j);
        own.b[j] = fmaf(f[i][j], own.b[j], a[i][j]);
        own.a[j] *= f[i][j];
      }
    if (at + step < T_) fetch(t0 + step);
    float h[VEC];
    enter<VEC, CL>(ex, buf, own, carry, h);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int t = t0 + i;
      Pack<float, VEC> out;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[j] = fmaf(f[i][j], h[j], a[i][j]);
        out.set(j, t < len ? h[j] : 0.f);
      }
      if (live && t < T_) out.store(y + base + (long long)t * D);
    }
  }
  if (fin && live && rank == 0 && w == 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) fin[(long long)b * D + ch + j] = carry[j];
}

template <class T, int VEC, int CL>
__global__ void __launch_bounds__(THREADS, 3)
scan_bwd_kernel(const T* __restrict__ x, const T* __restrict__ g, const float* __restrict__ y,
                const float* __restrict__ dy, const float* __restrict__ init,
                const float* __restrict__ dfin, const int* __restrict__ lens,
                float* __restrict__ dx, float* __restrict__ dg, float* __restrict__ dinit, int T_,
                int D, int slabs, DevCtl ctl) {
  constexpr int S = BWD_S, TILE = WARPS * S;
  __shared__ Exchange<VEC, CL> ex;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int rank = CL > 1 ? blockIdx.x % CL : 0, unit = blockIdx.x / CL;
  const int b = unit / slabs, ch = (unit % slabs) * 32 * VEC + lane * VEC;
  const bool live = ch < D;
  const int len = length_of(lens, b, T_, ctl);
  const long long base = (long long)b * T_ * D + ch, edge = (long long)b * D + ch;

  float carry[VEC];  // c = f G of the token behind
#pragma unroll
  for (int j = 0; j < VEC; ++j) carry[j] = live && dfin ? dfin[edge + j] : 0.f;

  const int step = TILE * CL;
  for (int at = 0, buf = 0; at < T_; at += step, buf ^= 1) {
    const int last = T_ - 1 - (at + rank * TILE + w * S);  // this warp's tokens, from the last
    Pack<T, VEC> xr[S], gr[S];
    Pack<float, VEC> dr[S], hr[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int t = last - i;
      if (live && t >= 0 && t < len) {
        const long long p = base + (long long)t * D;
        gr[i].load(g + p);
        dr[i].load(dy + p);
        xr[i].load(x + p);
        if (t > 0) hr[i].load(y + p - D);
        else if (init) hr[i].load(init + edge);
        else hr[i].fill(0.f);
      } else {
        gr[i].fill(INFINITY);
        dr[i].fill(0.f);
        xr[i].fill(0.f);
        hr[i].fill(0.f);
      }
    }
    Pair<VEC> own;
#pragma unroll
    for (int j = 0; j < VEC; ++j) { own.a[j] = 1.f; own.b[j] = 0.f; }
    float f[S][VEC], u[S][VEC];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        gates(gr[i].get(j), f[i][j], u[i][j]);
        own.b[j] = f[i][j] * (own.b[j] + dr[i].get(j));
        own.a[j] *= f[i][j];
      }
    float c[VEC];
    enter<VEC, CL>(ex, buf, own, carry, c);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int t = last - i;
      Pack<float, VEC> ox, og;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float G = dr[i].get(j) + c[j], v = u[i][j] * G;
        c[j] = f[i][j] * G;
        ox.set(j, v);  // past the sequence u = 0 and every operand is finite: zeros
        og.set(j, f[i][j] * v * (hr[i].get(j) - xr[i].get(j)));
      }
      if (live && t >= 0) {
        ox.store(dx + base + (long long)t * D);
        og.store(dg + base + (long long)t * D);
      }
    }
  }
  if (dinit && live && rank == 0 && w == 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dinit[edge + j] = carry[j];
}

// One token: state [.., D] in place.  Pure streaming, one thread per VEC channels; with a page
// table the state of row n, layer l is pool[page[n]][layer0 + l].
template <class T, int VEC>
__global__ void __launch_bounds__(256)
scan_decode_kernel(float* __restrict__ state, const int* __restrict__ page, int n_pages,
                   int pool_layers, int layer0, int L, const T* __restrict__ x,
                   const T* __restrict__ g, float* __restrict__ y, long long rows, int D,
                   int per_row, DevCtl ctl) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long row = i / per_row;
  if (row >= rows) return;
  const int ch = (int)(i - row * per_row) * VEC;
  const long long at = row * D + ch;
  Pack<T, VEC> xr, gr;
  xr.load(x + at);
  gr.load(g + at);
  long long s = row;
  if (page) {
    const int p = __ldg(page + row / L);
    if (p < 0 || p >= n_pages) {
      if (ch == 0) record_error(ctl, DEV_RANGE);
      return;
    }
    s = (long long)p * pool_layers + layer0 + row % L;
  }
  Pack<float, VEC> h;
  float* sp = state + s * D + ch;
  h.load(sp);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    float f, u;
    gates(gr.get(j), f, u);
    h.set(j, fmaf(f, h.get(j), u * xr.get(j)));
  }
  h.store(sp);
  h.store(y + at);
}

// CTAs of a cluster along the tokens: the fewest (1, 2, 4, 8) that give every SM two CTAs, and
// no more than there are tiles.
int pick_cluster(long long units, int T, int tile, int n_sm) {
  const int tiles = (T + tile - 1) / tile;
  int cl = 1;
  while (cl < 8 && units * cl < 2ll * n_sm && cl * 2 <= tiles) cl *= 2;
  return cl;
}

template <class K, class... A>
cudaError_t launch(K kernel, int cl, long long units, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * cl));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int VEC>
cudaError_t fwd_cl(const ScanArgs& a, int cl, long long units, int slabs, DevCtl ctl,
                   cudaStream_t stream) {
  auto go = [&](auto k) {
    return launch(k, cl, units, stream, (const T*)a.x, (const T*)a.g, a.init, a.lens, a.y, a.fin,
                  a.T, a.D, slabs, ctl);
  };
  switch (cl) {
    case 1: return go(scan_fwd_kernel<T, VEC, 1>);
    case 2: return go(scan_fwd_kernel<T, VEC, 2>);
    case 4: return go(scan_fwd_kernel<T, VEC, 4>);
    default: return go(scan_fwd_kernel<T, VEC, 8>);
  }
}
template <class T, int VEC>
cudaError_t bwd_cl(const ScanArgs& a, int cl, long long units, int slabs, DevCtl ctl,
                   cudaStream_t stream) {
  auto go = [&](auto k) {
    return launch(k, cl, units, stream, (const T*)a.x, (const T*)a.g, (const float*)a.y, a.dy,
                  a.init, a.dfin, a.lens, a.dx, a.dg, a.dinit, a.T, a.D, slabs, ctl);
  };
  switch (cl) {
    case 1: return go(scan_bwd_kernel<T, VEC, 1>);
    case 2: return go(scan_bwd_kernel<T, VEC, 2>);
    case 4: return go(scan_bwd_kernel<T, VEC, 4>);
    default: return go(scan_bwd_kernel<T, VEC, 8>);
  }
}

template <class T>
cudaError_t scan_typed(const ScanArgs& a, bool backward, int n_sm, DevCtl ctl,
                       cudaStream_t stream) {
  // two channels per lane where every row starts on a pair (D even), else one
  const int vec = a.D % 2 == 0 ? 2 : 1;
  const int slabs = (a.D + 32 * vec - 1) / (32 * vec);
  const long long units = (long long)a.B * slabs;
  const int cl = pick_cluster(units, a.T, WARPS * (backward ? BWD_S : FWD_S), n_sm);
  if (vec == 2)
    return backward ? bwd_cl<T, 2>(a, cl, units, slabs, ctl, stream)
                    : fwd_cl<T, 2>(a, cl, units, slabs, ctl, stream);
  return backward ? bwd_cl<T, 1>(a, cl, units, slabs, ctl, stream)
                  : fwd_cl<T, 1>(a, cl, units, slabs, ctl, stream);
}

template <class T>
cudaError_t decode_typed(const ScanDecodeArgs& a, DevCtl ctl, cudaStream_t stream) {
  const bool four = a.D % 4 == 0;
  const int per = four ? a.D / 4 : a.D;
  const long long n = a.rows * per;
  const unsigned grid = (unsigned)((n + 255) / 256);
  auto k = four ? scan_decode_kernel<T, 4> : scan_decode_kernel<T, 1>;
  k<<<grid, 256, 0, stream>>>(a.state, a.page, a.n_pages, a.pool_layers, a.layer0, a.L,
                              (const T*)a.x, (const T*)a.g, a.y, a.rows, a.D, per, ctl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, gla_dtype t, bool backward, int n_sm, DevCtl ctl,
                        cudaStream_t stream) {
  if (t == GLA_BF16) return scan_typed<__nv_bfloat16>(a, backward, n_sm, ctl, stream);
  if (t == GLA_FP16) return scan_typed<__half>(a, backward, n_sm, ctl, stream);
  return scan_typed<float>(a, backward, n_sm, ctl, stream);
}

cudaError_t launch_scan_decode(const ScanDecodeArgs& a, gla_dtype t, DevCtl ctl,
                               cudaStream_t stream) {
  if (t == GLA_BF16) return decode_typed<__nv_bfloat16>(a, ctl, stream);
  if (t == GLA_FP16) return decode_typed<__half>(a, ctl, stream);
  return decode_typed<float>(a, ctl, stream);
}

}  // namespace gla
