// layer_norm.cu -- layer norm over the D channels of each token, and its gradient.
//
//   m = mean_c x_c,  r = 1 / sqrt(mean_c (x_c - m)^2 + eps),  n_c = (x_c - m) r
//   y_c = n_c w_c + b_c
// and for the scalar loss sum(y . dy), with d_c = dy_c w_c:
//   dx_c = r (d_c - mean(d) - n_c mean(d n)),   dw_c = sum_tokens dy_c n_c,  db_c = sum_tokens dy_c
//
// Bound by HBM: each element is read once and written once (forward x -> y, backward x, dy ->
// dx), with ~8 and ~10 instructions.  Rows come through rings of bulk copies in shared memory, so
// that the next ones are on their way while one is worked on: forward a warp per row (squares
// about the row's mean, from registers), backward a CTA per two rows, whose threads keep the
// weights of their channels and the sums of their gradients in registers over all the rows of a
// persistent grid.  Rows that 16-byte accesses do not divide, longer ones, and few ones (a token's
// or a batch's decode step) are loaded to registers instead, a CTA per row or R rows; there the
// squares are taken per warp about the warp's own mean, and the warps' are joined by
//   m = sum(k_i m_i) / D,   q = sum(q_i + k_i (m_i - m)^2).
// dw and db: every thread adds the rows of its CTA one after the other, every CTA leaves its sums in
// the workspace, and a second kernel adds them up in the order of the CTAs, so results repeat bit for
// bit.  All arithmetic is fp32, with one rounding to the output's type; the chain of a thread is n over
// the CTAs rows long, and 65,536 rows leave dw off by 3e-7 of its size.  Measured: forward 65536 x 2048
// bf16 94 us (a plain copy of as many bytes 82), 136 before the rings; gradient 65536 x 1536, bf16 x,
// fp32 dy 155 us (a copy 149), before 258.  Rows that the rings do not take, of as many bytes as those:
// forward 32768 x 4096 bf16 142 us and 16384 x 8192 128 (floor 79), 65536 x 1001 bf16 160 (39) and fp32
// 161 (77); gradient 32768 x 4096 and 16384 x 8192, bf16 x, fp32 dy 339 us (198), 65536 x 1001 bf16 151
// (58).  Above 8,192 channels the gradient's 1,024 threads spill 160 to 240 bytes each.
#include <cuda_runtime.h>

#include <algorithm>

#include "elem.cuh"
#include "layer_norm.h"

namespace gla {
namespace {

constexpr int MAX_WARPS = 32;
constexpr int RING_MOST = 6;  // rows of a warp's ring in the forward
constexpr int RING_SPACE = 192 * 1024;
constexpr uint64_t DRAIN_NS = 4000000000ull;  // limit of the exit-time drain waits

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

// ---- rows of up to 2048 channels that 16-byte accesses divide: a warp per row, no barrier between
// warps.  Each warp has a ring of `stages` rows of its own, filled by bulk copies, so that the
// next rows are on their way while it works; the weights are in shared memory too.
template <class TX, class TY, int V, int NV>
__global__ void __launch_bounds__(384)
layer_norm_fwd_ring_kernel(const TX* __restrict__ x, const float* __restrict__ weight,
                           const float* __restrict__ bias, TY* __restrict__ y,
                           float* __restrict__ mean, float* __restrict__ rstd, long long n, int D,
                           float eps, int stages, DevCtl ctl) {
  extern __shared__ __align__(128) uint8_t smem[];  // the rings, then the weights
  __shared__ alignas(8) uint64_t full[12][RING_MOST], never;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int row_bytes = D * (int)sizeof(TX);
  float* const sw = reinterpret_cast<float*>(smem + warps * stages * row_bytes);
  float* const sb = sw + D;
  uint8_t* const ring = smem + w * stages * row_bytes;
  const long long first = (long long)blockIdx.x * warps + w, step = (long long)gridDim.x * warps;
  const int mine = first < n ? (int)((n - first + step - 1) / step) : 0;  // rows of this warp
  int armed = 0;  // rows fetched so far
  auto fetch = [&](int k) {  // one lane
    armed = k + 1;
    const uint32_t bar = smem_u32(&full[w][k % stages]);
    mbar_arrive_expect_tx(bar, row_bytes);
    bulk_load(smem_u32(ring) + (k % stages) * row_bytes, x + (first + k * step) * D, row_bytes, bar);
  };
  if (lane == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full[w][s]), 1);
    if (w == 0) mbar_init(smem_u32(&never), 1);
    fence_barrier_init();
    fence_proxy_async();
    for (int k = 0; k < stages && k < mine; ++k) fetch(k);
  }
  // four channels of every access, then the next four of every access: the 16 bytes that the lanes
  // of a warp read together lie side by side
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    const int at = (c % V / 4) * (D / V * 4) + c / V * 4 + c % 4;
    sw[at] = weight ? __ldg(weight + c) : 1.f;
    sb[at] = bias ? __ldg(bias + c) : 0.f;
  }
  __syncthreads();
  const float inv_D = 1.f / D;
  bool ok = true;
  for (int k = 0; k < mine; ++k) {
    const long long row = first + k * step;
    if (k == ctl.stall_step) ok = ok && mbar_wait(smem_u32(&never), 0, ctl);  // the diagnostic
    ok = ok && mbar_wait(smem_u32(&full[w][k % stages]), (k / stages) & 1, ctl);
    const TX* xt = reinterpret_cast<const TX*>(ring + (k % stages) * row_bytes);
    Pack<TX, V> in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + 32 * i) * V;
      if (c < D) in[i].load_shared(xt + c);
      else in[i].fill(0.f);
    }
    __syncwarp();
    if (lane == 0 && ok && k + stages < mine) fetch(k + stages);
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V / 2; j += 2) {
        a = add2(a, in[i].get2(j));
        b = add2(b, in[i].get2(j + 1));
      }
    a = add2(a, b);
    const float m = warp_sum(a.x + a.y) * inv_D;
    const float2 minus = make_float2(-m, -m);
    a = b = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((lane + 32 * i) * V < D)
#pragma unroll
        for (int j = 0; j < V / 2; j += 2) {
          const float2 c = add2(in[i].get2(j), minus), d = add2(in[i].get2(j + 1), minus);
          a = fma2(c, c, a);
          b = fma2(d, d, b);
        }
    a = add2(a, b);
    const float rs = 1.f / sqrtf(warp_sum(a.x + a.y) * inv_D + eps);
    const float2 scale = make_float2(rs, rs);
    TY* const yp = y + row * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + 32 * i) * V;
      if (c < D) {
        Pack<TY, V> out;
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
          const int at = j * (D / V * 4) + (lane + 32 * i) * 4;
          const float4 w4 = *reinterpret_cast<const float4*>(sw + at);
          const float4 b4 = *reinterpret_cast<const float4*>(sb + at);
          out.set2(2 * j, fma2(mul2(add2(in[i].get2(2 * j), minus), scale),
                               make_float2(w4.x, w4.y), make_float2(b4.x, b4.y)));
          out.set2(2 * j + 1, fma2(mul2(add2(in[i].get2(2 * j + 1), minus), scale),
                                   make_float2(w4.z, w4.w), make_float2(b4.z, b4.w)));
        }
        out.store(yp + c);
      }
    }
    if (lane == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = rs;
    }
  }
  // after a wait that gave up nothing is fetched any more; the copies in flight land before the
  // CTA's memory is given back
  if (!ok && lane == 0)
    for (int k = max(0, armed - stages); k < armed; ++k)
      mbar_wait(smem_u32(&full[w][k % stages]), (k / stages) & 1, ctl, DRAIN_NS);
}

// ---- gradient, rows that 16-byte accesses divide and of which the ring holds twelve: a CTA takes R
// rows at a time from a ring of bulk copies in shared memory, thread t the channels (t + threads i) V ..
// The 2 R sums of a warp are taken by halving the values with the lanes (6 shuffles for 4 sums
// in place of 20), and joined over the warps behind the one barrier the same way.
constexpr int RING_R = 2, RING_STAGES = 6;

template <class TX, class TY, int V, int NV>
__global__ void __launch_bounds__(512)
layer_norm_bwd_ring_kernel(const TY* __restrict__ dy, const TX* __restrict__ x,
                           const float* __restrict__ weight, const float* __restrict__ mean,
                           const float* __restrict__ rstd, TY* __restrict__ dx,
                           float* __restrict__ part, long long n, int D, DevCtl ctl) {
  constexpr int R = RING_R, P = NV * V / 2;
  griddep_launch_dependents();  // the reduction launched next waits for this whole grid
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ alignas(8) uint64_t full[RING_STAGES], never;
  __shared__ float4 stat[2][16];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, warps = blockDim.x >> 5;
  const int x_bytes = R * D * (int)sizeof(TX), stage = x_bytes + R * D * (int)sizeof(TY);
  const long long groups = (n + R - 1) / R;
  const int mine = (int)((groups - blockIdx.x + gridDim.x - 1) / gridDim.x);  // groups of this CTA
  int armed = 0;  // groups fetched so far
  auto fetch = [&](int k) {  // one thread
    armed = k + 1;
    const long long row0 = (blockIdx.x + (long long)k * gridDim.x) * R;
    const int rows = (int)min((long long)R, n - row0);
    const uint32_t bar = smem_u32(&full[k % RING_STAGES]);
    const uint32_t dst = smem_u32(smem) + (k % RING_STAGES) * stage;
    mbar_arrive_expect_tx(bar, rows * D * (int)(sizeof(TX) + sizeof(TY)));
    bulk_load(dst, x + row0 * D, rows * D * (int)sizeof(TX), bar);
    bulk_load(dst + x_bytes, dy + row0 * D, rows * D * (int)sizeof(TY), bar);
  };
  if (t == 0) {
    for (int s = 0; s < RING_STAGES; ++s) mbar_init(smem_u32(&full[s]), 1);
    mbar_init(smem_u32(&never), 1);
    fence_barrier_init();
    fence_proxy_async();
    for (int k = 0; k < RING_STAGES && k < mine; ++k) fetch(k);
  }
  float2 wv[P], dw[P], db[P];
  bool live[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + blockDim.x * i) * V;
    live[i] = c < D;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      wv[i * V / 2 + j] = live[i] && weight ? *reinterpret_cast<const float2*>(weight + c + 2 * j)
                                            : make_float2(1.f, 1.f);
      dw[i * V / 2 + j] = db[i * V / 2 + j] = make_float2(0.f, 0.f);
    }
  }
  const float inv_D = 1.f / D;
  auto stats_of = [&](int k, float (&m)[R], float (&rs)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = (blockIdx.x + (long long)k * gridDim.x) * R + r;
      const bool ok = k < mine && row < n;
      m[r] = ok ? __ldg(mean + row) : 0.f;
      rs[r] = ok ? __ldg(rstd + row) : 0.f;
    }
  };
  float m[R], rs[R], m_next[R], rs_next[R];
  stats_of(0, m, rs);
  __syncthreads();

  bool ok = true;
  for (int k = 0; k < mine; ++k) {
    const int s = k % RING_STAGES;
    const long long row0 = (blockIdx.x + (long long)k * gridDim.x) * R;
    stats_of(k + 1, m_next, rs_next);
    if (k == ctl.stall_step) ok = ok && mbar_wait(smem_u32(&never), 0, ctl);  // the diagnostic
    ok = ok && mbar_wait(smem_u32(&full[s]), (k / RING_STAGES) & 1, ctl);
    const TX* xt = reinterpret_cast<const TX*>(smem + s * stage);
    const TY* gt = reinterpret_cast<const TY*>(smem + s * stage + x_bytes);
    float2 nx[R][P], d[R][P];  // the normalised row and dy w
    float v[2 * R];            // sums of d and of d n
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 scale = make_float2(rs[r], rs[r]), minus = make_float2(-m[r], -m[r]);
      float2 s1 = make_float2(0.f, 0.f), s2 = s1;
      const bool row = row0 + r < n;  // rows past the end hold the ring's former ones
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + blockDim.x * i) * V;
        Pack<TX, V> xv;
        Pack<TY, V> gv;
        if (live[i] && row) {
          xv.load_shared(xt + r * D + c);
          gv.load_shared(gt + r * D + c);
        } else {
          xv.fill(0.f);
          gv.fill(0.f);
        }
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const int e = i * V / 2 + j;
          const float2 g = gv.get2(j);
          nx[r][e] = mul2(add2(xv.get2(j), minus), scale);
          d[r][e] = mul2(g, wv[e]);
          s1 = add2(s1, d[r][e]);
          s2 = fma2(d[r][e], nx[r][e], s2);
          dw[e] = fma2(g, nx[r][e], dw[e]);
          db[e] = add2(db[e], g);
        }
      }
      v[2 * r] = s1.x + s1.y;
      v[2 * r + 1] = s2.x + s2.y;
    }
    // lanes 0-15 keep values 0, 1 and lanes 16-31 values 2, 3; then bit 3 halves them again
    static_assert(R == 2, "four sums");
    const bool up = lane & 16, odd = lane & 8;
    float p0 = up ? v[2] : v[0], p1 = up ? v[3] : v[1];
    p0 += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
    p1 += __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
    float q = (odd ? p1 : p0) + __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 8);
    q += __shfl_xor_sync(0xffffffffu, q, 4);
    q += __shfl_xor_sync(0xffffffffu, q, 2);
    q += __shfl_xor_sync(0xffffffffu, q, 1);
    if ((lane & 7) == 0) reinterpret_cast<float*>(&stat[k & 1][w])[lane >> 3] = q;
    __syncthreads();  // also frees the ring's stage
    if (t == 0 && ok && k + RING_STAGES < mine) fetch(k + RING_STAGES);
    // lane l: value l % 4 of warps l / 4 and l / 4 + 8
    const float* st = reinterpret_cast<const float*>(stat[k & 1]);
    q = lane < 4 * warps ? st[lane] : 0.f;
    if (lane + 32 < 4 * warps) q += st[lane + 32];
    q += __shfl_xor_sync(0xffffffffu, q, 4);
    q += __shfl_xor_sync(0xffffffffu, q, 8);
    q += __shfl_xor_sync(0xffffffffu, q, 16);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float c1 = __shfl_sync(0xffffffffu, q, 2 * r) * inv_D;
      const float c2 = __shfl_sync(0xffffffffu, q, 2 * r + 1) * inv_D;
      if (row0 + r < n) {
        const float2 a = make_float2(-c1, -c1), b = make_float2(-c2, -c2);
        const float2 scale = make_float2(rs[r], rs[r]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (live[i]) {
            Pack<TY, V> out;
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
              const int e = i * V / 2 + j;
              out.set2(j, mul2(fma2(nx[r][e], b, add2(d[r][e], a)), scale));
            }
            out.store(dx + (row0 + r) * D + (t + blockDim.x * i) * V);
          }
      }
      m[r] = m_next[r];
      rs[r] = rs_next[r];
    }
  }
  // after a wait that gave up nothing is fetched any more; the copies in flight land before the
  // CTA's memory is given back
  if (!ok && t == 0)
    for (int k = max(0, armed - RING_STAGES); k < armed; ++k)
      mbar_wait(smem_u32(&full[k % RING_STAGES]), (k / RING_STAGES) & 1, ctl, DRAIN_NS);
  float* p = part + (long long)blockIdx.x * 2 * D;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live[i])
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const int c = (t + blockDim.x * i) * V + 2 * j;
        *reinterpret_cast<float2*>(p + c) = dw[i * V / 2 + j];
        *reinterpret_cast<float2*>(p + D + c) = db[i * V / 2 + j];
      }
}

// dw (columns 0..D-1 of a part) and db (D..2D-1): 32 warps take every 32nd part of 32 columns,
// then join in order.
__global__ void __launch_bounds__(1024)
layer_norm_sum_kernel(const float* __restrict__ part, int parts, int D, float* __restrict__ dw,
                      float* __restrict__ db) {
  __shared__ float acc[32][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();
  float s = 0.f;
  if (c < 2 * D)
#pragma unroll 4
    for (int k = w; k < parts; k += 32) s += part[(long long)k * 2 * D + c];
  acc[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < 2 * D) {
    s = acc[0][lane];
#pragma unroll
    for (int k = 1; k < 32; ++k) s += acc[k][lane];
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
Shape shape_of(int D, gla_dtype x_type, bool backward) {
  Shape s;
  const int wide = x_type == GLA_FP32 ? 4 : 8;
  s.V = D % wide == 0 ? wide : 1;
  const int units = D / s.V;
  if (s.V == 8) s.NV = units <= 512 ? 1 : 2;
  else if (s.V == 4) s.NV = units <= 256 && !backward ? 1 : units <= 1024 ? 2 : 4;
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

// CTAs of `threads` on an SM: 1024 threads, at most 16 CTAs.
int ctas_per_sm(int threads) { return std::max(1, std::min(16, 1024 / threads)); }
int persistent_grid(long long n, int threads, int R, int n_sm) {
  return (int)std::min<long long>((n + R - 1) / R, (long long)n_sm * ctas_per_sm(threads));
}

template <class TX, class TY>
struct Fwd {
  const LayerNormArgs& a;
  int threads, n_sm;
  DevCtl ctl;
  cudaStream_t stream;
  template <int V, int NV>
  cudaError_t go() const {
    // wide types only exist at their own vector width
    if constexpr (V > 1 && V * sizeof(TX) != 16) {
      return cudaErrorInvalidValue;
    } else {
      // A warp per row where there are more than 8 rows for every SM; a CTA per row where there are
      // not (16 rows of 2048: 22 us a call either way, the launch's), and above 2,048 channels, for
      // which the ring is not built (4096 channels: 142 us for the bytes that take 94 at 2048).
      if constexpr (V > 1) {
        if (a.D <= 2048 && a.n > 8ll * n_sm) {
          constexpr int U = 2048 / (32 * V);  // accesses of a lane for 2048 channels
          if (a.D <= 2048 / 4) return ring<V, U / 4>();
          if (a.D <= 2048 / 2) return ring<V, U / 2>();
          if (a.D <= 2048 / 4 * 3) return ring<V, U / 4 * 3>();
          return ring<V, U>();
        }
      }
      constexpr int R = V * NV > 8 ? 1 : V * NV == 8 ? 2 : 4;
      if constexpr (V * NV == 16)
        if (threads > 512) return run<V, NV, 1, 1024>();
      // a row per CTA until they fill the device, then R rows in flight
      if (a.n <= 2ll * n_sm) return run<V, NV, 1, 512>();
      return run<V, NV, R, 512>();
    }
  }
  // As many warps (at most 12: 94 us at 65536 x 2048 bf16, with 16 of fewer rows 97, with 8 102)
  // as have two rows each in the ring's space, and as many rows.
  template <int V, int NV>
  cudaError_t ring() const {
    const int row = a.D * (int)sizeof(TX), warps = std::min(12, RING_SPACE / (2 * row));
    const int stages = std::min(RING_MOST, RING_SPACE / (warps * row));
    const int smem = warps * stages * row + 2 * a.D * (int)sizeof(float);
    auto k = layer_norm_fwd_ring_kernel<TX, TY, V, NV>;
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<long long>((a.n + warps - 1) / warps, n_sm);
    k<<<grid, 32 * warps, smem, stream>>>((const TX*)a.x, a.weight, a.bias, (TY*)a.y, a.mean,
                                          a.rstd, a.n, a.D, a.eps, stages, ctl);
    return cudaGetLastError();
  }
  template <int V, int NV, int R, int MAX_T>
  cudaError_t run() const {
    const int grid = persistent_grid(a.n, threads, R, n_sm);
    layer_norm_fwd_kernel<TX, TY, V, NV, R, MAX_T><<<grid, threads, 0, stream>>>(
        (const TX*)a.x, a.weight, a.bias, (TY*)a.y, a.mean, a.rstd, a.n, a.D, a.eps);
    return cudaGetLastError();
  }
};

template <class TX, class TY>
struct Bwd {
  const LayerNormArgs& a;
  int threads, n_sm;
  DevCtl ctl;
  cudaStream_t stream;
  template <int V, int NV>
  cudaError_t go() const {
    if constexpr (V > 1 && V * sizeof(TX) != 16) {
      return cudaErrorInvalidValue;
    } else {
      if constexpr (V > 1 && V * NV == 8)
        if (ring_bytes() <= 200 * 1024) return ring<V, NV>();
      if constexpr (V * NV == 16)
        if (threads > 512) return run<V, NV, 1, 1024>();
      return run<V, NV, (V * NV > 8 ? 1 : 2), 512>();
    }
  }
  int ring_bytes() const { return RING_STAGES * RING_R * a.D * (int)(sizeof(TX) + sizeof(TY)); }
  template <int V, int NV>
  cudaError_t ring() const {
    auto k = layer_norm_bwd_ring_kernel<TX, TY, V, NV>;
    const int smem = ring_bytes();
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // CTAs that fit an SM's shared memory (228 KB, 1 KB of it each CTA's own) and threads
    const int per = std::max(1, std::min(ctas_per_sm(threads), 227 * 1024 / (smem + 2048)));
    const int grid = (int)std::min<long long>((a.n + RING_R - 1) / RING_R, (long long)n_sm * per);
    k<<<grid, threads, smem, stream>>>((const TY*)a.dy, (const TX*)a.x, a.weight, a.mean, a.rstd,
                                       (TY*)a.dx, a.part, a.n, a.D, ctl);
    return sum(grid);
  }
  template <int V, int NV, int R, int MAX_T>
  cudaError_t run() const {
    const int grid = persistent_grid(a.n, threads, R, n_sm);
    layer_norm_bwd_kernel<TX, TY, V, NV, R, MAX_T><<<grid, threads, 0, stream>>>(
        (const TY*)a.dy, (const TX*)a.x, a.weight, a.mean, a.rstd, (TY*)a.dx, a.part, a.n, a.D);
    return sum(grid);
  }
  cudaError_t sum(int parts) const {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.dw && !a.db)) return e;
    PdlLaunch l(dim3((2 * a.D + 31) / 32), dim3(1024), 0, stream, true);
    return cudaLaunchKernelEx(&l.cfg, layer_norm_sum_kernel, (const float*)a.part, parts, a.D,
                              a.dw, a.db);
  }
};

template <template <class, class> class Op>
cudaError_t dispatch(const LayerNormArgs& a, bool backward, int n_sm, DevCtl ctl,
                     cudaStream_t stream) {
  const Shape s = shape_of(a.D, a.x_type, backward);
  const bool wide = a.out_type == GLA_FP32;
  if (a.x_type == GLA_FP32)
    return with_shape(s, Op<float, float>{a, s.threads, n_sm, ctl, stream});
  if (a.x_type == GLA_BF16)
    return wide ? with_shape(s, Op<__nv_bfloat16, float>{a, s.threads, n_sm, ctl, stream})
                : with_shape(s, Op<__nv_bfloat16, __nv_bfloat16>{a, s.threads, n_sm, ctl, stream});
  return wide ? with_shape(s, Op<__half, float>{a, s.threads, n_sm, ctl, stream})
              : with_shape(s, Op<__half, __half>{a, s.threads, n_sm, ctl, stream});
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(long long n, int D, int n_sm) {
  // the widest grid over the input types
  int grid = 0;
  for (gla_dtype t : {GLA_BF16, GLA_FP32})
    grid = std::max(grid, persistent_grid(n, shape_of(D, t, true).threads, 1, n_sm));
  return (size_t)grid * 2 * D * sizeof(float);
}

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, int n_sm, DevCtl ctl,
                                  cudaStream_t stream) {
  return dispatch<Fwd>(a, false, n_sm, ctl, stream);
}
cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, int n_sm, DevCtl ctl,
                                  cudaStream_t stream) {
  if (a.n == 0) {  // no token: the weights' gradients are zero
    if (!a.dw && !a.db) return cudaSuccess;
    layer_norm_sum_kernel<<<(2 * a.D + 31) / 32, 1024, 0, stream>>>(nullptr, 0, a.D, a.dw, a.db);
    return cudaGetLastError();
  }
  return dispatch<Bwd>(a, true, n_sm, ctl, stream);
}

}  // namespace gla
