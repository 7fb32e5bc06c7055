// window_bwd.cu -- gradient of the windowed attention (window_fwd.cu) for the scalar loss
// sum(o . dO): with p_ts = exp(q_t . k_s - lse_t) over the visible pairs and
// delta_t = dO_t . o_t,
//   dz_ts = p_ts (dO_t . v_s - delta_t)
//   dq_t = sum_s dz_ts k_s,   dk_s = sum_t dz_ts q_t,   dv_s = sum_t p_ts dO_t
// where dk and dv also sum over the query heads that share the key head.
//
// Three kernels and no atomics, so that results repeat bit for bit: delta (a row sum); dk and dv
// with a key tile held and the queries that see it walked in order, head after head; dq with a
// query tile held and its keys walked.  Both recompute the scores.
#include <cuda_runtime.h>

#include <cmath>

#include "window_common.cuh"

namespace gla {
namespace {

// ---- delta[b,h,t] = dO . o, one warp per (token, head); 0 past a sequence's end
template <class T, class TO>
__global__ void __launch_bounds__(256)
window_delta_kernel(WindowArgs a, float* __restrict__ delta, DevCtl ctl) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);  // (b T + t) H + h
  const int lane = threadIdx.x & 31;
  if (row >= (long long)a.B * a.T * a.H) return;
  const int h = (int)(row % a.H);
  const long long bt = row / a.H;
  const int b = (int)(bt / a.T), t = (int)(bt % a.T);
  const int len = window_length(a.lens, b, a.T, ctl);
  float s = 0.f;
  if (t < len) {
    const T* g = static_cast<const T*>(a.dO) + row * kDV;
    const TO* o = static_cast<const TO*>(a.o) + b * a.o_stride[0] + t * a.o_stride[1] +
                  h * a.o_stride[2];
#pragma unroll
    for (int i = 0; i < kDV / 64; ++i) {
      const int c = i * 64 + lane * 2;
      float g0, g1, o0, o1;
      if constexpr (__is_same(T, __half)) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(g + c));
        g0 = x.x; g1 = x.y;
      } else {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(g + c));
        g0 = x.x; g1 = x.y;
      }
      if constexpr (sizeof(TO) == 4) {
        const float2 x = *reinterpret_cast<const float2*>(o + c);
        o0 = x.x; o1 = x.y;
      } else if constexpr (__is_same(TO, __half)) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(o + c));
        o0 = x.x; o1 = x.y;
      } else {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(o + c));
        o0 = x.x; o1 = x.y;
      }
      s = fmaf(g0, o0, fmaf(g1, o1, s));
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) delta[((long long)b * a.H + h) * a.T + t] = s;
}

// ---- dk, dv: a tile of 64 keys per CTA, 16 per warp; queries in tiles of 32
constexpr int KB = 64, QB = 32, THREADS = 128;
constexpr int KV_Q = QB * kDK * 2, KV_G = QB * kDV * 2, KV_STAGE = KV_Q + KV_G + QB * 8;
constexpr int KV_HELD = KB * (kDK + kDV) * 2, KV_SMEM = KV_HELD + 2 * KV_STAGE;

template <class T, class TO>
__global__ void __launch_bounds__(THREADS)
window_dkv_kernel(WindowArgs a, const float* __restrict__ delta, DevCtl ctl) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int tiles = (a.T + KB - 1) / KB, G = a.H / a.KV;
  const int kv = blockIdx.x % a.KV;
  const long long bt = blockIdx.x / a.KV;
  const int b = (int)(bt / tiles), s0 = (int)(bt % tiles) * KB;
  const int len = window_length(a.lens, b, a.T, ctl);
  const int g = lane >> 2, t2 = (lane & 3) * 2;

  float dk[kDK / 8][4], dv[kDV / 8][4];
#pragma unroll
  for (int n = 0; n < kDK / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) dk[n][j] = 0.f;
#pragma unroll
  for (int n = 0; n < kDV / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) dv[n][j] = 0.f;

  if (s0 < len) {
    const long long ktok = ((long long)b * a.T * a.KV + kv);
    const T* k = static_cast<const T*>(a.k) + ktok * kDK;
    const T* v = static_cast<const T*>(a.v) + ktok * kDV;
    const uint32_t vs = sm + KB * kDK * 2;
    copy_rows<kCK>(sm, k, (long long)a.KV * kDK, s0, KB, len, tid, THREADS);
    copy_rows<kCV>(vs, v, (long long)a.KV * kDV, s0, KB, len, tid, THREADS);
    copy_commit();

    // the queries that see a key of the tile: from its first key to the end of its last key's
    // window, or of the sequence where it holds a sink
    const int qend = s0 < a.sink ? len : (int)min((long long)len, (long long)s0 + KB - 1 + a.window);
    const int q_first = s0 / QB, per_head = (qend + QB - 1) / QB - q_first, n_it = per_head * G;
    auto fetch = [&](int i) {
      const uint32_t st = sm + KV_HELD + (i & 1) * KV_STAGE;
      const int h = kv * G + i / per_head, t0 = (q_first + i % per_head) * QB;
      const long long qtok = (long long)b * a.T * a.H + h;
      copy_rows<kCK>(st, static_cast<const T*>(a.q) + qtok * kDK, (long long)a.H * kDK, t0, QB,
                     len, tid, THREADS);
      copy_rows<kCV>(st + KV_Q, static_cast<const T*>(a.dO) + qtok * kDV, (long long)a.H * kDV, t0,
                     QB, len, tid, THREADS);
      if (tid < 2 * QB) {  // lse in base 2, then delta
        const int t = t0 + tid % QB;
        const long long at = ((long long)b * a.H + h) * a.T + t;
        float x = 0.f;
        if (t < len) x = tid < QB ? a.lse[at] * kLog2e : delta[at];
        reinterpret_cast<float*>(smem + KV_HELD + (i & 1) * KV_STAGE + KV_Q + KV_G)[tid] = x;
      }
      copy_commit();
    };
    fetch(0);
    for (int i = 0; i < n_it; ++i) {
      if (i + 1 < n_it) {
        fetch(i + 1);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      __syncthreads();
      const uint32_t qs = sm + KV_HELD + (i & 1) * KV_STAGE, gs = qs + KV_Q;
      const float* stat =
          reinterpret_cast<const float*>(smem + KV_HELD + (i & 1) * KV_STAGE + KV_Q + KV_G);
      const int t0 = (q_first + i % per_head) * QB;
      float z[QB / 8][4], dp[QB / 8][4];  // [keys, queries]
#pragma unroll
      for (int n = 0; n < QB / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = dp[n][j] = 0.f;
#pragma unroll
      for (int c = 0; c < kDK / 16; ++c) {
        uint32_t af[4];
        load_a<kCK>(af, sm, w * 16, 2 * c);
#pragma unroll
        for (int n = 0; n < QB / 8; n += 2) {
          uint32_t bf[4];
          load_b<kCK>(bf, qs, n * 8, 2 * c);
          mma16816<T>(z[n], af, bf[0], bf[1]);
          mma16816<T>(z[n + 1], af, bf[2], bf[3]);
        }
      }
#pragma unroll
      for (int c = 0; c < kDV / 16; ++c) {
        uint32_t af[4];
        load_a<kCV>(af, vs, w * 16, 2 * c);
#pragma unroll
        for (int n = 0; n < QB / 8; n += 2) {
          uint32_t bf[4];
          load_b<kCV>(bf, gs, n * 8, 2 * c);
          mma16816<T>(dp[n], af, bf[0], bf[1]);
          mma16816<T>(dp[n + 1], af, bf[2], bf[3]);
        }
      }
      const bool whole = s0 + KB - 1 <= t0 && t0 + QB <= len &&
                         (t0 + QB - 1 - s0 < a.window || s0 + KB <= a.sink);
#pragma unroll
      for (int n = 0; n < QB / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = n * 8 + t2 + (j & 1), t = t0 + c, s = s0 + w * 16 + g + (j >> 1) * 8;
          float p = ex2(fmaf(z[n][j], kLog2e, -stat[c]));
          if (!whole && (t >= len || !window_sees(t, s, a.window, a.sink))) p = 0.f;
          z[n][j] = p;
          dp[n][j] = p == 0.f ? 0.f : p * (dp[n][j] - stat[QB + c]);
        }
#pragma unroll
      for (int c = 0; c < QB / 16; ++c) {
        const uint32_t pf[4] = {pack2<T>(z[2 * c][0], z[2 * c][1]),
                                pack2<T>(z[2 * c][2], z[2 * c][3]),
                                pack2<T>(z[2 * c + 1][0], z[2 * c + 1][1]),
                                pack2<T>(z[2 * c + 1][2], z[2 * c + 1][3])};
        const uint32_t df[4] = {pack2<T>(dp[2 * c][0], dp[2 * c][1]),
                                pack2<T>(dp[2 * c][2], dp[2 * c][3]),
                                pack2<T>(dp[2 * c + 1][0], dp[2 * c + 1][1]),
                                pack2<T>(dp[2 * c + 1][2], dp[2 * c + 1][3])};
#pragma unroll
        for (int n = 0; n < kDV / 8; n += 2) {
          uint32_t bf[4];
          load_bt<kCV>(bf, gs, c * 16, n);
          mma16816<T>(dv[n], pf, bf[0], bf[1]);
          mma16816<T>(dv[n + 1], pf, bf[2], bf[3]);
        }
#pragma unroll
        for (int n = 0; n < kDK / 8; n += 2) {
          uint32_t bf[4];
          load_bt<kCK>(bf, qs, c * 16, n);
          mma16816<T>(dk[n], df, bf[0], bf[1]);
          mma16816<T>(dk[n + 1], df, bf[2], bf[3]);
        }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int s = s0 + w * 16 + g + 8 * r;
    if (s >= a.T) continue;
    const long long row = ((long long)b * a.T + s) * a.KV + kv;  // padding: the zeros it began with
    TO* ok = static_cast<TO*>(a.dk) + row * kDK;
    TO* ov = static_cast<TO*>(a.dv) + row * kDV;
    const bool live = s < len;
#pragma unroll
    for (int n = 0; n < kDK / 8; ++n)
      store2(ok + n * 8 + t2, live ? dk[n][2 * r] : 0.f, live ? dk[n][2 * r + 1] : 0.f);
#pragma unroll
    for (int n = 0; n < kDV / 8; ++n)
      store2(ov + n * 8 + t2, live ? dv[n][2 * r] : 0.f, live ? dv[n][2 * r + 1] : 0.f);
  }
}

// ---- dq: a tile of 64 queries per CTA, 16 per warp; keys in tiles of 64
constexpr int DQ_HELD = KB * (kDK + kDV) * 2, DQ_STAGE = KB * (kDK + kDV) * 2;
constexpr int DQ_SMEM = DQ_HELD + 2 * DQ_STAGE;

template <class T, class TO>
__global__ void __launch_bounds__(THREADS)
window_dq_kernel(WindowArgs a, const float* __restrict__ delta, DevCtl ctl) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem), gs = sm + KB * kDK * 2;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int tiles = (a.T + KB - 1) / KB;
  const int h = blockIdx.x % a.H;
  const long long bt = blockIdx.x / a.H;
  const int b = (int)(bt / tiles), q0 = (int)(bt % tiles) * KB;
  const int len = window_length(a.lens, b, a.T, ctl);
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int r0 = q0 + w * 16 + g;

  float dq[kDK / 8][4];
#pragma unroll
  for (int n = 0; n < kDK / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) dq[n][j] = 0.f;

  if (q0 < len) {
    const long long qtok = (long long)b * a.T * a.H + h;
    const int kv = h / (a.H / a.KV);
    const T* k = static_cast<const T*>(a.k) + ((long long)b * a.T * a.KV + kv) * kDK;
    const T* v = static_cast<const T*>(a.v) + ((long long)b * a.T * a.KV + kv) * kDV;
    copy_rows<kCK>(sm, static_cast<const T*>(a.q) + qtok * kDK, (long long)a.H * kDK, q0, KB, len,
                   tid, THREADS);
    copy_rows<kCV>(gs, static_cast<const T*>(a.dO) + qtok * kDV, (long long)a.H * kDV, q0, KB, len,
                   tid, THREADS);
    copy_commit();
    float lse[2], del[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = r0 + 8 * r;
      const long long at = ((long long)b * a.H + h) * a.T + t;
      lse[r] = t < len ? a.lse[at] * kLog2e : 0.f;
      del[r] = t < len ? delta[at] : 0.f;
    }
    const KeyTiles kt(q0, min(q0 + KB, len), KB, a.window, a.sink);
    auto fetch = [&](int i) {
      const uint32_t s = sm + DQ_HELD + (i & 1) * DQ_STAGE;
      const int s0 = kt.tile(i) * KB;
      copy_rows<kCK>(s, k, (long long)a.KV * kDK, s0, KB, len, tid, THREADS);
      copy_rows<kCV>(s + KB * kDK * 2, v, (long long)a.KV * kDV, s0, KB, len, tid, THREADS);
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
      const uint32_t ks = sm + DQ_HELD + (i & 1) * DQ_STAGE, vs = ks + KB * kDK * 2;
      const int s0 = kt.tile(i) * KB;
      float z[KB / 8][4], dp[KB / 8][4];
#pragma unroll
      for (int n = 0; n < KB / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = dp[n][j] = 0.f;
#pragma unroll
      for (int c = 0; c < kDK / 16; ++c) {
        uint32_t af[4];
        load_a<kCK>(af, sm, w * 16, 2 * c);
#pragma unroll
        for (int n = 0; n < KB / 8; n += 2) {
          uint32_t bf[4];
          load_b<kCK>(bf, ks, n * 8, 2 * c);
          mma16816<T>(z[n], af, bf[0], bf[1]);
          mma16816<T>(z[n + 1], af, bf[2], bf[3]);
        }
      }
#pragma unroll
      for (int c = 0; c < kDV / 16; ++c) {
        uint32_t af[4];
        load_a<kCV>(af, gs, w * 16, 2 * c);
#pragma unroll
        for (int n = 0; n < KB / 8; n += 2) {
          uint32_t bf[4];
          load_b<kCV>(bf, vs, n * 8, 2 * c);
          mma16816<T>(dp[n], af, bf[0], bf[1]);
          mma16816<T>(dp[n + 1], af, bf[2], bf[3]);
        }
      }
      const bool whole = s0 + KB - 1 <= q0 && s0 + KB <= len &&
                         (q0 + KB - 1 - s0 < a.window || s0 + KB <= a.sink);
#pragma unroll
      for (int n = 0; n < KB / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = r0 + (j >> 1) * 8, s = s0 + n * 8 + t2 + (j & 1);
          float p = ex2(fmaf(z[n][j], kLog2e, -lse[j >> 1]));
          if (t >= len || (!whole && (s >= len || !window_sees(t, s, a.window, a.sink)))) p = 0.f;
          dp[n][j] = p == 0.f ? 0.f : p * (dp[n][j] - del[j >> 1]);
        }
#pragma unroll
      for (int c = 0; c < KB / 16; ++c) {
        const uint32_t df[4] = {pack2<T>(dp[2 * c][0], dp[2 * c][1]),
                                pack2<T>(dp[2 * c][2], dp[2 * c][3]),
                                pack2<T>(dp[2 * c + 1][0], dp[2 * c + 1][1]),
                                pack2<T>(dp[2 * c + 1][2], dp[2 * c + 1][3])};
#pragma unroll
        for (int n = 0; n < kDK / 8; n += 2) {
          uint32_t bf[4];
          load_bt<kCK>(bf, ks, c * 16, n);
          mma16816<T>(dq[n], df, bf[0], bf[1]);
          mma16816<T>(dq[n + 1], df, bf[2], bf[3]);
        }
      }
      __syncthreads();
    }
  }
  TO* out = static_cast<TO*>(a.dq) + ((long long)b * a.T * a.H + h) * kDK;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int t = r0 + 8 * r;
    if (t >= a.T) continue;
#pragma unroll
    for (int n = 0; n < kDK / 8; ++n)  // past the sequence: the zeros it began with
      store2(out + (long long)t * a.H * kDK + n * 8 + t2, dq[n][2 * r], dq[n][2 * r + 1]);
  }
}

template <class T, class TO>
cudaError_t run(const WindowArgs& a, DevCtl ctl, cudaStream_t stream) {
  float* delta = static_cast<float*>(a.workspace);
  const long long rows = (long long)a.B * a.T * a.H, tiles = (a.T + KB - 1) / KB;
  window_delta_kernel<T, TO><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(a, delta, ctl);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto dkv = window_dkv_kernel<T, TO>;
  if ((e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, KV_SMEM)) !=
      cudaSuccess)
    return e;
  dkv<<<(unsigned)(a.B * tiles * a.KV), THREADS, KV_SMEM, stream>>>(a, delta, ctl);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  auto dq = window_dq_kernel<T, TO>;
  if ((e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, DQ_SMEM)) !=
      cudaSuccess)
    return e;
  dq<<<(unsigned)(a.B * tiles * a.H), THREADS, DQ_SMEM, stream>>>(a, delta, ctl);
  return cudaGetLastError();
}

}  // namespace

size_t window_bwd_workspace_bytes(int B, int T, int H, int KV, int window, int sink) {
  (void)KV; (void)window; (void)sink;
  return (size_t)B * T * H * sizeof(float);
}

cudaError_t launch_window_bwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  (void)n_sm;
  const bool wide = a.out_type == GLA_FP32;
  if (a.in_type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, ctl, stream);
  return wide ? run<__half, float>(a, ctl, stream) : run<__half, __half>(a, ctl, stream);
}

}  // namespace gla
