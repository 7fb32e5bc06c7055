// rotary.cu -- rotary positions: pairs of channels (a, b) of a head turned by an angle that grows
// with the token's position,
//
//   a' = s (a cos w - b sin w),  b' = s (a sin w + b cos w),  w = 2 pi turns_i pos
//
// for the R / 2 pairs of a head's first R channels (i, i + R / 2, or 2 i, 2 i + 1); the others pass.
// The gradient is the same with the angle negated.
//
// The angle is a fraction of a turn in units of 2^-64, so that pos * turns_i modulo a turn is one
// 64-bit product, exact for the table that is given, without reductions in fp64.  (A table made in double is off by
// a few 2^-53 of a pair's turns, which a position multiplies: less than 1e-9 radians a million tokens on.)  The
// nearest quarter turn is split off as whole numbers, and what is left (at most an eighth) goes to sincospi
// in fp32.
//
// Bound by HBM: each element is read and written once.  A thread has up to eight pairs of one token
// (two accesses of 16 bytes) and takes them through the heads of q and k, whose angles are the same, so
// that the sines cost about a quarter of its instructions; where tokens are few the heads are cut into
// groups for more threads.
#include <cuda_runtime.h>

#include <algorithm>

#include "elem.cuh"
#include "rotary.h"

namespace gla {
namespace {

constexpr int THREADS = 256, BATCH = 4;  // heads whose loads are in flight together

// cos and sin of a fraction of a turn in units of 2^-64.
__device__ __forceinline__ void turn(unsigned long long phase, float& c, float& s) {
  const unsigned quarter = (unsigned)((phase + (1ull << 61)) >> 62);
  const long long rest = (long long)(phase - ((unsigned long long)quarter << 62));
  float s0, c0;
  sincospif((float)(int)(rest >> 30) * 0x1p-33f, &s0, &c0);
  const float a = quarter & 1 ? s0 : c0, b = quarter & 1 ? c0 : s0;
  c = (quarter == 1 || quarter == 2) ? -a : a;
  s = quarter >= 2 ? -b : b;
}

// One rounding order for every variant, so that all give the same bits.
__device__ __forceinline__ float2 turned(float a, float b, float c, float s) {
  return make_float2(fmaf(a, c, -__fmul_rn(b, s)), fmaf(a, s, __fmul_rn(b, c)));
}
// A plain load: y may be x, which the read-only path must not see change.
template <class T, int A>
__device__ __forceinline__ void fetch(Pack<T, A>& x, const T* p) {
  if constexpr (Pack<T, A>::BYTES == 2) x.w[0] = *reinterpret_cast<const unsigned short*>(p);
  else x.load(p);
}

// A: elements of an access.  A unit is two accesses: A pairs, or up to 2 A channels that pass.
template <class TI, class TO, int A, bool INTER>
__global__ void __launch_bounds__(THREADS)
rotary_kernel(RotaryArgs a, int units, int heads_per, long long items) {
  const long long item = (long long)blockIdx.x * THREADS + threadIdx.x;
  if (item >= items) return;
  const long long token = item / units;
  const int u = (int)(item - token * units), half = a.R / 2;
  const long long b = token / a.T;
  const int t = (int)(token - b * a.T);
  const bool rot = u * A < half;
  int c0, c1;
  bool second = true;
  if (rot) {
    c0 = INTER ? 2 * A * u : A * u;
    c1 = INTER ? c0 + A : c0 + half;
  } else {
    c0 = a.R + 2 * A * (u - half / A);
    c1 = c0 + A;
    second = c1 < a.D;
  }
  float cs[A], sn[A];
  if (rot) {
    const long long pos = a.pos ? __ldg(a.pos + token) : t;
#pragma unroll
    for (int i = 0; i < A; ++i) {
      turn((unsigned long long)pos * __ldg(a.turns + u * A + i), cs[i], sn[i]);
      cs[i] *= a.scale;
      sn[i] *= a.inverse ? -a.scale : a.scale;
    }
  }
  const int all = a.q.heads + a.k.heads, h0 = blockIdx.y * heads_per;
  const int h1 = min(all, h0 + heads_per);
  for (int h = h0; h < h1; h += BATCH) {
    Pack<TI, A> x0[BATCH], x1[BATCH];
    TO* y[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const bool in_k = h + j >= a.q.heads;
      const RotaryTensor& r = in_k ? a.k : a.q;
      const int hh = in_k ? h + j - a.q.heads : h + j;
      y[j] = nullptr;
      if (h + j < h1 && (rot || r.x != r.y)) {
        const TI* x = static_cast<const TI*>(r.x) + b * r.stride[0] + t * r.stride[1] +
                      hh * r.stride[2];
        y[j] = static_cast<TO*>(r.y) + (token * r.heads + hh) * a.D;
        fetch(x0[j], x + c0);
        if (second) fetch(x1[j], x + c1);
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if (!y[j]) continue;
      Pack<TO, A> y0, y1;
      if constexpr (INTER && A > 1) {
#pragma unroll
        for (int i = 0; i < A / 2; ++i) {
          const float2 p = x0[j].get2(i), q = x1[j].get2(i);
          const float c = cs[i], s = sn[i], c2 = cs[A / 2 + i], s2 = sn[A / 2 + i];
          y0.set2(i, rot ? turned(p.x, p.y, c, s) : p);
          y1.set2(i, rot ? turned(q.x, q.y, c2, s2) : q);
        }
      } else {
#pragma unroll
        for (int i = 0; i < A; ++i) {
          const float p = x0[j].get(i), q = x1[j].get(i);
          const float2 y2 = rot ? turned(p, q, cs[i], sn[i]) : make_float2(p, q);
          y0.set(i, y2.x);
          y1.set(i, y2.y);
        }
      }
      y0.store(y[j] + c0);
      if (second) y1.store(y[j] + c1);
    }
  }
}

template <class TI, class TO, int A, bool INTER>
cudaError_t run(const RotaryArgs& a, int n_sm, cudaStream_t stream) {
  const int units = a.R / 2 / A + ((a.D - a.R) / A + 1) / 2, all = a.q.heads + a.k.heads;
  const long long items = (long long)a.B * a.T * units;
  // heads of a thread: all, or fewer where that leaves less than two CTAs an SM
  const long long fill = 2ll * n_sm * THREADS;
  int per = all;
  if (items < fill) per = (int)std::max(1ll, all * items / fill);
  const int groups = (all + per - 1) / per;
  per = (all + groups - 1) / groups;
  rotary_kernel<TI, TO, A, INTER>
      <<<dim3((unsigned)((items + THREADS - 1) / THREADS), (unsigned)groups), THREADS, 0, stream>>>(
          a, units, per, items);
  return cudaGetLastError();
}

// Whether accesses of A elements divide everything.
bool divides(const RotaryArgs& a, int A, int in_size, int out_size) {
  if (a.R / 2 % A || (a.D - a.R) % A || a.D % A) return false;
  for (const RotaryTensor* r : {&a.q, &a.k}) {
    if (!r->heads) continue;
    if (reinterpret_cast<uintptr_t>(r->x) % std::min(16, A * in_size) ||
        reinterpret_cast<uintptr_t>(r->y) % std::min(16, A * out_size))
      return false;
    for (long long s : r->stride)
      if (s % A) return false;
  }
  return true;
}

template <class TI, class TO>
cudaError_t pick(const RotaryArgs& a, int n_sm, cudaStream_t stream) {
  constexpr int W = 16 / (int)sizeof(TI);
  if (divides(a, W, sizeof(TI), sizeof(TO)))
    return a.interleaved ? run<TI, TO, W, true>(a, n_sm, stream) : run<TI, TO, W, false>(a, n_sm, stream);
  return a.interleaved ? run<TI, TO, 1, true>(a, n_sm, stream) : run<TI, TO, 1, false>(a, n_sm, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int n_sm, cudaStream_t stream) {
  const bool wide = a.out_type == GLA_FP32;
  if (a.in_type == GLA_BF16)
    return wide ? pick<__nv_bfloat16, float>(a, n_sm, stream)
                : pick<__nv_bfloat16, __nv_bfloat16>(a, n_sm, stream);
  if (a.in_type == GLA_FP16)
    return wide ? pick<__half, float>(a, n_sm, stream) : pick<__half, __half>(a, n_sm, stream);
  return pick<float, float>(a, n_sm, stream);
}

}  // namespace gla
