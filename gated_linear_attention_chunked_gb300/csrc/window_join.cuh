// window_join.cuh -- one row of the windowed attention from the parts of its keys, by one block:
//
//   o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p,  m = max_p m_p
//
// Bound by the latency of its loads, so all of them are on their way at once: a part's o by one of four teams
// of threads, up to 16 parts each, while one warp finds the factors.  (One thread's loads behind one another
// took 10 us for 43 parts, and 16 us for eight of 592 rows.)  Sums in a fixed order: the same bits each time.
#pragma once
#include "mma.cuh"
#include "window_common.cuh"

namespace gla {

constexpr int kMostParts = 64, JOIN_TEAMS = 4, JOIN_THREADS = JOIN_TEAMS * kDV / 2;

// ml(p): (m_p, l_p); o(p): row o_p, read also where m_p is -infinity, and then not used.
template <class TO, class ML, class O>
__device__ __forceinline__ void join_row(int parts, ML ml, O o, TO* out) {
  __shared__ float factor[kMostParts], inv;
  __shared__ float2 sums[JOIN_TEAMS][kDV / 2];
  constexpr int EACH = kMostParts / JOIN_TEAMS;
  const int tid = threadIdx.x, team = tid / (kDV / 2), pair = tid % (kDV / 2);
  float2 x[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int p = team + JOIN_TEAMS * i;
    x[i] = p < parts ? reinterpret_cast<const float2*>(o(p))[pair] : make_float2(0.f, 0.f);
  }
  if (tid < 32) {
    static_assert(kMostParts == 64, "two parts a lane");
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 a = tid < parts ? ml(tid) : none, b = tid + 32 < parts ? ml(tid + 32) : none;
    float top = fmaxf(a.x, b.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float fa = a.x == -INFINITY ? 0.f : ex2(a.x - top), fb = b.x == -INFINITY ? 0.f : ex2(b.x - top);
    float sum = (fa == 0.f ? 0.f : fa * a.y) + (fb == 0.f ? 0.f : fb * b.y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    factor[tid] = fa;
    factor[tid + 32] = fb;
    if (tid == 0) inv = 1.f / sum;  // the token itself is in one of the parts: sum > 0
  }
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const float f = factor[team + JOIN_TEAMS * i];
    if (f != 0.f) s = make_float2(fmaf(f, x[i].x, s.x), fmaf(f, x[i].y, s.y));
  }
  sums[team][pair] = s;
  __syncthreads();
  if (team) return;
#pragma unroll
  for (int i = 1; i < JOIN_TEAMS; ++i) s = make_float2(s.x + sums[i][pair].x, s.y + sums[i][pair].y);
  store2(out + 2 * pair, s.x * inv, s.y * inv);
}

}  // namespace gla
