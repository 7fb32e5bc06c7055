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
// sigmoid(-g), taken from the same exponential, so neither loses digits where it is small.  All
// arithmetic and the carried state are fp32, in which f near 1 (long memory) keeps 1 - f only to 2^-25,
// an error of the same sign at every token.  So a thread sums 1 - a beside a over its 16 (gradient: 8)
// tokens, 1 - f a = (1 - a) + a (1 - f), and a near 1 is rounded once, not token by token: at a constant
// g = 10, x ~ 1 + N(0,1) and 50,021 tokens the state is off by 2.6e-5 where a alone gave 4.7e-4.  (Pairs
// that carry 1 - a itself from thread to thread: 2e-6, but 238 us in place of 222 at B=2 T=50021 D=1536.)
//
// Bound by HBM: a token and channel cost 8 bytes forward (bf16 x, g in, fp32 y out) and 20
// backward (x, g, y, dy in, dx, dg out), against ~20 and ~30 instructions.  One pass over memory:
// a CTA owns one sequence and 64 channels (whole 128-byte lines of 16-bit inputs; 56 so that the
// CTAs fill the last round of SMs cost 57 us where 64 took 47) and walks the tokens in tiles that
// TMA brings into a ring of three, each of its warps taking consecutive tokens of the tile.  A
// warp composes its tokens' pairs, the warps' pairs meet in shared memory, and each thread then
// runs its tokens from the state entering them.  Where sequences x slabs leave SMs idle, a
// cluster of up to 8 CTAs takes consecutive tiles of the same slab and sends its CTAs' pairs
// around through distributed shared memory, counted on barriers there (a cluster barrier in
// their place also waited for the output stores: 272 us against 216 then at B=2 T=50021 D=1536); no
// flag in global memory, no workspace, and the order of composition is fixed by the sizes, so
// results repeat bit for bit.  Measured (bf16, against the copy rate): forward B=8 T=2048 D=2048
// 47.3 us (84 %), gradient B=8 T=2047 105 us (94 %), forward B=2 T=50021 D=1536 222 us (82 %), gradient
// B=2 T=20021 294 us (62 %: a tile of 147 KB leaves one CTA an SM, so that 384 of them take three rounds).
// Rows that 16 bytes do not divide go through registers, by pairs or singly: B=8 T=2048, forward D=1022
// fp32 36 us (floor 29.6) and D=1023 bf16 41 (19.8), gradient 82 (59.3) and 92 (49.4).  Decode step, 1,280
// rows of 2048 bf16: 6.0 us from a graph with the pool in L2, 9.2 from twelve pools in turn (6.2).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>

#include "elem.cuh"
#include "gated_scan.h"
#include "tmap.h"

namespace gla {
namespace {
namespace cg = cooperative_groups;

constexpr int FWD_W = 4, BWD_W = 8;   // warps of a CTA
constexpr int FWD_S = 16, BWD_S = 8;  // tokens per warp and round
constexpr int FWD_STAGES = 3, BWD_STAGES = 3;  // rounds in flight (TMA)

// sigmoid(g) and sigmoid(-g) from e = exp(-g): f = 1 / (1 + e), and 1 - f as e f where it is the
// smaller of the two.  g = +inf gives exactly (1, 0), -inf (0, 1).
__device__ __forceinline__ void gates(float g, float& f, float& u) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(1.f + e));
  u = g >= 0.f ? e * f : 1.f - f;
}

template <int VEC>
struct alignas(8 * VEC) Pair {
  float a[VEC], b[VEC];
};
__device__ __forceinline__ float2 vec(const float (&x)[2]) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ void put(float (&x)[2], float2 y) { x[0] = y.x; x[1] = y.y; }
// A thread's pair as it goes through its tokens: a, and 1 - a beside it (u).  token2: both channels in
// one instruction, with which the forward's sum costs nothing (47.3 us at B=8 T=2048 D=2048 either way,
// one by one 49.3).
template <int VEC>
struct Compose : Pair<VEC> {
  float u[VEC];
  __device__ __forceinline__ Compose() {
#pragma unroll
    for (int j = 0; j < VEC; ++j) { this->a[j] = 1.f; this->b[j] = u[j] = 0.f; }
  }
  __device__ __forceinline__ void token(int j, float f, float g) {  // f and 1 - f
    u[j] = fmaf(this->a[j], g, u[j]);
    this->a[j] *= f;
  }
  __device__ __forceinline__ void token2(const float (&f)[VEC], const float (&g)[VEC]) {
    put(u, fma2(vec(this->a), vec(g), vec(u)));
    put(this->a, mul2(vec(this->a), vec(f)));
  }
  __device__ __forceinline__ const Pair<VEC>& pair() {
#pragma unroll
    for (int j = 0; j < VEC; ++j) this->a[j] = u[j] < 0.5f ? 1.f - u[j] : this->a[j];
    return *this;
  }
};

constexpr uint64_t DRAIN_NS = 4000000000ull;  // limit of the exit-time drain waits

// What a CTA sends to another in a round: a pair of every lane.
template <int VEC>
constexpr uint32_t kSent = 32 * sizeof(Pair<VEC>);

template <int VEC, int CL, int WARPS>
struct Exchange {
  Pair<VEC> warp[2][WARPS][32];
  Pair<VEC> cta[CL > 1 ? 2 : 1][CL > 1 ? CL : 1][32];
  alignas(8) uint64_t bar[2];  // a round's pairs of all CTAs have arrived
  alignas(8) uint64_t never;   // nothing arrives here (the give-up path's diagnostic)
  int sent[CL];                // rounds that each CTA of the cluster has sent, once it is done

  // Before the first round.  A cluster's CTAs write into each other's memory: every one has to
  // be running, with its barriers set up.
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      if constexpr (CL > 1) {
        mbar_init(smem_u32(&bar[0]), 1);
        mbar_init(smem_u32(&bar[1]), 1);
      }
      mbar_init(smem_u32(&never), 1);
      fence_barrier_init();
    }
    if constexpr (CL > 1) cg::this_cluster().sync();
  }
  // The give-up path's diagnostic: at round `stall_step` one CTA of every cluster waits for what never
  // comes, gives up and leaves without its pair, so that the waits of the others run out as well.
  __device__ __forceinline__ void stall(int r, const DevCtl& ctl, bool& ok) {
    if (r == ctl.stall_step && cg::this_cluster().block_rank() == CL - 1)
      ok = ok && mbar_wait(smem_u32(&never), 0, ctl);
  }
  // After the last round, or the one before which the CTA gave up; `rounds`: the ones it has sent.
  // No CTA leaves while a pair may still be on its way into its memory.  One that has gone through
  // all its waits has everything that was ever sent to it.  One that gave up learns how far the
  // others got and waits for just that: of its last round the pairs of those that sent it, and of
  // the next one, which nobody can be past without this CTA's pair, the same.
  __device__ __forceinline__ void done(int rounds, bool ok, const DevCtl& ctl) {
    if constexpr (CL > 1) {
      ok = __syncthreads_and(ok);
      if (threadIdx.x < 32) {  // only these lanes' stores, not the outputs, are waited for
        if (threadIdx.x < CL)
          *cg::this_cluster().map_shared_rank(&sent[cg::this_cluster().block_rank()],
                                              threadIdx.x) = rounds;
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      } else {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      }
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (!ok && threadIdx.x == 0) {
        int behind = 0, ahead = 0;
        for (int k = 0; k < CL; ++k) {
          behind += sent[k] < rounds;
          ahead += sent[k] > rounds;
        }
        if (rounds > 0) {  // armed for all CTAs' pairs
          const uint32_t b = smem_u32(&bar[(rounds - 1) & 1]);
          if (behind) mbar_complete_tx(b, behind * kSent<VEC>);
          mbar_wait(b, ((rounds - 1) >> 1) & 1, ctl, DRAIN_NS);
        }
        if (ahead) {  // not armed
          const uint32_t b = smem_u32(&bar[rounds & 1]);
          mbar_arrive_expect_tx(b, ahead * kSent<VEC>);
          mbar_wait(b, (rounds >> 1) & 1, ctl, DRAIN_NS);
        }
      }
    }
  }
};

// A pair into CTA `to`'s copy of *p; its bytes count on that CTA's copy of the barrier.  (A
// cluster barrier in its place would wait for the round's output stores as well.)
template <int VEC>
__device__ __forceinline__ void send(const Pair<VEC>& v, const Pair<VEC>* p, const uint64_t* bar,
                                     int to) {
  uint32_t rp, rb;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rp) : "r"(smem_u32(p)), "r"(to));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(smem_u32(bar)), "r"(to));
  if constexpr (VEC == 2)
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
        ::"r"(rp), "r"(__float_as_uint(v.a[0])), "r"(__float_as_uint(v.a[1])),
          "r"(__float_as_uint(v.b[0])), "r"(__float_as_uint(v.b[1])), "r"(rb)
        : "memory");
  else
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(rp),
        "r"(__float_as_uint(v.a[0])), "r"(__float_as_uint(v.b[0])), "r"(rb)
        : "memory");
}

// The state entering this warp's tokens, from round r's pair of every warp (and CTA of the
// cluster) and the state `carry` entering the round, which becomes the one leaving it.  `ok`
// turns false where a CTA of the cluster did not answer in time.  A cluster's CTA in which a
// thread has given up sends no more: enter() is then false in all its threads, which leave.
template <int VEC, int CL, int WARPS>
__device__ __forceinline__ bool enter(Exchange<VEC, CL, WARPS>& ex, int r, const Pair<VEC>& own,
                                      float (&carry)[VEC], float (&in)[VEC], const DevCtl& ctl,
                                      bool& ok) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, buf = r & 1;
  ex.warp[buf][w][lane] = own;
  // The buffers alternate: a CTA sends round r + 2 only after it has this one's pairs of round
  // r + 1, which go out behind a barrier that every thread reaches after it has read round r's.
  if constexpr (CL > 1) {
    ex.stall(r, ctl, ok);
    if (!__syncthreads_and(ok)) return ok = false;
    const int rank = (int)cg::this_cluster().block_rank();
    if (threadIdx.x == 0) mbar_arrive_expect_tx(smem_u32(&ex.bar[buf]), CL * kSent<VEC>);
    if (w < CL) {
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
      for (int to = w; to < CL; to += WARPS)  // each warp hands the CTA's pair to some of them
        send(p, &ex.cta[buf][rank][lane], &ex.bar[buf], to);
    }
    ok = mbar_wait(smem_u32(&ex.bar[buf]), (r >> 1) & 1, ctl);
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
    __syncthreads();
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
  return true;
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
__global__ void __launch_bounds__(32 * FWD_W, 3)
scan_fwd_kernel(const T* __restrict__ x, const T* __restrict__ g, const float* __restrict__ init,
                const int* __restrict__ lens, float* __restrict__ y, float* __restrict__ fin,
                int T_, int D, int slabs, DevCtl ctl) {
  constexpr int S = FWD_S, WARPS = FWD_W, TILE = WARPS * S;
  __shared__ Exchange<VEC, CL, FWD_W> ex;
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
    if (t0 + S <= len && live) {
      const T* xp = x + base + (long long)t0 * D;
      const T* gp = g + base + (long long)t0 * D;
#pragma unroll
      for (int i = 0; i < S; ++i, xp += D, gp += D) {
        xr[i].load(xp);
        gr[i].load(gp);
      }
      return;
    }
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
  ex.init();
  bool ok = true;
  int r = 0;
  for (int at = 0; at < T_; at += step, t0 += step, ++r) {
    float f[S][VEC], a[S][VEC];
    Compose<VEC> own;
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float u;
        gates(gr[i].get(j), f[i][j], u);
        a[i][j] = u * xr[i].get(j);
        own.b[j] = fmaf(f[i][j], own.b[j], a[i][j]);
        own.token(j, f[i][j], u);
      }
    if (at + step < T_) fetch(t0 + step);
    float h[VEC];
    if (!enter(ex, r, own.pair(), carry, h, ctl, ok)) break;
    const bool whole = t0 + S <= len;
    float* yp = y + base + (long long)t0 * D;
#pragma unroll
    for (int i = 0; i < S; ++i, yp += D) {
      Pack<float, VEC> out;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        h[j] = fmaf(f[i][j], h[j], a[i][j]);
        out.set(j, whole || t0 + i < len ? h[j] : 0.f);
      }
      if (live && (whole || t0 + i < T_)) out.store(yp);
    }
  }
  if (fin && live && rank == 0 && w == 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) fin[(long long)b * D + ch + j] = carry[j];
  ex.done(r, ok, ctl);
}

template <class T, int VEC, int CL>
__global__ void __launch_bounds__(32 * BWD_W, 2)
scan_bwd_kernel(const T* __restrict__ x, const T* __restrict__ g, const float* __restrict__ y,
                const float* __restrict__ dy, const float* __restrict__ init,
                const float* __restrict__ dfin, const int* __restrict__ lens,
                float* __restrict__ dx, float* __restrict__ dg, float* __restrict__ dinit, int T_,
                int D, int slabs, DevCtl ctl) {
  constexpr int S = BWD_S, WARPS = BWD_W, TILE = WARPS * S;
  __shared__ Exchange<VEC, CL, BWD_W> ex;
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
  ex.init();
  bool ok = true;
  int r = 0;
  for (int at = 0; at < T_; at += step, ++r) {
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
    Compose<VEC> own;
    float f[S][VEC], u[S][VEC];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        gates(gr[i].get(j), f[i][j], u[i][j]);
        own.b[j] = f[i][j] * (own.b[j] + dr[i].get(j));
        own.token(j, f[i][j], u[i][j]);
      }
    float c[VEC];
    if (!enter(ex, r, own.pair(), carry, c, ctl, ok)) break;
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
  ex.done(r, ok, ctl);
}

// ---- the same with tiles brought in by TMA, where rows start on 16 bytes
//
// A ring of STAGES tiles of 64 channels in shared memory takes the place of the registers that
// held the next round's inputs: more rounds in flight, no address arithmetic.  The barrier of
// enter() also frees the tile just read.  Tokens past a sequence's end may hold anything: their
// tiles are read, and the values not used.
constexpr int SLAB = 64;  // channels of a CTA: whole 128-byte lines of 16-bit inputs

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int ch, int t, int b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ch), "r"(t), "r"(b), "r"(bar)
      : "memory");
}
// Two adjacent values of a row in shared memory.
template <class T>
__device__ __forceinline__ float2 tile_pair(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float2*>(p);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (__is_same(T, __half)) return __half22float2(reinterpret_cast<const __half2&>(w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}

template <class T, int CL, int STAGES>
__global__ void __launch_bounds__(32 * FWD_W)
scan_fwd_tma_kernel(const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_g, const float* __restrict__ init,
                    const int* __restrict__ lens, float* __restrict__ y, float* __restrict__ fin,
                    int T_, int D, int slabs, DevCtl ctl) {
  constexpr int S = FWD_S, WARPS = FWD_W, TILE = WARPS * S, BYTES = TILE * SLAB * (int)sizeof(T);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Exchange<2, CL, FWD_W> ex;
  __shared__ alignas(8) uint64_t full[STAGES];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = CL > 1 ? blockIdx.x % CL : 0, unit = blockIdx.x / CL;
  const int b = unit / slabs, ch0 = (unit % slabs) * SLAB, ch = ch0 + 2 * lane;
  const bool live = ch < D;
  const int len = length_of(lens, b, T_, ctl);
  const int step = TILE * CL, rounds = (int)(((long long)len + step - 1) / step);
  int armed = 0;  // rounds fetched so far
  auto fetch = [&](int r) {  // one thread
    armed = r + 1;
    const int s = r % STAGES;
    const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(smem) + s * 2 * BYTES;
    const int t = r * step + rank * TILE;
    mbar_arrive_expect_tx(bar, 2 * BYTES);
    load_tile(dst, &map_x, bar, ch0, t, b);
    load_tile(dst + BYTES, &map_g, bar, ch0, t, b);
  };
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_barrier_init();
    fence_proxy_async();
    for (int r = 0; r < STAGES && r < rounds; ++r) fetch(r);
  }
  float carry[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) carry[j] = live && init ? init[(long long)b * D + ch + j] : 0.f;
  ex.init();
  __syncthreads();
  float* const yb = y + (long long)b * T_ * D + ch;

  bool ok = true;
  int r = 0;
  for (; r < rounds; ++r) {
    const int s = r % STAGES;
    const T* xt = reinterpret_cast<const T*>(smem + s * 2 * BYTES) + w * S * SLAB + 2 * lane;
    const T* gt = xt + TILE * SLAB;
    const int t0 = r * step + rank * TILE + w * S;
    const bool whole = t0 + S <= len;
    // (without clusters the diagnostic takes the place of the tile's barrier: as a wait of its own
    // it cost 49.0 us in place of 47.2)
    const bool stall = CL == 1 && r == ctl.stall_step;
    ok = ok && mbar_wait(smem_u32(stall ? &ex.never : &full[s]), stall ? 0 : (r / STAGES) & 1, ctl);
    float f[S][2], a[S][2];
    Compose<2> own;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float2 xv = tile_pair(xt + i * SLAB), gv = tile_pair(gt + i * SLAB);
      float u[2];
      gates(gv.x, f[i][0], u[0]);
      gates(gv.y, f[i][1], u[1]);
      put(a[i], mul2(vec(u), xv));
      if (!whole && t0 + i >= len) {  // past the sequence: the identity
        f[i][0] = f[i][1] = 1.f;
        a[i][0] = a[i][1] = u[0] = u[1] = 0.f;
      }
      put(own.b, fma2(vec(f[i]), vec(own.b), vec(a[i])));
      own.token2(f[i], u);
    }
    float h[2];
    if (!enter(ex, r, own.pair(), carry, h, ctl, ok)) break;
    if (tid == 0 && ok && r + STAGES < rounds) fetch(r + STAGES);
    float* yp = yb + (long long)t0 * D;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      put(h, fma2(vec(f[i]), vec(h), vec(a[i])));
      if (live && (whole || t0 + i < T_))
        __stcs(reinterpret_cast<float2*>(yp + (long long)i * D),
               whole || t0 + i < len ? make_float2(h[0], h[1]) : make_float2(0.f, 0.f));
    }
  }
  // after a wait that gave up nothing is fetched any more; the copies in flight land before the
  // CTA's memory is given back
  if (!ok && tid == 0)
    for (int k = max(0, armed - STAGES); k < armed; ++k)
      mbar_wait(smem_u32(&full[k % STAGES]), (k / STAGES) & 1, ctl, DRAIN_NS);
  // the padding that no round has reached
  for (int t = rounds * step + rank * WARPS + w; t < T_; t += WARPS * CL)
    if (live) __stcs(reinterpret_cast<float2*>(yb + (long long)t * D), make_float2(0.f, 0.f));
  if (fin && live && rank == 0 && w == 0)
    *reinterpret_cast<float2*>(fin + (long long)b * D + ch) = make_float2(carry[0], carry[1]);
  ex.done(r, ok, ctl);
}

template <class T, int CL, int STAGES>
__global__ void __launch_bounds__(32 * BWD_W)
scan_bwd_tma_kernel(const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_g,
                    const __grid_constant__ CUtensorMap map_y,
                    const __grid_constant__ CUtensorMap map_dy, const float* __restrict__ init,
                    const float* __restrict__ dfin, const int* __restrict__ lens,
                    float* __restrict__ dx, float* __restrict__ dg, float* __restrict__ dinit,
                    int T_, int D, int slabs, DevCtl ctl) {
  constexpr int S = BWD_S, WARPS = BWD_W, TILE = WARPS * S, BX = TILE * SLAB * (int)sizeof(T);
  constexpr int BY = TILE * SLAB * 4, STAGE = 2 * BX + 2 * BY;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Exchange<2, CL, BWD_W> ex;
  __shared__ alignas(8) uint64_t full[STAGES];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = CL > 1 ? blockIdx.x % CL : 0, unit = blockIdx.x / CL;
  const int b = unit / slabs, ch0 = (unit % slabs) * SLAB, ch = ch0 + 2 * lane;
  const bool live = ch < D;
  const int len = length_of(lens, b, T_, ctl);
  const long long edge = (long long)b * D + ch;
  const int step = TILE * CL, rounds = (int)(((long long)len + step - 1) / step);
  // round r, from the sequence's last token: this CTA's tile starts at token
  auto tile_at = [&](int r) { return len - (r * step + rank * TILE) - TILE; };
  int armed = 0;  // rounds fetched so far
  auto fetch = [&](int r) {  // one thread; a tile may begin before the sequence: zeros there
    armed = r + 1;
    const int s = r % STAGES, t = tile_at(r);
    const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(smem) + s * STAGE;
    mbar_arrive_expect_tx(bar, STAGE);
    load_tile(dst, &map_x, bar, ch0, t, b);
    load_tile(dst + BX, &map_g, bar, ch0, t, b);
    load_tile(dst + 2 * BX, &map_y, bar, ch0, t - 1, b);
    load_tile(dst + 2 * BX + BY, &map_dy, bar, ch0, t, b);
  };
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_barrier_init();
    fence_proxy_async();
    for (int r = 0; r < STAGES && r < rounds; ++r) fetch(r);
  }
  float carry[2], first[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    carry[j] = live && dfin ? dfin[edge + j] : 0.f;
    first[j] = live && init ? init[edge + j] : 0.f;
  }
  ex.init();
  __syncthreads();
  float* const xb = dx + (long long)b * T_ * D + ch;
  float* const gb = dg + (long long)b * T_ * D + ch;

  bool ok = true;
  int r = 0;
  for (; r < rounds; ++r) {
    const int s = r % STAGES;
    const int row = TILE - 1 - w * S, last = tile_at(r) + row;  // this warp's last token
    const T* xt = reinterpret_cast<const T*>(smem + s * STAGE) + row * SLAB + 2 * lane;
    const T* gt = xt + TILE * SLAB;
    const float* yt =
        reinterpret_cast<const float*>(smem + s * STAGE + 2 * BX) + row * SLAB + 2 * lane;
    const float* dt = yt + TILE * SLAB;
    const bool whole = last - S >= 0;  // past its first token too
    const bool stall = CL == 1 && r == ctl.stall_step;
    ok = ok && mbar_wait(smem_u32(stall ? &ex.never : &full[s]), stall ? 0 : (r / STAGES) & 1, ctl);
    float f[S][2], v[S][2], d[S][2], k[S][2];  // f, 1 - f, dy, f (1 - f) (h_{t-1} - x)
    Compose<2> own;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float2 x2 = tile_pair(xt - i * SLAB), g2 = tile_pair(gt - i * SLAB);
      const float2 y2 = tile_pair(yt - i * SLAB), d2 = tile_pair(dt - i * SLAB);
      const float xs[2] = {x2.x, x2.y}, gs[2] = {g2.x, g2.y};
      float ys[2] = {y2.x, y2.y};
      d[i][0] = d2.x;
      d[i][1] = d2.y;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        gates(gs[j], f[i][j], v[i][j]);
        if (!whole && last - i == 0) ys[j] = first[j];
        k[i][j] = f[i][j] * v[i][j] * (ys[j] - xs[j]);
        if (!whole && last - i < 0) {  // before the sequence: the identity
          f[i][j] = 1.f;
          v[i][j] = d[i][j] = k[i][j] = 0.f;
        }
      }
      // (in one instruction for both channels; in a cluster that was slower, 304 us against 297 at B=2
      // T=20021 D=1536)
      if constexpr (CL == 1) {
        put(own.b, mul2(vec(f[i]), add2(vec(own.b), vec(d[i]))));
        own.token2(f[i], v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          own.b[j] = f[i][j] * (own.b[j] + d[i][j]);
          own.token(j, f[i][j], v[i][j]);
        }
      }
    }
    float c[2];
    if (!enter(ex, r, own.pair(), carry, c, ctl, ok)) break;
    if (tid == 0 && ok && r + STAGES < rounds) fetch(r + STAGES);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float G[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        G[j] = d[i][j] + c[j];
        c[j] = f[i][j] * G[j];
      }
      if (live && (whole || last - i >= 0)) {
        const long long p = (long long)(last - i) * D;
        __stcs(reinterpret_cast<float2*>(xb + p), make_float2(v[i][0] * G[0], v[i][1] * G[1]));
        __stcs(reinterpret_cast<float2*>(gb + p), make_float2(k[i][0] * G[0], k[i][1] * G[1]));
      }
    }
  }
  // after a wait that gave up nothing is fetched any more; the copies in flight land before the
  // CTA's memory is given back
  if (!ok && tid == 0)
    for (int k = max(0, armed - STAGES); k < armed; ++k)
      mbar_wait(smem_u32(&full[k % STAGES]), (k / STAGES) & 1, ctl, DRAIN_NS);
  for (int t = len + rank * WARPS + w; t < T_; t += WARPS * CL)  // padding
    if (live) {
      __stcs(reinterpret_cast<float2*>(xb + (long long)t * D), make_float2(0.f, 0.f));
      __stcs(reinterpret_cast<float2*>(gb + (long long)t * D), make_float2(0.f, 0.f));
    }
  if (dinit && live && rank == 0 && w == 0)
    *reinterpret_cast<float2*>(dinit + edge) = make_float2(carry[0], carry[1]);
  ex.done(r, ok, ctl);
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
    // h + u (x - h) where f is near 1 (of an infinite h that would be none)
    const float xj = xr.get(j), hj = h.get(j), r = fmaf(u, xj - hj, hj);
    h.set(j, u < 0.5f && fabsf(r) < INFINITY ? r : fmaf(f, hj, u * xj));
  }
  h.store(sp);
  h.store(y + at);
}

// CTAs of a cluster along the tokens: the fewest (1, 2, 4, 8) that give the SMs one and a half
// CTAs each, and no more than there are tiles.
int pick_cluster(long long units, int T, int tile, int n_sm) {
  const int tiles = (T + tile - 1) / tile;
  int cl = 1;
  while (cl < 8 && units * cl * 2 < 3ll * n_sm && cl * 2 <= tiles) cl *= 2;
  return cl;
}

template <class K, class... A>
cudaError_t launch(K kernel, int cl, int warps, long long units, int smem, cudaStream_t stream, A... args) {
  if (smem > 0) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * cl));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// f.go<CL>() for the cluster size at hand.
template <class F>
cudaError_t with_cluster(int cl, const F& f) {
  return cl == 1 ? f.template go<1>() : cl == 2 ? f.template go<2>()
         : cl == 4 ? f.template go<4>() : f.template go<8>();
}

// [B, T, D] as {D, T, B}, in boxes of SLAB channels and `rows` tokens.
template <class T>
bool scan_map(CUtensorMap* m, const void* p, const ScanArgs& a, int rows) {
  const unsigned long long dims[3] = {(unsigned long long)a.D, (unsigned long long)a.T,
                                      (unsigned long long)a.B};
  const unsigned long long strides[2] = {a.D * sizeof(T), a.D * sizeof(T) * a.T};
  const unsigned box[3] = {(unsigned)SLAB, (unsigned)rows, 1};
  const CUtensorMapDataType t = sizeof(T) == 4          ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : __is_same(T, __half) ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return make_tmap_3d(m, p, t, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <class T>
struct FwdTma {
  const ScanArgs& a;
  long long units;
  int slabs;
  DevCtl ctl;
  cudaStream_t stream;
  template <int CL>
  cudaError_t go() const {
    constexpr int ST = FWD_STAGES, TILE = FWD_W * FWD_S;
    CUtensorMap x, g;
    if (!scan_map<T>(&x, a.x, a, TILE) || !scan_map<T>(&g, a.g, a, TILE))
      return cudaErrorInvalidValue;
    return launch(scan_fwd_tma_kernel<T, CL, ST>, CL, FWD_W, units,
                  ST * 2 * TILE * SLAB * (int)sizeof(T), stream, x, g, a.init, a.lens, a.y, a.fin,
                  a.T, a.D, slabs, ctl);
  }
};
template <class T>
struct BwdTma {
  const ScanArgs& a;
  long long units;
  int slabs;
  DevCtl ctl;
  cudaStream_t stream;
  template <int CL>
  cudaError_t go() const {
    constexpr int ST = BWD_STAGES, TILE = BWD_W * BWD_S;
    CUtensorMap x, g, y, dy;
    if (!scan_map<T>(&x, a.x, a, TILE) || !scan_map<T>(&g, a.g, a, TILE) ||
        !scan_map<float>(&y, a.y, a, TILE) || !scan_map<float>(&dy, a.dy, a, TILE))
      return cudaErrorInvalidValue;
    return launch(scan_bwd_tma_kernel<T, CL, ST>, CL, BWD_W, units,
                  ST * 2 * TILE * SLAB * ((int)sizeof(T) + 4), stream, x, g, y, dy, a.init, a.dfin,
                  a.lens, a.dx, a.dg, a.dinit, a.T, a.D, slabs, ctl);
  }
};
template <class T, int VEC>
struct FwdReg {
  const ScanArgs& a;
  long long units;
  int slabs;
  DevCtl ctl;
  cudaStream_t stream;
  template <int CL>
  cudaError_t go() const {
    return launch(scan_fwd_kernel<T, VEC, CL>, CL, FWD_W, units, 0, stream, (const T*)a.x,
                  (const T*)a.g, a.init, a.lens, a.y, a.fin, a.T, a.D, slabs, ctl);
  }
};
template <class T, int VEC>
struct BwdReg {
  const ScanArgs& a;
  long long units;
  int slabs;
  DevCtl ctl;
  cudaStream_t stream;
  template <int CL>
  cudaError_t go() const {
    return launch(scan_bwd_kernel<T, VEC, CL>, CL, BWD_W, units, 0, stream, (const T*)a.x,
                  (const T*)a.g, (const float*)a.y, a.dy, a.init, a.dfin, a.lens, a.dx, a.dg,
                  a.dinit, a.T, a.D, slabs, ctl);
  }
};

template <class T>
cudaError_t scan_typed(const ScanArgs& a, bool backward, int n_sm, DevCtl ctl,
                       cudaStream_t stream) {
  // TMA where rows of the inputs start on 16 bytes, two channels per lane where they start on a
  // pair (D even), else one
  const bool tma = a.D % (16 / (int)sizeof(T)) == 0;
  const int vec = a.D % 2 == 0 ? 2 : 1;
  const int slabs = (a.D + 32 * vec - 1) / (32 * vec);
  const long long units = (long long)a.B * slabs;
  const int cl = pick_cluster(units, a.T, backward ? BWD_W * BWD_S : FWD_W * FWD_S, n_sm);
  if (tma)
    return backward ? with_cluster(cl, BwdTma<T>{a, units, slabs, ctl, stream})
                    : with_cluster(cl, FwdTma<T>{a, units, slabs, ctl, stream});
  if (vec == 2)
    return backward ? with_cluster(cl, BwdReg<T, 2>{a, units, slabs, ctl, stream})
                    : with_cluster(cl, FwdReg<T, 2>{a, units, slabs, ctl, stream});
  return backward ? with_cluster(cl, BwdReg<T, 1>{a, units, slabs, ctl, stream})
                  : with_cluster(cl, FwdReg<T, 1>{a, units, slabs, ctl, stream});
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
