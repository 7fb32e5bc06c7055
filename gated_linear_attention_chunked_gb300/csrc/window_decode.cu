// window_decode.cu -- the windowed attention (window_fwd.cu) one token at a time, over caches of
// fixed size: a sequence's page holds its first `sink` tokens in slots 0 .. sink - 1 and the
// last `window` others in a ring behind them, token t in slot sink + (t - sink) % window.  After
// token t the filled slots 0 .. min(t + 1, sink + window) - 1 are exactly the keys that t sees,
// so the step needs no mask, and a softmax does not ask for their order.
//
// Bound by HBM: each key and value of the page is read once (576 bytes of 16-bit type) and used
// by the H / KV heads that share it.  Those heads are the 16 rows of a tensor-core product, of
// which a head count below 16 leaves some idle: the products stay far below the memory time.  A
// CTA takes one sequence, key head and part of the slots; its warps walk the slots in tiles of 16
// with rings of their own in shared memory (asynchronous copies, no barrier between warps) and
// running maxima and sums of their own, which they join at the end.
//
// The device holds two CTAs an SM (rings of three stages; with four, one fits, 123 us in place of the
// 101 then at 256 sequences of mixed ages, 1,028 slots, four key heads).  As many whole units (sequence, key head,
// group of query heads) as fill it one or more times run uncut; the slots of the others are cut
// into the parts that fill the last round, joined by a second kernel in a fixed order.  Measured,
// bf16, 1,028 slots, all filled, 16 heads on four, from a graph: 8 sequences 11.9 us (with parts for
// two rounds of all units 16.0), 64: 29.5 (42.1), 100: 49.0 (54.3), 128: 55.8 (68.5), 256: 106.1
// (111.8; 84 % of the copy rate); 2 sequences of 8,196 slots, 32 heads on four: 19.9 (28.5).  256
// sequences of mixed ages, a quarter of them still filling their page (79 us at the copy rate): 95.2,
// 97 a call.  The cache fill, one warp a slot, copies 64 prompts of 2,048 tokens into such pages in 56 us
// (45 at the copy rate), 256 in 211 (179), one of 8,192 in 2.9.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "window_common.cuh"

namespace gla {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS, SB = 16, STAGES = 3, HB = 16;
constexpr int STAGE = SB * (kDK + kDV) * 2;  // 9,216 bytes: a warp's tile of 16 slots
constexpr int RING = WARPS * STAGES * STAGE;
constexpr int SMEM = RING + HB * kDK * 2;

// CTAs: a unit each for the first `whole` units, `parts` for each of the `cut` others.
struct DecodePlan {
  int whole, cut, parts, part_slots;
};

__device__ __forceinline__ int slot_of(int t, int window, int sink) {
  return t < sink ? t : sink + (t - sink) % window;
}

template <class T, class TO>
__global__ void __launch_bounds__(THREADS)
window_decode_kernel(WindowDecodeArgs a, DecodePlan plan, int groups, DevCtl ctl) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int KV = a.c.KV, G = a.H / KV;
  griddep_launch_dependents();  // the join waits for this whole grid
  const int cut = (int)blockIdx.x - plan.whole;  // < 0: a whole unit
  const int parts = cut < 0 ? 1 : plan.parts, part = cut < 0 ? 0 : cut % parts;
  const int part_slots = cut < 0 ? 1 << 30 : plan.part_slots;
  const int unit = cut < 0 ? (int)blockIdx.x : plan.whole + cut / parts;
  const int grp = unit % groups, nk = unit / groups;
  const int kv = nk % KV, n = nk / KV;
  const int h0 = grp * HB, heads = min(HB, G - h0);  // of this key head's query heads
  const int page = __ldg(a.c.page + n), pos = __ldg(a.pos + n);
  const bool ok = page >= 0 && page < a.c.n_pages && pos >= 0;  // the same for the whole CTA
  if (!ok && tid == 0) record_error(ctl, DEV_RANGE);
  if (!ok && parts == 1) return;

  const int slots = a.c.window + a.c.sink;
  const int held = ok ? (int)min((long long)pos + 1, (long long)slots) : 0;
  const int lo = part * part_slots, hi = min(held, lo + part_slots);
  const int mine = ok ? slot_of(pos, a.c.window, a.c.sink) : 0;
  const long long at = ((long long)(ok ? page : 0) * a.c.pool_layers + a.c.layer) * slots;
  T* pk = static_cast<T*>(a.c.k) + (at * KV + kv) * kDK;
  T* pv = static_cast<T*>(a.c.v) + (at * KV + kv) * kDV;
  const T* nk_ = static_cast<const T*>(a.k) + ((long long)n * KV + kv) * kDK;
  const T* nv_ = static_cast<const T*>(a.v) + ((long long)n * KV + kv) * kDV;
  const T* q = static_cast<const T*>(a.q) + ((long long)n * a.H + kv * G + h0) * kDK;

  // the new token's key and value go into their slot (read below from the call's own tensors)
  if (ok && grp == 0 && mine >= lo && mine < hi && tid < kCK + kCV) {
    if (tid < kCK)
      reinterpret_cast<uint4*>(pk + (long long)mine * KV * kDK)[tid] =
          __ldg(reinterpret_cast<const uint4*>(nk_) + tid);
    else
      reinterpret_cast<uint4*>(pv + (long long)mine * KV * kDV)[tid - kCK] =
          __ldg(reinterpret_cast<const uint4*>(nv_) + tid - kCK);
  }

  const uint32_t ring = sm + w * STAGES * STAGE;
  const int tiles = hi > lo ? (hi - lo + SB * WARPS - 1) / (SB * WARPS) : 0;
  auto fetch = [&](int i) {  // warp w's tile i: slots lo + (i WARPS + w) SB ..
    if (i < tiles) {
      const int s0 = lo + (i * WARPS + w) * SB;
      const uint32_t st = ring + (i % STAGES) * STAGE;
#pragma unroll
      for (int e = 0; e < SB * kCK / 32; ++e) {
        const int x = e * 32 + lane, r = x / kCK, c = x % kCK, s = s0 + r;
        copy16(st + tile_off<kCK>(r, c),
               (s == mine ? nk_ : pk + (long long)(s < hi ? s : lo) * KV * kDK) + c * 8, s < hi);
      }
#pragma unroll
      for (int e = 0; e < SB * kCV / 32; ++e) {
        const int x = e * 32 + lane, r = x / kCV, c = x % kCV, s = s0 + r;
        copy16(st + SB * kDK * 2 + tile_off<kCV>(r, c),
               (s == mine ? nv_ : pv + (long long)(s < hi ? s : lo) * KV * kDV) + c * 8, s < hi);
      }
    }
    copy_commit();
  };
  // queries: 16 rows, zeros behind the group's heads
  for (int x = tid; x < HB * kCK; x += THREADS) {
    const int r = x / kCK, c = x % kCK;
    copy16(sm + RING + tile_off<kCK>(r, c), q + (r < heads ? r : 0) * kDK + c * 8, r < heads);
  }
  copy_commit();
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  copy_wait<STAGES - 1>();
  __syncthreads();
  uint32_t qf[kDK / 16][4];
#pragma unroll
  for (int c = 0; c < kDK / 16; ++c) load_a<kCK>(qf[c], sm + RING, 0, 2 * c);

  const int g = lane >> 2, t2 = (lane & 3) * 2;
  float acc[kDV / 8][4];
#pragma unroll
  for (int c = 0; c < kDV / 8; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[c][j] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int i = 0; i < tiles; ++i) {
    fetch(i + STAGES - 1);
    copy_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t ks = ring + (i % STAGES) * STAGE, vs = ks + SB * kDK * 2;
    const int s0 = lo + (i * WARPS + w) * SB;
    float z[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) z[c][j] = 0.f;
#pragma unroll
    for (int c = 0; c < kDK / 16; ++c) {
      uint32_t bf[4];
      load_b<kCK>(bf, ks, 0, 2 * c);
      mma16816<T>(z[0], qf[c], bf[0], bf[1]);
      mma16816<T>(z[1], qf[c], bf[2], bf[3]);
    }
    if (s0 + SB > hi)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (s0 + c * 8 + t2 + (j & 1) >= hi) z[c][j] = -INFINITY;
    float p[2][4];
    uint32_t pf[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = fmaxf(fmaxf(z[0][2 * r], z[0][2 * r + 1]), fmaxf(z[1][2 * r], z[1][2 * r + 1]));
      top = fmaxf(m[r], quad_max(top));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = ex2((m[r] - base) * kLog2e);
      m[r] = top;
      l[r] *= keep;
#pragma unroll
      for (int c = 0; c < kDV / 8; ++c) {
        acc[c][2 * r] *= keep;
        acc[c][2 * r + 1] *= keep;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p[c][2 * r + j] = ex2((z[c][2 * r + j] - base) * kLog2e);
          l[r] += p[c][2 * r + j];
        }
      pf[r] = pack2<T>(p[0][2 * r], p[0][2 * r + 1]);
      pf[2 + r] = pack2<T>(p[1][2 * r], p[1][2 * r + 1]);
    }
#pragma unroll
    for (int c = 0; c < kDV / 8; c += 2) {
      uint32_t bf[4];
      load_bt<kCV>(bf, vs, 0, c);
      mma16816<T>(acc[c], pf, bf[0], bf[1]);
      mma16816<T>(acc[c + 1], pf, bf[2], bf[3]);
    }
    __syncwarp();  // the stage is free for the copy of the next round
  }
  copy_wait<0>();
  __syncthreads();

  // join the warps: o, m and l of each row through shared memory (the ring is idle now)
  float* so = reinterpret_cast<float*>(smem);              // [WARPS][HB][kDV]
  float* sml = so + WARPS * HB * kDV;                      // [WARPS][HB][2]
  static_assert(WARPS * HB * (kDV + 2) * 4 <= RING, "the join fits the ring");
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = g + 8 * r;
    const float sum = quad_sum(l[r]);
    if ((lane & 3) == 0) {
      sml[(w * HB + row) * 2] = m[r];
      sml[(w * HB + row) * 2 + 1] = sum;
    }
#pragma unroll
    for (int c = 0; c < kDV / 8; ++c)
      *reinterpret_cast<float2*>(so + (w * HB + row) * kDV + c * 8 + t2) =
          make_float2(acc[c][2 * r], acc[c][2 * r + 1]);
  }
  __syncthreads();
  const long long head = (long long)n * a.H + kv * G + h0;
  for (int x = tid; x < heads * (kDV / 2); x += THREADS) {
    const int row = x / (kDV / 2), c = x % (kDV / 2) * 2;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) top = fmaxf(top, sml[(k * HB + row) * 2]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float f = ex2((sml[(k * HB + row) * 2] - base) * kLog2e);
      const float2 o = *reinterpret_cast<const float2*>(so + (k * HB + row) * kDV + c);
      sum = fmaf(f, sml[(k * HB + row) * 2 + 1], sum);
      o0 = fmaf(f, o.x, o0);
      o1 = fmaf(f, o.y, o1);
    }
    if (parts == 1) {
      const float inv = 1.f / sum;  // the new token is always there: sum > 0
      store2(static_cast<TO*>(a.o) + (head + row) * kDV + c, o0 * inv, o1 * inv);
    } else {
      float* pw = static_cast<float*>(a.workspace) +
                  ((long long)(unit - plan.whole) * HB + row) * parts * (kDV + 2) + part * (kDV + 2);
      *reinterpret_cast<float2*>(pw + c) = make_float2(o0, o1);
      if (c == 0) *reinterpret_cast<float2*>(pw + kDV) = make_float2(top, sum);
    }
  }
}

// Joins the parts of one head of a cut unit: o = sum_p exp(m_p - m) o_p / sum_p exp(m_p - m) l_p, in order.
template <class TO>
__global__ void __launch_bounds__(kDV / 2)
window_join_kernel(WindowDecodeArgs a, DecodePlan plan, int groups, int rows) {
  griddep_wait();
  const int cut = blockIdx.x / rows, row = blockIdx.x % rows, unit = plan.whole + cut;
  const int grp = unit % groups, nk = unit / groups, KV = a.c.KV, G = a.H / KV;
  const int n = nk / KV, c = threadIdx.x * 2, h = grp * HB + row, parts = plan.parts;
  if (h >= G) return;
  const int p = __ldg(a.c.page + n);
  if (p < 0 || p >= a.c.n_pages || __ldg(a.pos + n) < 0) return;  // recorded; o is left as it was
  const float* pw =
      static_cast<const float*>(a.workspace) + ((long long)cut * HB + row) * parts * (kDV + 2);
  float top = -INFINITY;
  for (int k = 0; k < parts; ++k) top = fmaxf(top, pw[k * (kDV + 2) + kDV]);
  float sum = 0.f, o0 = 0.f, o1 = 0.f;
  for (int k = 0; k < parts; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(pw + k * (kDV + 2) + kDV);
    const float2 x = *reinterpret_cast<const float2*>(pw + k * (kDV + 2) + c);
    const float f = ml.x == -INFINITY ? 0.f : ex2((ml.x - top) * kLog2e);
    sum = fmaf(f, ml.y, sum);
    o0 = fmaf(f, x.x, o0);
    o1 = fmaf(f, x.y, o1);
  }
  const float inv = 1.f / sum;
  store2(static_cast<TO*>(a.o) + ((long long)n * a.H + nk % KV * G + h) * kDV + c, o0 * inv, o1 * inv);
}

// One warp per (sequence, slot): the latest of the prompt's tokens that belongs there.
__global__ void __launch_bounds__(256)
window_fill_kernel(WindowCache c, const uint4* __restrict__ k, const uint4* __restrict__ v,
                   const int* __restrict__ lens, int T, DevCtl ctl) {
  const int slots = c.window + c.sink, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)c.n * slots) return;
  const int n = (int)(row / slots), s = (int)(row % slots);
  const int page = __ldg(c.page + n);
  if (page < 0 || page >= c.n_pages) {
    if (lane == 0) record_error(ctl, DEV_RANGE);
    return;
  }
  int len = T;
  if (lens) {
    len = __ldg(lens + n);
    if (len < 0 || len > T) {
      if (lane == 0) record_error(ctl, DEV_RANGE);
      len = len < 0 ? 0 : T;
    }
  }
  if (s >= len) return;  // slot s is first filled by token s
  const int t = s < c.sink ? s : s + (len - 1 - s) / c.window * c.window;
  const long long src = ((long long)n * T + t) * c.KV;
  const long long dst = (((long long)page * c.pool_layers + c.layer) * slots + s) * c.KV;
  uint4* pk = static_cast<uint4*>(c.k) + dst * kCK;
  uint4* pv = static_cast<uint4*>(c.v) + dst * kCV;
  for (int x = lane; x < c.KV * kCK; x += 32) pk[x] = __ldg(k + src * kCK + x);
  for (int x = lane; x < c.KV * kCV; x += 32) pv[x] = __ldg(v + src * kCV + x);
}

int groups_of(int KV, int H) { return (H / KV + HB - 1) / HB; }

// Parts of at least one round of the warps' tiles (64 slots) each; nothing is cut where two do not
// fit into the last round.
DecodePlan make_plan(int n, int KV, int H, int slots, int n_sm) {
  const long long units = (long long)n * KV * groups_of(KV, H);
  const int hold = std::max(2 * n_sm, 1), unit = SB * WARPS, rest = (int)(units % hold);
  const int most = std::min((slots + unit - 1) / unit, 64);
  const int parts = rest ? std::min(hold / rest, most) : 1;
  if (parts < 2) return DecodePlan{(int)units, 0, 1, 0};
  const int part_slots = ((slots + parts - 1) / parts + unit - 1) / unit * unit;
  return DecodePlan{(int)(units - rest), rest, parts, part_slots};
}

template <class T, class TO>
cudaError_t run(const WindowDecodeArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const int slots = a.c.window + a.c.sink, KV = a.c.KV;
  const DecodePlan plan = make_plan(a.c.n, KV, a.H, slots, n_sm);
  const int groups = groups_of(KV, a.H), rows = std::min(HB, a.H / KV);
  auto kern = window_decode_kernel<T, TO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(plan.whole + plan.cut * plan.parts), THREADS, SMEM, stream>>>(a, plan, groups,
                                                                                 ctl);
  if ((e = cudaGetLastError()) != cudaSuccess || !plan.cut) return e;
  PdlLaunch l(dim3((unsigned)(plan.cut * rows)), dim3(kDV / 2), 0, stream, true);
  return cudaLaunchKernelEx(&l.cfg, window_join_kernel<TO>, a, plan, groups, rows);
}

}  // namespace

size_t window_decode_workspace_bytes(int n, int KV, int H, int slots, int n_sm) {
  const DecodePlan p = make_plan(n, KV, H, slots, n_sm);
  return (size_t)p.cut * HB * p.parts * (kDV + 2) * sizeof(float);
}

cudaError_t launch_window_decode(const WindowDecodeArgs& a, int n_sm, DevCtl ctl,
                                 cudaStream_t stream) {
  const bool wide = a.out_type == GLA_FP32;
  if (a.c.type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, n_sm, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, n_sm, ctl, stream);
  return wide ? run<__half, float>(a, n_sm, ctl, stream) : run<__half, __half>(a, n_sm, ctl, stream);
}

cudaError_t launch_window_fill(const WindowCache& c, const void* k, const void* v, const int* lens,
                               int T, DevCtl ctl, cudaStream_t stream) {
  const long long rows = (long long)c.n * (c.window + c.sink);
  window_fill_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(
      c, static_cast<const uint4*>(k), static_cast<const uint4*>(v), lens, T, ctl);
  return cudaGetLastError();
}

}  // namespace gla
