// window_bwd.cu -- gradient of the windowed attention (window_fwd.cu) for the scalar loss
// sum(o . dO): with p_ts = exp(q_t . k_s - lse_t) over the visible pairs and
// delta_t = dO_t . o_t,
//   dz_ts = p_ts (dO_t . v_s - delta_t)
//   dq_t = sum_s dz_ts k_s,   dk_s = sum_t dz_ts q_t,   dv_s = sum_t p_ts dO_t
// where dk and dv also sum over the query heads that share the key head.
//
// window_delta_kernel takes delta (bound by HBM); window_bwd_kernel does the rest on tcgen05, in
// three kinds, each with a tile of 128 rows held and tiles of 64 rows streamed by:
//   VALUES   keys held (k), the queries that see them streamed (q, dO), head after head:
//              S = K Q^T, dv += P dO
//   KEYS     the same with k, v held:  S = K Q^T, D = V dO^T, dk += Z Q
//   QUERIES  queries held (q, dO), the keys they see streamed (k, v):
//              S = Q K^T, D = dO V^T, dq += Z K
// with P and Z (dz) written back to tensor memory in 16 bits as the left operand.  All three
// recompute the scores: eight products where five would do, but no sum crosses a CTA, so there are
// no atomics on results and they repeat bit for bit; and apart the kinds have the tensor memory
// for two tiles of scores each and for all held operands (Z takes the place of its S, which the
// next scores there, issued behind the sum that reads Z, may overwrite): an operand of 128 x 16 from
// shared memory next to one of 64 x 16 takes 1.5 times as long to read as the product takes, and
// the held tile's shared memory is free for the next item's as soon as it has been copied.  The
// grids are programmatic dependents of one another: KEYS waits for delta, the others for nothing, so
// that a CTA of the next kind starts where one of the last has no item left.  They may read delta and
// the counters all the same: a CTA of KEYS lets its dependent start only behind its own wait, that is
// when delta's grid is complete and its writes are in memory, VALUES starts when all of them have, and
// QUERIES when all of VALUES has started; and no cache holds older values, as nothing reads either
// between the start of delta's grid and its end.  That rests on KEYS being launched first.
//   warp 8       takes items from a counter and issues the TMA loads: the held tile, and a ring of
//                four streamed tiles
//   warp 9       lse and delta of the streamed queries, into shared memory (VALUES, KEYS)
//   warp 10      tcgen05 issuer and TMEM owner; the scores run two tiles ahead of the sums
//   warps 0..7   two groups that take an item's tiles in turn (thread = row): mask, P, Z
//   warps 11..14 the held operands of the next item into tensor memory, then the output rows of
//                this one, while the others are on the next
// Keys that hold sinks are seen by every query behind them.  Those far queries are items of their
// own, at least as long as an ordinary one and at most 16 of a key tile, whose sums go to the
// workspace as fp32 and are added in order by window_sink_kernel.  Past four tiles of sinks the
// items of a tile are many enough as they are, and one item takes all queries of its keys.
//
// Bound by the hand-over of a tile from its scores to P or Z and on to the sums, and by the issue of
// 22 (VALUES: 10) products per 64 streamed rows: ~1,300 cycles a tile where the products take 770.
// Measured, bf16, B=8 T=2048, 16 heads on 4, window 512, 4 sinks: 340 us, with 10,600 of the 16,384
// tokens live 237, 9,097 208, 6,609 169 (delta 21, the sinks' sums 4).  As the mean of the last two,
// 192 now (waits whose limit follows the CTA's steps cost 2 of them), before: 277 with the three kinds
// in one grid and every operand from shared memory; 207 with half of the held operands in tensor
// memory, copied by the warps of P and Z; 202 with all of them; 196 with delta and the sinks' sums
// chained to the kinds; 191 with an issuer that keeps its descriptors.  No faster: masks by the tile's
// position in place of votes (+2 us), an issuer that takes the next item's scores ahead of this item's
// last sums (+4 us).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tmap.h"
#include "window_common.cuh"
#include "window_wait.cuh"

namespace gla {
namespace {

using scan::Cta;
using scan::DRAIN_NS;

constexpr int BH = 128, BS = 64, STAGES = 4;  // rows held, rows streamed
constexpr int kSums = kDK + kDV;              // dk and dv of a key
constexpr uint32_t HX_BOX = 8192, HY_BOX = 16384, SX_BOX = 4096, SY_BOX = 8192;
constexpr uint32_t H_BYTES = 3 * (HX_BOX + HY_BOX), S_BYTES = 3 * (SX_BOX + SY_BOX);
constexpr uint32_t OFF_HX = 0, OFF_HY = 3 * HX_BOX, OFF_S = H_BYTES;
constexpr uint32_t OFF_STAT = OFF_S + STAGES * S_BYTES;  // float [STAGES][2][64]: lse, delta
constexpr uint32_t OFF_STG = OFF_STAT + STAGES * 512;  // output staging, 2 KB per output warp
constexpr uint32_t OFF_BAR = OFF_STG + 4 * 2048;
enum Bar : uint32_t {
  FULL = 0,        // +stage
  EMPTY = 4,       // +stage: the tile has been added
  STAT_FULL = 8,   // +stage
  STAT_EMPTY = 12, // +stage
  HELD_FULL = 16,
  HELD_EMPTY = 17, // the item's scores are complete: the held operands may be replaced
  HELD_READY = 18, // the held operands are in tensor memory (and no more read from shared memory)
  ITEM_FULL = 19,  // +slot
  ITEM_EMPTY = 21, // +slot
  S_FULL = 23,     // +group: its S and D are in tensor memory
  P_READY = 25,    // +group: ... and have been read, and P or Z written
  SUM_DONE = 27,   // an item's sums are complete
  SUM_FREE = 28,   // ... and have been read
  DRAIN = 29,
  NBAR = 30
};
constexpr uint32_t OFF_ITEM = OFF_BAR + NBAR * 8;  // int4 item[2][2]
static_assert(OFF_ITEM % 16 == 0, "items are read by 16 bytes");
constexpr uint32_t OFF_TMEM = OFF_ITEM + 64, OFF_ABORT = OFF_TMEM + 4;
// The opt-in maximum; the kernel aligns its base to 1024 bytes and does not run (GLA_ERR_LAYOUT)
// if the padding that takes would not fit.  Dynamic shared memory normally starts aligned.
constexpr uint32_t SMEM_USED = OFF_ABORT + 4 * kWaitWords, SMEM_BYTES = 232448;
static_assert(SMEM_USED <= SMEM_BYTES, "shared memory budget");
enum Kind : int { VALUES = 0, KEYS = 1, QUERIES = 2 };
// Tensor memory columns.  VALUES: dv 192, S twice 64, P twice 32, k 48.  The others: S and D twice
// 64 (Z takes the place of its S, from the front), dk or dq 96, v or dO 96, k or q 48.
template <int KIND>
struct Tm {
  static constexpr bool V = KIND == VALUES;
  static constexpr uint32_t SUM = V ? 0 : 256, HX = V ? 384 : 448, HY = 352;
  __device__ static uint32_t s(int g) { return V ? 192 + 64 * g : 128 * g; }
  __device__ static uint32_t d(int g) { return 64 + 128 * g; }
  __device__ static uint32_t p(int g) { return V ? 320 + 32 * g : s(g); }
};

constexpr int EW = 8, LOAD_WARP = 8, STAT_WARP = 9, MMA_WARP = 10, OUT_WARP = 11, GROUP = 128;
constexpr int THREADS = 15 * 32;

// How the work is cut into items, the same for every part of the call.
struct BwdPlan {
  int tiles;       // of 128 rows, of a sequence
  int steps;       // streamed query tiles of an ordinary item of held keys, per head
  int far_steps;   // ... of a far one
  int sink_tiles;  // key tiles that hold sinks and have far queries
  int far_parts;   // most far items of one of them
  long long keys, far, queries;  // items: ordinary and far ones of held keys, of held queries
  __host__ __device__ int total(int kind) const { return (int)(kind == QUERIES ? queries : keys + far); }
  // First streamed tile past the window's of key tile j.
  __host__ __device__ int far_begin(int j) const { return j * (BH / BS) + steps; }
  // Far items of key tile j of a sequence of `len` tokens.
  __host__ __device__ int far_of(int j, int len) const {
    const int n = (len + BS - 1) / BS - far_begin(j);
    return n > 0 ? (n + far_steps - 1) / far_steps : 0;
  }
};
BwdPlan make_plan(int B, int T, int H, int KV, int window, int sink) {
  BwdPlan p;
  p.tiles = (T + BH - 1) / BH;
  p.steps = (int)(((long long)BH - 1 + window + BS - 1) / BS);
  p.far_steps = std::max(p.steps, ((T + BS - 1) / BS + 15) / 16);
  p.sink_tiles = 0;
  p.far_parts = p.far_of(0, T);
  while (sink <= 4 * BH && p.sink_tiles * BH < sink && p.sink_tiles < p.tiles && p.far_of(p.sink_tiles, T) > 0)
    ++p.sink_tiles;
  if (!p.sink_tiles) p.far_parts = 0;
  p.keys = (long long)B * KV * p.tiles;
  p.far = (long long)B * KV * p.sink_tiles * p.far_parts;
  p.queries = (long long)B * H * p.tiles;
  return p;
}
// fp32 sums of sink rows: [B][KV][sink rows][1 + far_parts][kSums].
__host__ __device__ inline int sink_rows(const BwdPlan& p, int sink) {
  return p.sink_tiles * BH < sink ? p.sink_tiles * BH : sink;
}

// ---- delta[b,h,t] = dO . o, eight lanes per (token, head); 0 past a sequence's end
template <class T, class TO>
__global__ void __launch_bounds__(256)
window_delta_kernel(WindowArgs a, float* __restrict__ delta, int* __restrict__ counter, DevCtl ctl) {
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < 3) counter[threadIdx.x] = 0;  // one a kind
  const long long rows = (long long)a.B * a.T * a.H;
  const long long row = (long long)blockIdx.x * 32 + (threadIdx.x >> 3);  // (b T + t) H + h
  const int l = threadIdx.x & 7;
  float s = 0.f;
  int h = 0, b = 0, t = 0;
  if (row < rows) {
    h = (int)(row % a.H);
    const long long bt = row / a.H;
    b = (int)(bt / a.T);
    t = (int)(bt - (long long)b * a.T);
    int len = a.T;
    if (a.lens) {
      len = __ldg(a.lens + b);
      if ((len < 0 || len > a.T) && t == 0 && h == 0) record_error(ctl, DEV_RANGE);
    }
    if (t < len) {
      const T* g = static_cast<const T*>(a.dO) + row * kDV;
      const TO* o = static_cast<const TO*>(a.o) + b * a.o_stride[0] + t * a.o_stride[1] +
                    h * a.o_stride[2];
      Pack<T, 8> x[3];
      Pack<TO, 8> y[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        x[i].template load<false>(g + (i * 8 + l) * 8);  // read again by the kernel behind
        y[i].load(o + (i * 8 + l) * 8);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(x[i].get(j), y[i].get(j), s);
    }
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (row < rows && l == 0) delta[((long long)b * a.H + h) * a.T + t] = s;
}

// One item, as every role of a CTA sees it.
template <int KIND>
struct Item {
  static constexpr bool HELD_KEYS = KIND != QUERIES;
  int b, head, row0;      // sequence, key or (QUERIES) query head, first held row
  int len;                // tokens of the sequence
  int part;               // far part, or -1
  int first, per_head;    // held keys: first streamed tile and tiles per head
  int n;                  // streamed tiles in all
  KeyTiles kt;            // QUERIES: the key tiles
  __device__ Item() : b(0), head(0), row0(0), len(0), part(-1), first(0), per_head(0), n(0), kt(0, 1, BS, 1, 0) {}
  __device__ void set(int i, const WindowArgs& a, const BwdPlan& p) {
    unsigned r = i;
    auto take = [&](unsigned m) {  // r mod m, then r / m
      const unsigned q = r / m, x = r - q * m;
      r = q;
      return (int)x;
    };
    part = -1;
    const bool far = HELD_KEYS && i >= (int)p.keys;
    if (far) r -= (unsigned)p.keys;
    head = take(HELD_KEYS ? a.KV : a.H);
    if (far) part = take(p.far_parts);
    row0 = take(far ? p.sink_tiles : p.tiles) * BH;
    b = (int)r;
    len = a.T;
    if (a.lens) len = min(max(__ldg(a.lens + b), 0), a.T);
    n = 0;
    if (row0 >= len) return;
    if (HELD_KEYS) {
      const int all = (len + BS - 1) / BS;  // streamed tiles of the sequence
      first = row0 / BS;
      int last = row0 < a.sink && row0 / BH >= p.sink_tiles ? all : first + p.steps;
      if (far) {
        first = p.far_begin(row0 / BH) + part * p.far_steps;
        last = first + p.far_steps;
      }
      per_head = max(0, min(last, all) - first);
      n = per_head * (a.H / a.KV);
    } else {
      kt = KeyTiles(row0, min(row0 + BH, len), BS, a.window, a.sink);
      n = kt.n;
    }
  }
  // Through shared memory, so that only the warp that takes the item divides.
  __device__ void put(int4* p) const {
    p[0] = make_int4(b, head, row0, len);
    p[1] = make_int4(part, HELD_KEYS ? first : kt.lo, HELD_KEYS ? per_head : kt.far, n);
  }
  __device__ bool get(const int4* p) {
    const int4 x = p[0], y = p[1];
    b = x.x; head = x.y; row0 = x.z; len = x.w;
    part = y.x; n = y.w;
    if (HELD_KEYS) { first = y.y; per_head = y.z; }
    else { kt.lo = y.y; kt.far = y.z; kt.n = y.w; }
    return b >= 0;
  }
  // columns of streamed tile i that count: fewer in the sinks' tiles in front of the window
  __device__ int cols(int i, int sink) const {
    return !HELD_KEYS && i < kt.far ? min(BS, (sink - kt.tile(i) * BS + 15) & ~15) : BS;
  }
};

// The streamed tiles of an item in order: first row, and the head they are of.
template <int KIND>
struct Walk {
  const Item<KIND>& it;
  int i = 0, x = 0, head;  // tile, tile within the head (held keys), head
  __device__ Walk(const Item<KIND>& it_, int G)
      : it(it_), head(KIND != QUERIES ? it_.head * G : it_.head / G) {}
  __device__ int row() const { return (KIND != QUERIES ? it.first + x : it.kt.tile(i)) * BS; }
  __device__ void next() {
    ++i;
    if (KIND != QUERIES && ++x == it.per_head) {
      x = 0;
      ++head;
    }
  }
};

template <class T, class TO, int KIND>
__global__ void __launch_bounds__(THREADS, 1)
window_bwd_kernel(const __grid_constant__ CUtensorMap held_x,
                  const __grid_constant__ CUtensorMap held_y,
                  const __grid_constant__ CUtensorMap str_x,
                  const __grid_constant__ CUtensorMap str_y, WindowArgs a, BwdPlan plan,
                  const float* __restrict__ delta, int* __restrict__ counter,
                  float* __restrict__ sink_sums, DevCtl ctl) {
  constexpr bool BF16 = !__is_same(T, __half), STATS = KIND != QUERIES;
  using M = Tm<KIND>;
  if (KIND != KEYS) griddep_launch_dependents();  // the next kind needs SMs, nothing of this one
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Cta cta;
  cta.base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  if ((uint32_t)(cta.base - smem_raw) + SMEM_USED > SMEM_BYTES) {
    if (threadIdx.x == 0) record_error(ctl, DEV_LAYOUT);
    griddep_wait();
    return;
  }
  cta.sb = smem_u32(cta.base);
  cta.bar_off = OFF_BAR;
  cta.abort_off = OFF_ABORT;
  uint8_t* const base = cta.base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* tmem_slot = (uint32_t*)(base + OFF_TMEM);
  int4* const items = (int4*)(base + OFF_ITEM);
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (tid == LOAD_WARP * 32) {
    for (uint32_t s = 0; s < STAGES; ++s) {
      mbar_init(cta.bar(FULL + s), 1);
      mbar_init(cta.bar(EMPTY + s), 1);
      mbar_init(cta.bar(STAT_FULL + s), 32);
      mbar_init(cta.bar(STAT_EMPTY + s), GROUP);
    }
    mbar_init(cta.bar(HELD_FULL), 1);
    mbar_init(cta.bar(HELD_EMPTY), 1);
    mbar_init(cta.bar(HELD_READY), 128);
    for (uint32_t s = 0; s < 2; ++s) {
      mbar_init(cta.bar(ITEM_FULL + s), 1);
      mbar_init(cta.bar(ITEM_EMPTY + s), EW + 4 + (STATS ? 2 : 1));
      mbar_init(cta.bar(S_FULL + s), 1);
      mbar_init(cta.bar(P_READY + s), GROUP);
    }
    mbar_init(cta.bar(SUM_DONE), 1);
    mbar_init(cta.bar(SUM_FREE), 128);
    mbar_init(cta.bar(DRAIN), 1);
    for (uint32_t i = 0; i < kWaitWords; ++i) cta.abort_flag()[i] = 0;
    fence_barrier_init();
  }
  if (KIND == KEYS) {  // the first kind: delta and the counters, for itself and the others
    griddep_wait();
    griddep_launch_dependents();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = a.H / a.KV;

  // The next item as a consumer sees it (slot m & 1): false at the end or after a give-up.  Called
  // by whole warps, or by the single MMA thread.
  auto next_item = [&](Item<KIND>& it, int m, bool whole_warp) -> bool {
    const uint32_t s = m & 1;
    if (whole_warp ? !await_warp(cta, cta.bar(ITEM_FULL + s), (m >> 1) & 1, ctl)
                   : !await(cta, cta.bar(ITEM_FULL + s), (m >> 1) & 1, ctl))
      return false;
    const bool some = it.get(items + 2 * s);
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(cta.bar(ITEM_EMPTY + s));
    return some;
  };

  if (warp == LOAD_WARP) {
    // ------------------------------------------------------------ items and TMA loads
    if (lane == 0) {
      Item<KIND> it;
      int n = 0, held = 0;
      bool ok = true;
      int ticket = atomicAdd(counter + KIND, 1);
      for (int m = 0; ok; ++m) {
        const uint32_t slot = m & 1;
        if (m >= 2 && !await(cta, cta.bar(ITEM_EMPTY + slot), ((m >> 1) - 1) & 1, ctl)) break;
        const bool end = ticket >= plan.total(KIND);
        if (end) it.b = -1;
        else it.set(ticket, a, plan);
        it.put(items + 2 * slot);
        mbar_arrive(cta.bar(ITEM_FULL + slot));
        if (end) break;
        ticket = atomicAdd(counter + KIND, 1);
        if (it.n == 0) continue;
        if (held > 0 && !await(cta, cta.bar(HELD_READY), (held - 1) & 1, ctl)) break;
        ++held;
        mbar_arrive_expect_tx(cta.bar(HELD_FULL), KIND == VALUES ? 3 * HX_BOX : H_BYTES);
        for (int j = 0; j < 3; ++j) {
          tma_load_4d(cta.sb + OFF_HX + j * HX_BOX, &held_x, cta.bar(HELD_FULL), 32 * j, it.head,
                      it.row0, it.b);
          if (KIND != VALUES)
            tma_load_4d(cta.sb + OFF_HY + j * HY_BOX, &held_y, cta.bar(HELD_FULL), 64 * j, it.head,
                        it.row0, it.b);
        }
        for (Walk<KIND> k(it, G); k.i < it.n; k.next(), ++n) {
          const uint32_t s = n % STAGES, st = cta.sb + OFF_S + s * S_BYTES;
          if (n >= STAGES && !(ok = await(cta, cta.bar(EMPTY + s), (n / STAGES - 1) & 1, ctl)))
            break;
          const int r = k.row();
          mbar_arrive_expect_tx(cta.bar(FULL + s), S_BYTES);
          for (int j = 0; j < 3; ++j) {
            tma_load_4d(st + j * SX_BOX, &str_x, cta.bar(FULL + s), 32 * j, k.head, r, it.b);
            tma_load_4d(st + 3 * SX_BOX + j * SY_BOX, &str_y, cta.bar(FULL + s), 64 * j, k.head, r,
                        it.b);
          }
        }
      }
      // every armed load has landed before the CTA may exit
      for (int s = 0; s < STAGES; ++s)
        if (n > s) mbar_wait(cta.bar(FULL + s), ((n - 1 - s) / STAGES) & 1, ctl, DRAIN_NS);
      if (held) mbar_wait(cta.bar(HELD_FULL), (held - 1) & 1, ctl, DRAIN_NS);
    }
  } else if (warp == STAT_WARP) {
    // ------------------------------------------------------------ lse and delta of the queries
    if constexpr (STATS) {
      Item<KIND> it;
      bool ok = true;
      for (int m = 0, n = 0; ok && next_item(it, m, true); ++m) {
        for (Walk<KIND> k(it, G); k.i < it.n; k.next(), ++n) {
          const uint32_t s = n % STAGES;
          const int t0 = k.row();
          const long long at = ((long long)it.b * a.H + k.head) * a.T + t0;
          float x[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = lane + 32 * j;
            x[j] = t0 + c < it.len ? -__ldg(a.lse + at + c) * kLog2e : 0.f;
            x[2 + j] = t0 + c < it.len ? -__ldg(delta + at + c) : 0.f;
          }
          if (n >= STAGES && !(ok = await_warp(cta, cta.bar(STAT_EMPTY + s), (n / STAGES - 1) & 1,
                                              ctl)))
            break;
          float* st = (float*)(base + OFF_STAT + s * 512);
#pragma unroll
          for (int j = 0; j < 4; ++j) st[lane + 32 * j] = x[j];
          mbar_arrive(cta.bar(STAT_FULL + s));
        }
      }
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t ID_S = idesc_f16(128, 0, BF16, BF16, false, false);
      constexpr uint32_t ID_SUM = idesc_f16(128, KIND == VALUES ? kDV : kDK, BF16, BF16, false, true);
      Item<KIND> it;
      int n = 0, held = 0;       // streamed tiles and items with work so far
      uint32_t phase = 0;        // bit g: parity of the group's tiles so far
      bool ok = true;
      // stage 0's descriptors (they count in 16 bytes): for the scores, and for the sums
      const uint64_t sx0 = smem_desc(cta.sb + OFF_S, 16, 512, SW_64);
      const uint64_t sy0 = smem_desc(cta.sb + OFF_S + 3 * SX_BOX, 16, 1024, SW_128);
      const uint64_t sum0 = KIND == VALUES
                                ? smem_desc(cta.sb + OFF_S + 3 * SX_BOX, SY_BOX, 1024, SW_128)
                                : smem_desc(cta.sb + OFF_S, SX_BOX, 512, SW_64);
      auto scores = [&](int i, int at) -> bool {  // S, D of the item's tile i, tile `at` in all
        const uint32_t s = at % STAGES;
        const int g = i & 1;
        if (!await(cta, cta.bar(FULL + s), (at / STAGES) & 1, ctl)) return false;
        tc_fence_after();
        const uint32_t id = ID_S | ((uint32_t)((KIND == QUERIES ? it.cols(i, a.sink) : BS) >> 3) << 17);
        const uint64_t sx = sx0 + s * (S_BYTES >> 4), sy = sy0 + s * (S_BYTES >> 4);
#pragma unroll
        for (int c = 0; c < 6; ++c)
          mma_f16_ts(tmem + M::s(g), tmem + M::HX + 8 * c,
                     sx + (((c >> 1) * SX_BOX + (c & 1) * 32) >> 4), id, c > 0);
        if constexpr (KIND != VALUES) {
#pragma unroll
          for (int c = 0; c < 12; ++c)
            mma_f16_ts(tmem + M::d(g), tmem + M::HY + 8 * c,
                       sy + (((c >> 2) * SY_BOX + (c & 3) * 32) >> 4), id, c > 0);
        }
        mma_commit(cta.bar(S_FULL + g));
        if (i == it.n - 1) mma_commit(cta.bar(HELD_EMPTY));
        return true;
      };
      for (int m = 0; ok && next_item(it, m, false); ++m) {
        if (it.n == 0) continue;
        ++held;
        if (!(ok = await(cta, cta.bar(HELD_READY), (held - 1) & 1, ctl))) break;
        if (!(ok = scores(0, n))) break;
        if (it.n > 1 && !(ok = scores(1, n + 1))) break;
        for (int i = 0; i < it.n; ++i, ++n) {
          const uint32_t s = n % STAGES;
          const int g = i & 1;
          if (n == ctl.stall_step) {  // the give-up path's diagnostic (see chunk_fwd.cu)
            await(cta, cta.bar(DRAIN), 0, ctl);
            ok = false;
            break;
          }
          if (i == 0 && held > 1 && !(ok = await(cta, cta.bar(SUM_FREE), (held - 2) & 1, ctl)))
            break;
          if (!(ok = await(cta, cta.bar(P_READY + g), (phase >> g) & 1, ctl))) break;
          phase ^= 1u << g;
          tc_fence_after();
          const uint64_t sum = sum0 + s * (S_BYTES >> 4);
          if constexpr (KIND == VALUES) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mma_f16_ts(tmem + M::SUM, tmem + M::p(g) + 8 * c, sum + (c * 2048 >> 4), ID_SUM,
                         i > 0 || c > 0);
          } else {
            const int steps = KIND == QUERIES ? it.cols(i, a.sink) >> 4 : 4;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c < steps)
                mma_f16_ts(tmem + M::SUM, tmem + M::p(g) + 8 * c, sum + (c * 1024 >> 4), ID_SUM,
                           i > 0 || c > 0);
          }
          mma_commit(cta.bar(EMPTY + s));
          made_step(cta, STEP_TILE, n + 1);
          if (i == it.n - 1) mma_commit(cta.bar(SUM_DONE));
          // the group has read its scores, and the commit behind the new ones also says that the
          // sum above is done: P or Z may be written again
          if (i + 2 < it.n && !(ok = scores(i + 2, n + 2))) break;
        }
      }
      mma_commit(cta.bar(DRAIN));
      mbar_wait(cta.bar(DRAIN), 0, ctl, DRAIN_NS);
    }
  } else if (warp < EW) {
    // ------------------------------------------------------------ P and Z
    const int q4 = warp & 3, g = warp >> 2, row = 32 * q4 + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    Item<KIND> it;
    int n0 = 0;            // streamed tiles before this item
    uint32_t used = 0;     // tiles of this group so far
    bool ok = true;
    for (int m = 0; ok && next_item(it, m, true); ++m) {
      if (it.n == 0) continue;
      const int r = it.row0 + row, len = it.len;  // this thread's key or query
      float lse = 0.f, del = 0.f;                 // negated, lse in base 2
      if (!STATS && r < len) {
        const long long at = ((long long)it.b * a.H + it.head) * a.T + r;
        lse = -__ldg(a.lse + at) * kLog2e;
        del = -__ldg(delta + at);
      }
      Walk<KIND> k(it, G);
      if (g && it.n > 1) k.next();
      for (int i = g; i < it.n; i += 2) {
        const int n = n0 + i, x0 = k.row();
        // the 32 columns from c that the row sees, or is seen by
        auto sees = [&](int c) -> uint32_t {
          return STATS ? queries_seeing(r, x0 + c, len, a.window, a.sink)
                       : keys_seen(r, x0 + c, len, a.window, a.sink);
        };
        const bool whole = STATS ? it.row0 + BH - 1 <= x0 && x0 + BS <= len &&
                                       (x0 + BS - 1 - it.row0 < a.window || it.row0 + BH <= a.sink)
                                 : x0 + BS - 1 <= it.row0 && x0 + BS <= len &&
                                       (it.row0 + BH - 1 - x0 < a.window || x0 + BS <= a.sink);
        if (!(ok = await_warp(cta, cta.bar(S_FULL + g), used++ & 1, ctl))) break;
        // (behind the scores' wait: every earlier tile of the stage has been through here)
        if (STATS &&
            !(ok = await_warp(cta, cta.bar(STAT_FULL + n % STAGES), (n / STAGES) & 1, ctl)))
          break;
        tc_fence_after();
        const float* stat = (const float*)(base + OFF_STAT + (n % STAGES) * 512);
        const float2 l2e = make_float2(kLog2e, kLog2e);
        // 32 columns: P = exp2(S log2(e) - lse) or Z = P (D - delta) as pairs
        auto half = [&](int c, uint32_t see, bool masked) {
          uint32_t z[32], d[32], out[16];
          tmem_ld32(trow + M::s(g) + c, z);
          if constexpr (KIND != VALUES) tmem_ld32(trow + M::d(g) + c, d);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 l = make_float2(lse, lse), e = make_float2(del, del);
            if constexpr (STATS) {
              l = *reinterpret_cast<const float2*>(stat + c + 2 * j);
              if constexpr (KIND != VALUES)
                e = *reinterpret_cast<const float2*>(stat + 64 + c + 2 * j);
            }
            float2 p = fma2(make_float2(__uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1])),
                            l2e, l);
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            if constexpr (KIND != VALUES)
              p = mul2(p, add2(make_float2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1])),
                               e));
            if (masked) {  // selected, not multiplied: padding may hold anything
              p.x = (see >> (2 * j)) & 1 ? p.x : 0.f;
              p.y = (see >> (2 * j + 1)) & 1 ? p.y : 0.f;
            }
            out[j] = pack2<T>(p.x, p.y);
          }
          tmem_st16(trow + M::p(g) + c / 2, out);
        };
        if (whole) {
          half(0, 0u, false);
          half(32, 0u, false);
        } else {
#pragma unroll 1
          for (int c = 0; c < BS; c += 32) {
            const uint32_t see = sees(c);
            if (__any_sync(0xffffffffu, see != 0u)) {
              half(c, see, true);
            } else {
              const uint32_t none[16] = {};
              tmem_st16(trow + M::p(g) + c / 2, none);
            }
          }
        }
        if (STATS) mbar_arrive(cta.bar(STAT_EMPTY + n % STAGES));
        if (x0 + BS > len && len < a.T) {
          // rows of padding may hold anything, and 0 x NaN is NaN: zero them (the scores, which
          // also read them, are done)
          const int r0 = len - x0, cnt = (BS - r0) * 36;  // 12 + 24 chunks of 16 bytes a row
          uint8_t* const tile = base + OFF_S + (n % STAGES) * S_BYTES;
          for (int x = row; x < cnt; x += GROUP) {
            const int rr = r0 + x / 36, c = x % 36;
            uint8_t* p = c < 12 ? tile + (c >> 2) * SX_BOX + rr * 64 + (c & 3) * 16
                                : tile + 3 * SX_BOX + ((c - 12) >> 3) * SY_BOX + rr * 128 +
                                      ((c - 12) & 7) * 16;
            *(uint4*)p = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(cta.bar(P_READY + g));
        k.next();
        k.next();
      }
      n0 += it.n;
    }
  } else {
    // ------------------------------------------------------------ output rows
    const int q4 = warp & 3, row = 32 * q4 + lane;  // the quadrant that the warp may read
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    uint8_t* const stg = base + OFF_STG + q4 * 2048;
    constexpr int CB = 64 / (int)sizeof(TO);  // channels of 64 bytes
    constexpr int D = KIND == VALUES ? kDV : kDK;
    const int held_sinks = sink_rows(plan, a.sink), heads = STATS ? a.KV : a.H;
    TO* const dst = static_cast<TO*>(KIND == VALUES ? a.dv : KIND == KEYS ? a.dk : a.dq);
    // The held operands of an item into tensor memory, once the item before has no more scores to
    // take with them
    int held = 0;
    auto hold = [&]() -> bool {
      if (held > 0 && !await_warp(cta, cta.bar(HELD_EMPTY), (held - 1) & 1, ctl)) return false;
      if (!await_warp(cta, cta.bar(HELD_FULL), held & 1, ctl)) return false;
      ++held;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < (KIND == VALUES ? 12 : 36); c += 2) {  // 16-byte chunks of a row
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int ch = c < 12 ? c + e : c - 12 + e;
          const uint4 u = *(const uint4*)(
              c < 12 ? base + OFF_HX + (ch >> 2) * HX_BOX + swz_off(row, ch & 3, 64)
                     : base + OFF_HY + (ch >> 3) * HY_BOX + swz_off(row, ch & 7, 128));
          w[4 * e] = u.x; w[4 * e + 1] = u.y; w[4 * e + 2] = u.z; w[4 * e + 3] = u.w;
        }
        tmem_st8(trow + (c < 12 ? M::HX + 4 * c : M::HY + 4 * (c - 12)), w);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(cta.bar(HELD_READY));
      return true;
    };
    Item<KIND> it, ahead;
    int done = 0;  // items with work so far
    bool some = next_item(ahead, 0, true), ok = !some || ahead.n == 0 || hold();
    for (int m = 0; ok && some; ++m) {
      it = ahead;
      some = next_item(ahead, m + 1, true);
      if (some && ahead.n > 0 && !(ok = hold())) break;
      const int r = it.row0 + row;
      const bool live = r < it.len && it.n > 0;
      // rows whose sums are added up later, as fp32 (held keys); the others go out here
      const bool sums = STATS && r < held_sinks;
      float* const ss = sink_sums + ((((long long)it.b * a.KV + it.head) * held_sinks + (sums ? r : 0)) *
                                         (1 + plan.far_parts) + 1 + it.part) * kSums +
                        (KIND == VALUES ? 0 : kDV);
      const int from = STATS ? held_sinks : 0, to = it.part < 0 ? a.T : 0;
      if (it.n > 0) {
        if (!await_warp(cta, cta.bar(SUM_DONE), done & 1, ctl)) break;
        ++done;
        tc_fence_after();
      }
      TO* const p = dst + (((long long)it.b * a.T + it.row0 + 32 * q4) * heads + it.head) * D;
#pragma unroll 1
      for (int k = 0; k < D; k += CB) {
        uint32_t x[CB];
        if (it.n > 0) {
          if constexpr (CB == 16) tmem_ld16(trow + M::SUM + k, x);
          else tmem_ld32(trow + M::SUM + k, x);
          tmem_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) x[c] = live ? x[c] : 0u;
        if (sums)
#pragma unroll
          for (int c = 0; c < CB / 4; ++c)
            reinterpret_cast<uint4*>(ss + k)[c] =
                make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
        if (k + CB == D && it.n > 0) {
          tc_fence_before();
          mbar_arrive(cta.bar(SUM_FREE));
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 u;
          if constexpr (CB == 16) {
            u = make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          } else {
            u.x = pack2<TO>(__uint_as_float(x[8 * c]), __uint_as_float(x[8 * c + 1]));
            u.y = pack2<TO>(__uint_as_float(x[8 * c + 2]), __uint_as_float(x[8 * c + 3]));
            u.z = pack2<TO>(__uint_as_float(x[8 * c + 4]), __uint_as_float(x[8 * c + 5]));
            u.w = pack2<TO>(__uint_as_float(x[8 * c + 6]), __uint_as_float(x[8 * c + 7]));
          }
          *(uint4*)(stg + swz_off(lane, c, 64)) = u;
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // four lanes write the 64 bytes of a row
          const int o = 8 * c + (lane >> 2), t = it.row0 + 32 * q4 + o;
          const uint4 u = *(const uint4*)(stg + swz_off(o, lane & 3, 64));
          if (t >= from && t < to)
            reinterpret_cast<uint4*>(p + (long long)o * heads * D + k)[lane & 3] = u;
        }
      }
      if (tid == OUT_WARP * 32) made_step(cta, STEP_ITEM, m + 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // this grid is complete only after the one ahead of it: what follows on the stream waits for
  // both by waiting for this one
  griddep_wait();
}

// dk, dv of the sinks' keys: the window's sums and the far parts', in order.
template <class TO>
__global__ void __launch_bounds__(kSums / 2)
window_sink_kernel(WindowArgs a, BwdPlan plan, const float* __restrict__ sums) {
  griddep_wait();
  const int rows = sink_rows(plan, a.sink);
  const int s = blockIdx.x % rows;
  const long long bk = blockIdx.x / rows;
  const int b = (int)(bk / a.KV), kv = (int)(bk % a.KV), c = threadIdx.x * 2;
  int len = a.T;
  if (a.lens) len = min(max(__ldg(a.lens + b), 0), a.T);
  float x = 0.f, y = 0.f;
  if (s < len) {
    const float* p = sums + (bk * rows + s) * (1 + plan.far_parts) * kSums + c;
    const int parts = 1 + plan.far_of(s / BH, len);
    for (int k = 0; k < parts; ++k) {
      const float2 v = *reinterpret_cast<const float2*>(p + (long long)k * kSums);
      x += v.x;
      y += v.y;
    }
  }
  const long long row = ((long long)b * a.T + s) * a.KV + kv;
  if (c < kDV) store2(static_cast<TO*>(a.dv) + row * kDV + c, x, y);
  else store2(static_cast<TO*>(a.dk) + row * kDK + c - kDV, x, y);
}

// Workspace: the item counter, delta, the sinks' sums.
size_t delta_bytes(int B, int T, int H) { return ((size_t)B * T * H * 4 + 255) & ~(size_t)255; }
size_t sink_bytes(const BwdPlan& p, int B, int KV, int sink) {
  return p.sink_tiles ? (size_t)B * KV * sink_rows(p, sink) * (1 + p.far_parts) * kSums * 4 : 0;
}

template <class T, class TO>
cudaError_t run(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  constexpr bool bf16 = !__is_same(T, __half);
  const BwdPlan plan = make_plan(a.B, a.T, a.H, a.KV, a.window, a.sink);
  int* counter = static_cast<int*>(a.workspace);
  float* delta = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + 256);
  float* sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(delta) +
                                         delta_bytes(a.B, a.T, a.H));
  const long long rows = (long long)a.B * a.T * a.H;
  window_delta_kernel<T, TO><<<(unsigned)((rows + 31) / 32), 256, 0, stream>>>(a, delta, counter,
                                                                              ctl);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CUtensorMap hq, hk, hv, hg, sq, sk, sv, sg;
  auto x = [&](CUtensorMap* m, const void* p, int heads, int rows_) {
    return make_tmap_seq_16bit(m, p, kDK, heads, a.T, a.B, 32, rows_, CU_TENSOR_MAP_SWIZZLE_64B, bf16);
  };
  auto y = [&](CUtensorMap* m, const void* p, int heads, int rows_) {
    return make_tmap_seq_16bit(m, p, kDV, heads, a.T, a.B, 64, rows_, CU_TENSOR_MAP_SWIZZLE_128B, bf16);
  };
  if (!x(&hq, a.q, a.H, BH) || !x(&hk, a.k, a.KV, BH) || !y(&hv, a.v, a.KV, BH) ||
      !y(&hg, a.dO, a.H, BH) || !x(&sq, a.q, a.H, BS) || !x(&sk, a.k, a.KV, BS) ||
      !y(&sv, a.v, a.KV, BS) || !y(&sg, a.dO, a.H, BS))
    return cudaErrorInvalidValue;
  auto kind = [&](auto kern, int k, const CUtensorMap& hx, const CUtensorMap& hy,
                  const CUtensorMap& sx, const CUtensorMap& sy) -> cudaError_t {
    const cudaError_t f =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (f != cudaSuccess) return f;
    PdlLaunch l(dim3((unsigned)std::min(plan.total(k), n_sm)), dim3(THREADS), SMEM_BYTES, stream,
                true);
    return cudaLaunchKernelEx(&l.cfg, kern, hx, hy, sx, sy, a, plan, (const float*)delta, counter,
                              sums, ctl);
  };
  // the kind of the longest items first
  if ((e = kind(window_bwd_kernel<T, TO, KEYS>, KEYS, hk, hv, sq, sg)) != cudaSuccess ||
      (e = kind(window_bwd_kernel<T, TO, VALUES>, VALUES, hk, hv, sq, sg)) != cudaSuccess ||
      (e = kind(window_bwd_kernel<T, TO, QUERIES>, QUERIES, hq, hg, sk, sv)) != cudaSuccess)
    return e;
  if (!plan.sink_tiles) return cudaSuccess;
  PdlLaunch l(dim3((unsigned)((long long)a.B * a.KV * sink_rows(plan, a.sink))), dim3(kSums / 2), 0,
              stream, true);
  return cudaLaunchKernelEx(&l.cfg, window_sink_kernel<TO>, a, plan, (const float*)sums);
}

}  // namespace

size_t window_bwd_workspace_bytes(int B, int T, int H, int KV, int window, int sink) {
  return 256 + delta_bytes(B, T, H) +
         sink_bytes(make_plan(B, T, H, KV, window, sink), B, KV, sink);
}

cudaError_t launch_window_bwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const bool wide = a.out_type == GLA_FP32;
  if (a.in_type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, n_sm, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, n_sm, ctl, stream);
  return wide ? run<__half, float>(a, n_sm, ctl, stream) : run<__half, __half>(a, n_sm, ctl, stream);
}

}  // namespace gla
