// window_rows8.cuh -- the windowed attention of few new tokens per sequence over pages of 8 bits: one each
// (the decode step) or a handful (drafts).  8 NT rows, (token, query head) of one key head, are a unit; a
// CTA takes a unit, or a part of its page's slots, in rounds of 128: its four warps take 32 slots each from a
// ring that one thread's TMA fills, with running maxima and sums of their own, and join them at the end.
//
//   z = 2^e (c . q),  o = sum p 2^e c / sum p   with the rows' codes c as fp16 operands, exactly
//
// whatever the call's type: fp16 is a byte permute and a subtraction away from a code (0x6400 | u is 1024 +
// u), bf16 twice as much.  Queries of bf16 are scaled by a power of two per row into fp16's range; the
// values' 2^e goes into the weight, relative to the largest e of the tiles so far, so that a weight rounds
// by 2^-11 of itself or by 2^-25 of the weight of the page's largest row.  The new tokens' own keys and values are
// taken as given, in the call's type, a tile of 16 at a time straight from global memory.
//
// The codes are the products' first operand (16 slots by channels; 16 channels by slots), the rows their
// columns, eight at a time: most calls have four or eight rows, and a row takes 24 registers of sums a
// thread where as the first operand's it would take 48.  Keys are read eight channels at a time, in
// an order of the channels that the query's registers share; values by transposed loads of pairs of
// channels, which come apart in the permutes that make operands of them.  Weights go from the scores' layout
// to an operand's by matrix transposes between the lanes.
//
// Bound by the instructions: a code costs 1.25 of them, and the floor is HBM's 290 bytes a slot and key head.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "tmap.h"
#include "window_packed.cuh"

namespace gla {
namespace rows8 {

constexpr int WARPS = 4, THREADS = 32 * WARPS, SB = 32, STAGES = 2;
constexpr int ROUND = WARPS * SB;                        // slots of a stage, a tile of 32 for each warp
constexpr int V_BOX = ROUND * 64, OFF_KEYS = 3 * V_BOX;  // values in 3 boxes of 64 channels, keys
constexpr int STAGE = OFF_KEYS + ROUND * kDK;            // 36,864 bytes
constexpr int RING = STAGES * STAGE;
constexpr int JOIN_ROW = kDV + 4;                        // floats; the rows of a store in different banks
constexpr int OFF_BAR = RING;                            // mbarrier [stage], int [stage]: warps done with it
constexpr int OFF_FOUND = OFF_BAR + STAGES * 16;         // int [4]: the unit
constexpr int OFF_FACTORS = OFF_FOUND + 16;              // float2 [warp][32]: a tile's 2^e; before, sums
constexpr int EXPS = 2 * SB + 16;                        // a tile's exponents, from a word's start
constexpr int OFF_EXPS = OFF_FACTORS + WARPS * 32 * 8;   // [warp][stage]
constexpr int SMEM = OFF_EXPS + WARPS * STAGES * EXPS + 1024;
static_assert(3 * (SMEM + 1024) <= 228 * 1024, "three CTAs on an SM");
static_assert((THREADS + 1 + WARPS) * 4 <= WARPS * 32 * 8, "the sums fit where the factors go");
constexpr uint64_t DRAIN_NS = 4000000000ull;

struct Args {
  ServeCache cache;
  Packed tok;        // tok.start null: one token each, which goes into its page
  const void* q;
  const void* k;
  const void* v;
  void* o;
  int H;
  void* workspace;
};
// CTAs: a unit each for the first `whole` units, `parts` for each of the others.
struct Plan {
  long long units;   // at most
  int whole, parts, part_slots, rows;  // rows of a unit: 8 or 16
};
struct Maps {
  CUtensorMap k, v;
};

// What the join has to know: how many units there are, and of each cut one its rows.
struct CutUnit {
  int first, row0, rows, kv;  // the sequence's first packed row; its (token, head) rows from row0
};
__host__ __device__ inline size_t table_bytes(long long cut) {
  return ((cut + 1) * sizeof(CutUnit) + 255) / 256 * 256;
}
__host__ __device__ inline size_t workspace_bytes(const Plan& p) {
  const long long cut = p.units - p.whole;
  return p.parts > 1 && cut > 0
             ? table_bytes(cut) + (size_t)cut * p.rows * p.parts * (kDV + 2) * sizeof(float)
             : 0;
}

// Bits of a tile's 32 slots from c0 that the token at position p of a sequence sees; pos tokens are there.
struct Seen {
  int ns, a_hi, base, slots, sink;  // as in window_chunk.cuh
  __device__ __forceinline__ Seen(const WindowCache& c, int pos) {
    slots = c.window + c.sink;
    sink = c.sink;
    ns = min(sink, pos);
    a_hi = base = 0;
    if (pos > sink) {
      const int lr = (pos - 1 - sink) % c.window;
      base = pos - 1 - lr;
      a_hi = sink + lr + 1;
    }
  }
  __device__ __forceinline__ uint32_t bits(int p, int c0) const {
    const int window = slots - sink, x = p - base - window + 1;
    return bits_to(ns - 1 - c0) | (bits_to(a_hi - 1 - c0) & ~bits_to(sink + max(0, x) - 1 - c0)) |
           (base > sink && a_hi > 0 ? bits_to(slots - 1 - c0) & ~bits_to(max(a_hi, sink + x + window) - 1 - c0)
                                    : 0u);
  }
};

// Four bytes global -> shared, of which `bytes` are read and the others zeros.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Codes as fp16 values of whole numbers: bytes 0, 1 and 2, 3, or (EVEN) 0, 2 and 1, 3.
template <bool EVEN>
__device__ __forceinline__ void whole16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  whole_of<__half, EVEN>(w, lo, hi);
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // 8 x 8 of 16 bits between the lanes
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <class T, class TO, int NT>
__global__ void __launch_bounds__(THREADS, 3)
rows8_kernel(const __grid_constant__ Maps maps, Args a, Plan plan, DevCtl ctl) {
  constexpr int HB = 8 * NT, NR = 2 * NT;  // rows of a unit, and those of a thread's scores
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sm = smem_u32(smem);
  const WindowCache& c = a.cache.c;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int KV = c.KV, G = a.H / KV;
  griddep_launch_dependents();  // the join waits for this whole grid
  const int cut = (int)blockIdx.x - plan.whole;  // < 0: a whole unit
  const int parts = cut < 0 ? 1 : plan.parts, part = cut < 0 ? 0 : cut % parts;
  const int part_slots = cut < 0 ? 1 << 30 : plan.part_slots;
  const int unit = cut < 0 ? (int)blockIdx.x : plan.whole + cut / parts;
  const uint32_t bar = sm + OFF_BAR;
  int* const found = reinterpret_cast<int*>(smem + OFF_FOUND);
  int* const passed = reinterpret_cast<int*>(smem + OFF_BAR + STAGES * 8);
  if (tid < STAGES) {
    mbar_init(bar + 8 * tid, 1);
    passed[tid] = 0;
    fence_barrier_init();
  }
  if (tid == 0) {
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }

  // ---- the unit: sequence b, key head kv, rows 16 grp .. of its (token, head) rows
  Sequence s;
  int b, kv, grp;
  if (!a.tok.start) {
    const int groups = (G + HB - 1) / HB;
    grp = unit % groups;
    kv = unit / groups % KV;
    b = unit / groups / KV;
    s.first = b;
    s.tokens = 1;
    {
      // the token's rows, which are asked for one behind the other below: 128 bytes a thread
      const T* q = static_cast<const T*>(a.q) + ((long long)b * a.H + kv * G + grp * HB) * kDK;
      const int n = (min(HB, G - grp * HB) * kDK + 63) / 64;
      if (tid < n) prefetch_l2(q + 64 * tid);
      else if (tid >= 32 && tid < 35)
        prefetch_l2(static_cast<const T*>(a.v) + ((long long)b * KV + kv) * kDV + 64 * (tid - 32));
      else if (tid >= 64 && tid < 66)
        prefetch_l2(static_cast<const T*>(a.k) + ((long long)b * KV + kv) * kDK + 64 * (tid - 64));
    }
    s.pos = __ldg(a.tok.pos + b);
    s.page = __ldg(c.page + b);
    if (s.page < 0 || s.page >= c.n_pages || s.pos < 0) {
      if (tid == 0) record_error(ctl, DEV_RANGE);
      s.tokens = 0;
    }
    __syncthreads();
  } else {
    // sums of groups over a slice of the sequences a thread, and a search
    int* const upto = reinterpret_cast<int*>(smem + OFF_FACTORS);
    int* const sums = upto + THREADS + 1;
    const int slice = (c.n + THREADS - 1) / THREADS;
    const int lo = min(tid * slice, c.n), hi = min(lo + slice, c.n);
    int mine = 0;
    for (int i = lo; i < hi; ++i) mine += (sequence(c, a.tok, i, ctl).tokens * G + HB - 1) / HB;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += y;
    }
    if (lane == 31) sums[w] = sum;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < w; ++i) before += sums[i];
    upto[tid + 1] = before + sum;
    if (tid == 0) upto[0] = 0;
    __syncthreads();
    const long long total = (long long)upto[THREADS] * KV;
    if (blockIdx.x == 0 && tid == 0 && plan.parts > 1) *(int*)a.workspace = (int)total;
    if (unit >= total) return;
    if ((long long)upto[tid] * KV <= unit && unit < (long long)upto[tid + 1] * KV) {
      int left = unit - upto[tid] * KV, i = lo;
      for (;; ++i) {
        const int n = (sequence(c, a.tok, i, ctl).tokens * G + HB - 1) / HB * KV;
        if (left < n) {
          found[0] = i;
          found[1] = left / (n / KV);
          found[2] = left % (n / KV);
          break;
        }
        left -= n;
      }
    }
    __syncthreads();
    b = found[0];
    kv = found[1];
    grp = found[2];
    s = sequence(c, a.tok, b, ctl);
  }
  const int rows = min(HB, s.tokens * G - grp * HB);  // <= 0: a sequence that is left as it is
  if (!a.tok.start && plan.parts > 1 && blockIdx.x == 0 && tid == 0) *(int*)a.workspace = (int)plan.units;
  if (cut >= 0 && part == 0 && tid == 0 && plan.parts > 1)
    static_cast<CutUnit*>(a.workspace)[1 + cut / parts] = CutUnit{s.first, grp * HB, max(rows, 0), kv};
  if (rows <= 0) return;

  const Seen seen(c, s.pos);
  const int held = min(s.pos, seen.slots);
  const int lo = part * part_slots, hi = min(held, lo + part_slots);
  const int page = s.page * c.pool_layers + c.layer;
  const int i0 = grp * HB / G, i1 = (grp * HB + rows - 1) / G;  // the rows' tokens
  // slots that all rows see: 0 .. s_end-1, a_from .. a_end-1, b_from ..
  int s_end = seen.ns, a_from = 0, a_end = 0, b_from = seen.slots;
  {
    const int window = c.window, y = s.pos + i1 - seen.base - window + 1;
    if (seen.a_hi > 0) {
      a_from = min(c.sink + max(0, y), seen.a_hi);
      a_end = seen.a_hi;
      if (seen.base > c.sink) b_from = min(max(seen.a_hi, c.sink + y + window), seen.slots);
      if (b_from == a_end) a_end = seen.slots;
      if (a_from == s_end) {
        s_end = a_end;
      }
    }
  }
  auto whole = [&](int s0) {
    return s0 + SB <= hi && (s0 + SB <= s_end || (s0 >= a_from && s0 + SB <= a_end) || s0 >= b_from);
  };

  const int tiles = hi > lo ? (hi - lo + SB * WARPS - 1) / (SB * WARPS) : 0;
  auto first_slot = [&](int i) { return lo + i * ROUND + w * SB; };
  const signed char* pe = a.cache.exps + ((long long)page * KV + kv) * seen.slots * 2;
  const int skew = (int)(reinterpret_cast<uintptr_t>(pe) & 2);
  auto fetch = [&](int i) {  // round i, by one thread: slots lo + i ROUND ..
    if (i >= tiles) return;
    const uint32_t st = sm + i % STAGES * STAGE, full = bar + 8 * (i % STAGES);
    mbar_arrive_expect_tx(full, STAGE);
#pragma unroll
    for (int j = 0; j < 3; ++j)
      tma_load_4d(st + j * V_BOX, &maps.v, full, 64 * j, kv, lo + i * ROUND, page);
    tma_load_4d(st + OFF_KEYS, &maps.k, full, 0, kv, lo + i * ROUND, page);
  };
  auto fetch_exps = [&](int i) {  // of the warp's tile of round i
    // exponents, two bytes a slot, in words: where the row starts in the middle of one, from there
    const int s0 = first_slot(i);
    if (i < tiles && s0 < hi && lane <= SB / 2) {
      const long long from = 2ll * s0 - skew + 4 * lane;  // byte of the row
      copy4(sm + OFF_EXPS + (w * STAGES + i % STAGES) * EXPS + 4 * lane,
            pe + (from < 2ll * hi ? from : 2ll * s0 - skew), (int)min(max(2ll * hi - from, 0ll), 4ll));
    }
    copy_commit();
  };
  if (tid == 0)
    for (int i = 0; i < STAGES; ++i) fetch(i);
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch_exps(i);

  // ---- queries: row 8 n + g of the unit's (the last one again behind them); step 2 j + h of the product
  // has channels 32 j + 8 t + 4 h .. + 3 of thread t of a row's four
  const int g = lane >> 2, t = lane & 3, t2 = t * 2;
  auto token = [&](int r) { return (grp * HB + min(r, rows - 1)) / G; };  // of row r
  uint32_t qf[NT][kDK / 16][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int R = grp * HB + min(8 * n + g, rows - 1), i = R / G;
    const T* q = static_cast<const T*>(a.q) + ((long long)(s.first + i) * a.H + kv * G + R - i * G) * kDK;
#pragma unroll
    for (int j = 0; j < kDK / 16; ++j) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(q + 32 * (j >> 1) + 8 * t + 4 * (j & 1)));
      qf[n][j][0] = x.x;
      qf[n][j][1] = x.y;
    }
  }
  // A thread's scores are of slots g, g + 8 and rows 8 n + t2, + 1 (NR of them); its sums of channels
  // 16 c + 2 g (0, 1) and + 1 (2, 3) and the same rows.
  int at[NR];  // the rows' positions
#pragma unroll
  for (int r = 0; r < NR; ++r) at[r] = s.pos + token(8 * (r >> 1) + t2 + (r & 1));
  float acc[kDV / 16][NT][4];
#pragma unroll
  for (int j = 0; j < kDV / 16; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j][n][k] = 0.f;
  float m[NR], l[NR];  // base 2; l of this thread's slots
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  int e_ref = 0;  // acc is in units of 2^e_ref (-60 at least: what is below 2^-78 in a page is lost)

  // The maxima of a tile's scores (base 2) over its slots; o and the sums go to a new reference only when
  // one passes the old by more than 8 (weights of up to 2^8 lose nothing in fp16).
  auto refer = [&](float (&top)[NR]) {
    bool up = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
      up |= top[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float now = top[r] > m[r] + 8.f ? top[r] : m[r];
        const float keep = now == m[r] || m[r] == -INFINITY ? 1.f : ex2(m[r] - now);
        m[r] = now;
        l[r] *= keep;
#pragma unroll
        for (int j = 0; j < kDV / 16; ++j) {
          acc[j][r >> 1][r & 1] *= keep;
          acc[j][r >> 1][2 + (r & 1)] *= keep;
        }
      }
    }
  };

  // ---- the new tokens, by tiles of 16 in turn
  if (part == 0) {
    const int sinks = max(c.sink - s.pos, 0);
    const T* nk = static_cast<const T*>(a.k) + ((long long)s.first * KV + kv) * kDK;
    const T* nv = static_cast<const T*>(a.v) + ((long long)s.first * KV + kv) * kDV;
#pragma unroll 1
    for (int j0 = 16 * (WARPS - 1 - w); j0 <= i1; j0 += 16 * WARPS) {  // (the last warp has a tile less)
      if (j0 + 15 <= i0 - c.window && j0 >= sinks) continue;
      float z[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[n][k] = 0.f;
      const bool in0 = j0 + g <= i1, in1 = j0 + g + 8 <= i1;
      const T* key = nk + (long long)(j0 + g) * KV * kDK + 8 * t;
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j) {
        uint2 x = make_uint2(0u, 0u), y = x;
        if (in0) x = __ldg(reinterpret_cast<const uint2*>(key + 32 * (j >> 1) + 4 * (j & 1)));
        if (in1)
          y = __ldg(reinterpret_cast<const uint2*>(key + 8ll * KV * kDK + 32 * (j >> 1) + 4 * (j & 1)));
        const uint32_t x4[4] = {x.x, y.x, x.y, y.y};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<T>(z[n], x4, qf[n][j][0], qf[n][j][1]);
      }
      float top[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const uint32_t see = keys_seen(at[r] - s.pos, j0, i1 + 1, c.window, sinks) >> g;
        float &z0 = z[r >> 1][r & 1], &z1 = z[r >> 1][2 + (r & 1)];
        z0 = see & 1 ? z0 * kLog2e : -INFINITY;
        z1 = (see >> 8) & 1 ? z1 * kLog2e : -INFINITY;
        top[r] = fmaxf(z0, z1);
      }
      refer(top);
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float p[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = 2 * n + j;
            p[j] = ex2(z[n][2 * k + j] - (m[r] == -INFINITY ? 0.f : m[r]));
            l[r] += p[j];
          }
          pf[n][k] = transposed(pack2<T>(p[0], p[1]));
        }
      // channels 16 j + 2 g, + 1 of tokens t2, + 1 and + 8, + 9
      const T* val = nv + (long long)(j0 + t2) * KV * kDV + 2 * g;
#pragma unroll
      for (int j = 0; j < kDV / 16; ++j) {
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int d = (k & 1) + 8 * (k >> 1);
          x[k] = 0u;
          if (j0 + t2 + d <= i1)
            x[k] = __ldg(reinterpret_cast<const uint32_t*>(val + (long long)d * KV * kDV + 16 * j));
        }
        const uint32_t x4[4] = {__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                                __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[2], x[3], 0x7632)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<T>(acc[j][n], x4, pf[n][0], pf[n][1]);
      }
    }
    // a single token's codes go into its slot, which it does not see
    if (!a.tok.start && grp == 0 && w == WARPS - 2) {
      uint4 x[3];
      uint2 o[3];
      const bool key = lane < 4, value = lane >= 8 && lane < 16;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        x[i] = key     ? __ldg(reinterpret_cast<const uint4*>(nk) + 4 * i + lane)
               : value ? __ldg(reinterpret_cast<const uint4*>(nv) + 8 * i + lane - 8)
                       : make_uint4(0u, 0u, 0u, 0u);
      const int e = code_row<T, 8>(x, o);  // lanes 4 .. 7 are zeros
      const int mine = slot_at(s.pos, c.window, c.sink);
      const long long dst = ((long long)page * seen.slots + mine) * KV + kv;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (key) static_cast<uint2*>(c.k)[dst * kCK + 4 * i + lane] = o[i];
        if (value) static_cast<uint2*>(c.v)[dst * kCV + 8 * i + lane - 8] = o[i];
      }
      signed char* to = const_cast<signed char*>(pe) + 2ll * mine;
      if (lane == 0) to[0] = (signed char)e;
      if (lane == 8) to[1] = (signed char)e;
    }
  }

  // ---- queries as fp16, scaled into its range by a power of two per row
  float zs[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) zs[r] = 1.f;
  if constexpr (!__is_same(T, __half)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j) top = top2<T>(top, top2<T>(qf[n][j][0], qf[n][j][1]));
      top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float2 f = halves<T>(top);
      const int e = min(max((int)(__float_as_uint(fmaxf(f.x, f.y)) >> 23) - 127, -100), 100);
      const float down = pow2(-e);
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 x = halves<T>(qf[n][j][h]);
          qf[n][j][h] = pack2<__half>(x.x * down, x.y * down);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) zs[2 * n + j] = pow2(__shfl_sync(0xffffffffu, e, 4 * (t2 + j)));
    }
  }

  // ---- the page
  float2* const factors = reinterpret_cast<float2*>(smem + OFF_FACTORS) + 32 * w;
  // where the lane's 16 bytes of a transposed load lie: chunks lane / 16, and + 2
  const int row = lane & 15, swz = (row >> 1) & 3;
  const uint32_t v_at[2] = {(uint32_t)(row * 64 + (((lane >> 4) ^ swz) << 4)),
                            (uint32_t)(row * 64 + (((2 + (lane >> 4)) ^ swz) << 4))};
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) {
    const int s0 = first_slot(i);
    if (s0 >= hi) break;  // (in the last round)
    copy_wait<STAGES - 1>();
    __syncwarp();
    if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * (i % STAGES), (i / STAGES) & 1, ctl))) {
      // the loads on their way land before the ring is used again and before the CTA may exit
      for (int j = i; j < min(i + STAGES, tiles); ++j)
        mbar_wait(bar + 8 * (j % STAGES), (j / STAGES) & 1, ctl, DRAIN_NS);
      break;
    }
    const uint32_t so = i % STAGES * STAGE + w * SB * 64;  // the warp's values, in the first box
    const uint8_t* keys = smem + i % STAGES * STAGE + OFF_KEYS + w * SB * kDK;
    float z[2][NT][4];  // slots 16 h + g, + 8
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[h][n][k] = 0.f;
#pragma unroll
    for (int j = 0; j < kDK / 32; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 x = *reinterpret_cast<const uint2*>(keys + (16 * h + g) * kDK + 32 * j + 8 * t);
        const uint2 y = *reinterpret_cast<const uint2*>(keys + (16 * h + 8 + g) * kDK + 32 * j + 8 * t);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t x4[4];
          whole16<false>(k ? x.y : x.x, x4[0], x4[2]);
          whole16<false>(k ? y.y : y.x, x4[1], x4[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<__half>(z[h][n], x4, qf[n][2 * j + k][0], qf[n][2 * j + k][1]);
        }
      }
    // the largest exponent of the values that are seen so far: o in its units.  (The first row sees what any
    // does.  A slot that none sees may be written meanwhile.)
    const bool all = whole(s0);
    const char2 ex = reinterpret_cast<const char2*>(smem + OFF_EXPS + (w * STAGES + i % STAGES) * EXPS +
                                                    skew)[lane];
    int ev = (signed char)ex.y;
    if (!all && !((seen.bits(s.pos + i0, s0) >> lane) & 1)) ev = -128;
    const int e_top = max(__reduce_max_sync(0xffffffffu, ev), -60);
    if (e_top > e_ref || i == 0) {
      const float f = pow2(max(e_ref - e_top, -126));
      e_ref = e_top;
      if (i > 0 || part == 0)
#pragma unroll
        for (int j = 0; j < kDV / 16; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][n][k] *= f;
    }
    // factors of slot `lane`, and then of this thread's, 8 k + g
    factors[lane] = make_float2(scale_of((signed char)ex.x) * kLog2e, pow2(max(ev - e_ref, -126)));
    __syncwarp();
    float2 f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = factors[8 * k + g];
    float top[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) top[r] = -INFINITY;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k >> 1][r >> 1][2 * (k & 1) + (r & 1)] *= f[k].x;
    if (!all) {
      const uint32_t there = bits_to(hi - 1 - s0);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const uint32_t see = (seen.bits(at[r], s0) & there) >> g;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!((see >> (8 * k)) & 1)) z[k >> 1][r >> 1][2 * (k & 1) + (r & 1)] = -INFINITY;
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int k = 0; k < 4; ++k) top[r] = fmaxf(top[r], z[k >> 1][r >> 1][2 * (k & 1) + (r & 1)]);
      top[r] *= zs[r];
    }
    refer(top);
    uint32_t pf[2][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float base[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) base[j] = m[2 * n + j] == -INFINITY ? 0.f : m[2 * n + j];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p[j] = ex2(fmaf(z[k >> 1][n][2 * (k & 1) + j], zs[2 * n + j], -base[j]));
          l[2 * n + j] += p[j];
        }
        pf[k >> 1][n][k & 1] = transposed(pack2<__half>(p[0] * f[k].y, p[1] * f[k].y));
      }
    }
    // codes of slots 16 h + t2, + 1 (x[0]) and + 8, + 9 (x[1]), channels 16 ch + 2 g, + 1; x[2], x[3]:
    // channels 16 ch + 16 + ..; a row's chunks are swizzled by row / 2 & 3, the same for both h
#pragma unroll
    for (int h = 0; h < 2; ++h)  // slots 16 h ..
#pragma unroll
      for (int ch = 0; ch < kDV / 16; ch += 2) {
        uint32_t x[4];
        ldsm4t(x, sm + so + (ch & 2 ? v_at[1] : v_at[0]) + (ch >> 2) * V_BOX + h * 1024);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t x4[4];
          whole16<true>(x[2 * y], x4[0], x4[1]);
          whole16<true>(x[2 * y + 1], x4[2], x4[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<__half>(acc[ch + y][n], x4, pf[h][n][0], pf[h][n][1]);
        }
      }
    // the warp that is the last to leave the stage has it filled again: one thread's loads for all four (by
    // each warp for itself they take 1,000 of a tile's 4,000 cycles)
    __syncwarp();
    fetch_exps(i + STAGES);
    if (lane == 0) {
      __threadfence_block();
      if (atomicAdd(passed + i % STAGES, 1) == WARPS - 1) {
        passed[i % STAGES] = 0;
        fence_proxy_async();
        fetch(i + STAGES);
      }
    }
    __syncwarp();
  }
  copy_wait<0>();
  __syncthreads();

  // ---- join the warps: o, m and l of each row through shared memory
  float* so = reinterpret_cast<float*>(smem);              // [WARPS][HB][JOIN_ROW]
  float* sml = so + WARPS * HB * JOIN_ROW;                 // [WARPS][HB][2]
  static_assert(WARPS * HB * (JOIN_ROW + 2) * 4 <= RING, "the join fits the ring");
  const float unit_of = pow2(min(max(e_ref, -126), 127));
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = 8 * (r >> 1) + t2 + (r & 1);
    float sum = l[r];
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (g == 0) {
      sml[(w * HB + row) * 2] = m[r];
      sml[(w * HB + row) * 2 + 1] = sum;
    }
#pragma unroll
    for (int j = 0; j < kDV / 16; ++j)
      *reinterpret_cast<float2*>(so + (w * HB + row) * JOIN_ROW + 16 * j + 2 * g) =
          make_float2(acc[j][r >> 1][r & 1] * unit_of, acc[j][r >> 1][2 + (r & 1)] * unit_of);
  }
  __syncthreads();
  for (int x = tid; x < rows * (kDV / 2); x += THREADS) {
    const int row = x / (kDV / 2), ch = x % (kDV / 2) * 2;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) top = fmaxf(top, sml[(k * HB + row) * 2]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float f = ex2(sml[(k * HB + row) * 2] - base);
      const float2 o = *reinterpret_cast<const float2*>(so + (k * HB + row) * JOIN_ROW + ch);
      sum = fmaf(f, sml[(k * HB + row) * 2 + 1], sum);
      o0 = fmaf(f, o.x, o0);
      o1 = fmaf(f, o.y, o1);
    }
    if (parts == 1) {
      const int R = grp * HB + row, i = R / G;
      const float inv = 1.f / sum;  // the token itself is there: sum > 0
      store2(static_cast<TO*>(a.o) + ((long long)(s.first + i) * a.H + kv * G + R - i * G) * kDV + ch,
             o0 * inv, o1 * inv);
    } else {
      const long long cuts = plan.units - plan.whole;
      float* pw = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + table_bytes(cuts)) +
                  (((long long)(unit - plan.whole) * HB + row) * parts + part) * (kDV + 2);
      *reinterpret_cast<float2*>(pw + ch) = make_float2(o0, o1);
      if (ch == 0) *reinterpret_cast<float2*>(pw + kDV) = make_float2(top, sum);
    }
  }
}

// Joins the parts of a row of a cut unit, in order: o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.
template <class TO>
__global__ void __launch_bounds__(kDV / 2)
rows8_join_kernel(Args a, Plan plan) {
  griddep_wait();
  const int HB = plan.rows, cut = blockIdx.x / HB, row = blockIdx.x % HB, parts = plan.parts;
  const CutUnit* table = static_cast<const CutUnit*>(a.workspace);
  if (plan.whole + cut >= table->first) return;  // (the first word: units)
  const CutUnit u = table[1 + cut];
  if (row >= u.rows) return;
  const float* pw = reinterpret_cast<const float*>(static_cast<const char*>(a.workspace) +
                                                   table_bytes(plan.units - plan.whole)) +
                    ((long long)cut * HB + row) * parts * (kDV + 2);
  const int c = threadIdx.x * 2;
  float top = -INFINITY;
  for (int k = 0; k < parts; ++k) top = fmaxf(top, pw[k * (kDV + 2) + kDV]);
  float sum = 0.f, o0 = 0.f, o1 = 0.f;
  for (int k = 0; k < parts; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(pw + k * (kDV + 2) + kDV);
    const float2 x = *reinterpret_cast<const float2*>(pw + k * (kDV + 2) + c);
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    sum = fmaf(f, ml.y, sum);
    o0 = fmaf(f, x.x, o0);
    o1 = fmaf(f, x.y, o1);
  }
  const float inv = 1.f / sum;
  const int KV = a.cache.c.KV, G = a.H / KV, R = u.row0 + row, i = R / G;
  store2(static_cast<TO*>(a.o) + ((long long)(u.first + i) * a.H + u.kv * G + R - i * G) * kDV + c, o0 * inv,
         o1 * inv);
}

// `units` at most, `likely` so many: as many whole ones as fill the device one or more times, and parts of
// the others that fill it once more, of at least one round of the warps' tiles (128 slots); nothing is
// cut where two do not fit.
inline Plan make_plan(long long units, long long likely, int rows, int slots, int n_sm) {
  const int hold = std::max(3 * n_sm, 1), unit = SB * WARPS, rest = (int)(likely % hold);
  const int most = std::min((slots + unit - 1) / unit, 64);
  const int parts = rest ? std::min(hold / rest, most) : 1;
  if (parts < 2) return Plan{units, (int)units, 1, 0, rows};
  const int part_slots = ((slots + parts - 1) / parts + unit - 1) / unit * unit;
  return Plan{units, (int)(likely - rest), parts, part_slots, rows};
}

inline bool make_maps(Maps* m, const ServeCache& cache) {
  auto fn = encode_tiled_fn();
  if (!fn) return false;
  const WindowCache& c = cache.c;
  const long long slots = c.window + c.sink, pages = (long long)c.n_pages * c.pool_layers;
  for (int i = 0; i < 2; ++i) {
    const int d = i ? kDV : kDK;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)c.KV, (cuuint64_t)slots, (cuuint64_t)pages};
    cuuint64_t strides[3] = {(cuuint64_t)d, (cuuint64_t)d * c.KV, (cuuint64_t)d * c.KV * slots};
    cuuint32_t box[4] = {i ? 64u : (cuuint32_t)kDK, 1u, (cuuint32_t)ROUND, 1u};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    if (fn(i ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? c.v : c.k, dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, i ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

template <class T, class TO, int NT>
cudaError_t run(const Args& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  Maps m;
  if (!make_maps(&m, a.cache)) return cudaErrorInvalidValue;
  auto kern = rows8_kernel<T, TO, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long cut = plan.units - plan.whole;
  kern<<<(unsigned)(plan.whole + cut * plan.parts), THREADS, SMEM, stream>>>(m, a, plan, ctl);
  if ((e = cudaGetLastError()) != cudaSuccess || plan.parts == 1) return e;
  PdlLaunch l(dim3((unsigned)(cut * plan.rows)), dim3(kDV / 2), 0, stream, true);
  return cudaLaunchKernelEx(&l.cfg, rows8_join_kernel<TO>, a, plan);
}

template <class T, class TO>
cudaError_t run(const Args& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  return plan.rows == 8 ? run<T, TO, 1>(a, plan, ctl, stream) : run<T, TO, 2>(a, plan, ctl, stream);
}
inline cudaError_t launch(const Args& a, gla_dtype out, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  const bool wide = out == GLA_FP32;
  if (a.cache.c.type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, plan, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, plan, ctl, stream);
  return wide ? run<__half, float>(a, plan, ctl, stream) : run<__half, __half>(a, plan, ctl, stream);
}

}  // namespace rows8
}  // namespace gla
