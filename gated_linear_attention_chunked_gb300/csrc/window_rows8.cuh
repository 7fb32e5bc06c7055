// window_rows8.cuh -- the windowed attention of few new tokens per sequence over pages of 8 bits: one each
// (the decode step) or a handful (drafts).  16 rows, (token, query head) of one key head, are a unit and the
// rows of a warp-level tensor-core product; a CTA takes a unit, or a part of its page's slots, its four
// warps walk the slots in tiles of 32 with rings of their own (TMA), running maxima and sums of their own,
// and join them at the end.
//
//   z = 2^e (q . c),  o = sum p 2^e c / sum p   with the rows' codes c as fp16 operands, exactly
//
// whatever the call's type: fp16 is a byte permute and a subtraction away from a code (0x6400 | u is 1024 +
// u), bf16 twice as much.  Queries of bf16 are scaled by a power of two per row into fp16's range; the
// values' 2^e goes into the weight, relative to the largest e of the tiles so far, so that a weight rounds
// by 2^-11 of itself or by 2^-25 of the weight of the page's largest row.  The new tokens' own keys and values are
// taken as given, in the call's type, a tile of 16 at a time straight from global memory.
//
// Bound by HBM: 290 bytes a slot and key head, with 600 instructions a warp and tile; three CTAs an SM
// hide the latencies of each other's begin and end.  Keys are read eight channels at a time, in an order of
// the channels that the query's registers share; values by transposed loads of pairs of channels, which come
// apart in the same permutes.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "tmap.h"
#include "window_packed.cuh"

namespace gla {
namespace rows8 {

constexpr int WARPS = 4, THREADS = 32 * WARPS, SB = 32, STAGES = 2, HB = 16;
constexpr int V_BOX = SB * 64, OFF_KEYS = 3 * V_BOX;  // a stage: values in 3 boxes of 64 channels, keys
constexpr int STAGE = OFF_KEYS + SB * kDK;             // 9,216 bytes
constexpr int RING = WARPS * STAGES * STAGE;
constexpr int OFF_BAR = RING;                          // mbarrier [warp][stage]
constexpr int SMEM = RING + WARPS * STAGES * 8 + 1024;
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
  int whole, parts, part_slots;
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
             ? table_bytes(cut) + (size_t)cut * HB * p.parts * (kDV + 2) * sizeof(float)
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

// Codes as fp16 values of whole numbers: bytes 0, 1 and 2, 3, or (EVEN) 0, 2 and 1, 3.
template <bool EVEN>
__device__ __forceinline__ void whole16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  whole_of<__half, EVEN>(w, lo, hi);
}

template <class T, class TO>
__global__ void __launch_bounds__(THREADS, 3)
rows8_kernel(const __grid_constant__ Maps maps, Args a, Plan plan, DevCtl ctl) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ int found[4];
  const uint32_t sm = smem_u32(smem);
  const WindowCache& c = a.cache.c;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int KV = c.KV, G = a.H / KV;
  griddep_launch_dependents();  // the join waits for this whole grid
  const int cut = (int)blockIdx.x - plan.whole;  // < 0: a whole unit
  const int parts = cut < 0 ? 1 : plan.parts, part = cut < 0 ? 0 : cut % parts;
  const int part_slots = cut < 0 ? 1 << 30 : plan.part_slots;
  const int unit = cut < 0 ? (int)blockIdx.x : plan.whole + cut / parts;
  const uint32_t bar = sm + OFF_BAR + w * STAGES * 8;
  if (tid < WARPS * STAGES) {
    mbar_init(sm + OFF_BAR + 8 * tid, 1);
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
    s.pos = __ldg(a.tok.pos + b);
    s.page = __ldg(c.page + b);
    if (s.page < 0 || s.page >= c.n_pages || s.pos < 0) {
      if (tid == 0) record_error(ctl, DEV_RANGE);
      s.tokens = 0;
    }
    __syncthreads();
  } else {
    // sums of groups over a slice of the sequences a thread, and a search
    __shared__ int upto[THREADS + 1], sums[WARPS];
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
  auto first_slot = [&](int i) { return lo + (i * WARPS + w) * SB; };
  const signed char* pe = a.cache.exps + ((long long)page * KV + kv) * seen.slots * 2;
  auto fetch = [&](int i) {  // warp w's tile i: slots lo + (i WARPS + w) SB ..
    const int s0 = first_slot(i);
    if (i < tiles && s0 < hi && lane == 0) {
      const uint32_t st = sm + (w * STAGES + i % STAGES) * STAGE, full = bar + 8 * (i % STAGES);
      mbar_arrive_expect_tx(full, STAGE);
#pragma unroll
      for (int j = 0; j < 3; ++j) tma_load_4d(st + j * V_BOX, &maps.v, full, 64 * j, kv, s0, page);
      tma_load_4d(st + OFF_KEYS, &maps.k, full, 0, kv, s0, page);
    }
  };
  auto exponents = [&](int i) -> uint32_t {  // of slot `lane` of the tile, two bytes; 0x8080: none
    const int slot = first_slot(i) + lane;
    return i < tiles && slot < hi ? __ldg(reinterpret_cast<const unsigned short*>(pe) + slot) : 0x8080u;
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch(i);
  uint32_t ex_next = exponents(0);

  // ---- queries: rows g and g + 8 (zeros behind the unit's); step 2 j + h of the product has channels
  // 32 j + 8 t + 4 h .. + 3 of thread t of a row's four
  const int g = lane >> 2, t = lane & 3, t2 = t * 2;
  int at[2];  // the rows' positions
  uint32_t qf[kDK / 16][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int R = grp * HB + min(g + 8 * r, rows - 1), i = R / G;
    at[r] = s.pos + i;
    const T* q = static_cast<const T*>(a.q) + ((long long)(s.first + i) * a.H + kv * G + R - i * G) * kDK;
#pragma unroll
    for (int j = 0; j < kDK / 16; ++j) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(q + 32 * (j >> 1) + 8 * t + 4 * (j & 1)));
      qf[j][r] = x.x;
      qf[j][2 + r] = x.y;
    }
  }
  float acc[kDV / 8][4];
#pragma unroll
  for (int j = 0; j < kDV / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // base 2; l of this thread's columns
  int e_ref = 0;  // acc is in units of 2^e_ref (-60 at least: what is below 2^-78 in a page is lost)

  // The maxima of a tile's scores (base 2) over the quad; o and the sums go to a new reference only
  // when one passes the old by more than 8 (weights of up to 2^8 lose nothing in fp16).
  auto refer = [&](float (&top)[2]) {
    bool up = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = quad_max(top[r]);
      up |= top[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float now = top[r] > m[r] + 8.f ? top[r] : m[r];
        const float keep = now == m[r] || m[r] == -INFINITY ? 1.f : ex2(m[r] - now);
        m[r] = now;
        l[r] *= keep;
#pragma unroll
        for (int j = 0; j < kDV / 8; ++j) {
          acc[j][2 * r] *= keep;
          acc[j][2 * r + 1] *= keep;
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
    for (int j0 = 16 * w; j0 <= i1; j0 += 16 * WARPS) {
      if (j0 + 15 <= i0 - c.window && j0 >= sinks) continue;
      float z[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int tok = j0 + 8 * n + g;
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = 0.f;
#pragma unroll
        for (int j = 0; j < kDK / 16; ++j) {
          uint2 x = make_uint2(0u, 0u);
          if (tok <= i1)
            x = __ldg(reinterpret_cast<const uint2*>(nk + (long long)tok * KV * kDK + 32 * (j >> 1) +
                                                     8 * t + 4 * (j & 1)));
          mma16816<T>(z[n], qf[j], x.x, x.y);
        }
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t see = keys_seen(at[r] - s.pos, j0, i1 + 1, c.window, sinks);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& x = z[n][2 * r + j];
            x = (see >> (8 * n + t2 + j)) & 1 ? x * kLog2e : -INFINITY;
            top[r] = fmaxf(top[r], x);
          }
      }
      refer(top);
      uint32_t pf[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(z[n][2 * r] - base), p1 = ex2(z[n][2 * r + 1] - base);
          l[r] += p0 + p1;
          pf[2 * n + r] = pack2<T>(p0, p1);
        }
      }
      // channels 16 j + 2 g, + 1 of tokens t2, + 1 and + 8, + 9
#pragma unroll
      for (int j = 0; j < kDV / 16; ++j) {
        uint32_t x[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int tok = j0 + t2 + (n & 1) + 8 * (n >> 1);
          x[n] = 0u;
          if (tok <= i1)
            x[n] = __ldg(reinterpret_cast<const uint32_t*>(nv + (long long)tok * KV * kDV + 16 * j + 2 * g));
        }
        mma16816<T>(acc[2 * j], pf, __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
        mma16816<T>(acc[2 * j + 1], pf, __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
      }
    }
    // a single token's codes go into its slot, which it does not see
    if (!a.tok.start && grp == 0 && w == WARPS - 1) {
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
  float zs[2] = {kLog2e, kLog2e};
  if constexpr (!__is_same(T, __half)) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j) top = top2<T>(top, top2<T>(qf[j][r], qf[j][2 + r]));
      top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float2 f = halves<T>(top);
      const int e = min(max((int)(__float_as_uint(fmaxf(f.x, f.y)) >> 23) - 127, -100), 100);
      const float down = pow2(-e);
      zs[r] = pow2(e) * kLog2e;
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 x = halves<T>(qf[j][2 * h + r]);
          qf[j][2 * h + r] = pack2<__half>(x.x * down, x.y * down);
        }
    }
  }

  // ---- the page
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) {
    const int s0 = first_slot(i);
    if (s0 >= hi) break;  // (and so are the warp's later tiles)
    const uint32_t ex = ex_next;
    ex_next = exponents(i + 1);
    if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * (i % STAGES), (i / STAGES) & 1, ctl))) {
      // the loads on their way land before the ring is used again and before the CTA may exit
      for (int j = i; j < min(i + STAGES, tiles) && first_slot(j) < hi; ++j)
        mbar_wait(bar + 8 * (j % STAGES), (j / STAGES) & 1, ctl, DRAIN_NS);
      break;
    }
    const uint32_t so = (w * STAGES + i % STAGES) * STAGE;
    const uint8_t* keys = smem + so + OFF_KEYS;
    float z[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // slots 8 n ..
#pragma unroll
      for (int j = 0; j < 4; ++j) z[n][j] = 0.f;
#pragma unroll
      for (int j = 0; j < kDK / 32; ++j) {
        const uint2 x = *reinterpret_cast<const uint2*>(keys + (8 * n + g) * kDK + 32 * j + 8 * t);
        uint32_t b0, b1;
        whole16<false>(x.x, b0, b1);
        mma16816<__half>(z[n], qf[2 * j], b0, b1);
        whole16<false>(x.y, b0, b1);
        mma16816<__half>(z[n], qf[2 * j + 1], b0, b1);
      }
    }
    // the largest exponent of the values that are seen so far: o in its units.  (The first row sees what any
    // does.  A slot that none sees may be written meanwhile.)
    uint32_t see[2] = {~0u, ~0u};
    int e_top = (int)(signed char)(ex >> 8);
    if (!whole(s0)) {
      const uint32_t there = bits_to(hi - 1 - s0);
#pragma unroll
      for (int r = 0; r < 2; ++r) see[r] = seen.bits(at[r], s0) & there;
      if (!((seen.bits(s.pos + i0, s0) >> lane) & 1)) e_top = -128;
    }
    e_top = max(__reduce_max_sync(0xffffffffu, e_top), -60);
    if (e_top > e_ref || i == 0) {
      const float f = pow2(max(e_ref - e_top, -126));
      e_ref = e_top;
      if (i > 0 || part == 0)
#pragma unroll
        for (int j = 0; j < kDV / 8; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[j][k] *= f;
    }
    // this thread's columns: slots 8 n + t2, + 1
    float sv[4][2], top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t e = __shfl_sync(0xffffffffu, ex, 8 * n + t2 + j);
        const float sk = scale_of((signed char)(e & 255));
        sv[n][j] = pow2(max((int)(signed char)(e >> 8) - e_ref, -126));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float& x = z[n][2 * r + j];
          x = (see[r] >> (8 * n + t2 + j)) & 1 ? x * (sk * zs[r]) : -INFINITY;
          top[r] = fmaxf(top[r], x);
        }
      }
    refer(top);
    uint32_t pf[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float p0 = ex2(z[n][2 * r] - base), p1 = ex2(z[n][2 * r + 1] - base);
        l[r] += p0 + p1;
        pf[n >> 1][2 * (n & 1) + r] = pack2<__half>(p0 * sv[n][0], p1 * sv[n][1]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)  // slots 16 h ..
#pragma unroll
      for (int ch = 0; ch < kDV / 16; ch += 2) {
        // codes of slots 16 h + t2, + 1 (x[0]) and + 8, + 9 (x[1]), channels 16 ch + 2 g, + 1; x[2],
        // x[3]: channels 16 ch + 16 + ..
        const int row = 16 * h + (lane & 15), cc = ch + (lane >> 4);
        uint32_t x[4];
        ldsm4t(x, sm + so + (cc >> 2) * V_BOX + row * 64 + (((cc & 3) ^ ((row >> 1) & 3)) << 4));
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t e0, o0, e1, o1;
          whole16<true>(x[2 * y], e0, o0);
          whole16<true>(x[2 * y + 1], e1, o1);
          mma16816<__half>(acc[2 * (ch + y)], pf[h], e0, e1);
          mma16816<__half>(acc[2 * (ch + y) + 1], pf[h], o0, o1);
        }
      }
    __syncwarp();  // the stage is free for the copy of the next round
    fetch(i + STAGES);
  }
  __syncthreads();

  // ---- join the warps: o, m and l of each row through shared memory
  float* so = reinterpret_cast<float*>(smem);              // [WARPS][HB][kDV]
  float* sml = so + WARPS * HB * kDV;                      // [WARPS][HB][2]
  static_assert(WARPS * HB * (kDV + 2) * 4 <= RING, "the join fits the ring");
  const float unit_of = pow2(min(max(e_ref, -126), 127));
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = g + 8 * r;
    const float sum = quad_sum(l[r]);
    if (t == 0) {
      sml[(w * HB + row) * 2] = m[r];
      sml[(w * HB + row) * 2 + 1] = sum;
    }
    // columns t2, t2 + 1 of the even block are channels 16 j + 4 t, + 2, of the odd one + 1, + 3
#pragma unroll
    for (int j = 0; j < kDV / 16; ++j)
      *reinterpret_cast<float4*>(so + (w * HB + row) * kDV + 16 * j + 4 * t) =
          make_float4(acc[2 * j][2 * r] * unit_of, acc[2 * j + 1][2 * r] * unit_of,
                      acc[2 * j][2 * r + 1] * unit_of, acc[2 * j + 1][2 * r + 1] * unit_of);
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
      const float2 o = *reinterpret_cast<const float2*>(so + (k * HB + row) * kDV + ch);
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
  const int cut = blockIdx.x / HB, row = blockIdx.x % HB, parts = plan.parts;
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
inline Plan make_plan(long long units, long long likely, int slots, int n_sm) {
  const int hold = std::max(3 * n_sm, 1), unit = SB * WARPS, rest = (int)(likely % hold);
  const int most = std::min((slots + unit - 1) / unit, 64);
  const int parts = rest ? std::min(hold / rest, most) : 1;
  if (parts < 2) return Plan{units, (int)units, 1, 0};
  const int part_slots = ((slots + parts - 1) / parts + unit - 1) / unit * unit;
  return Plan{units, (int)(likely - rest), parts, part_slots};
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
    cuuint32_t box[4] = {i ? 64u : (cuuint32_t)kDK, 1u, (cuuint32_t)SB, 1u};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    if (fn(i ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? c.v : c.k, dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, i ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

template <class T, class TO>
cudaError_t run(const Args& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  Maps m;
  if (!make_maps(&m, a.cache)) return cudaErrorInvalidValue;
  auto kern = rows8_kernel<T, TO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  const long long cut = plan.units - plan.whole;
  kern<<<(unsigned)(plan.whole + cut * plan.parts), THREADS, SMEM, stream>>>(m, a, plan, ctl);
  if ((e = cudaGetLastError()) != cudaSuccess || plan.parts == 1) return e;
  PdlLaunch l(dim3((unsigned)(cut * HB)), dim3(kDV / 2), 0, stream, true);
  return cudaLaunchKernelEx(&l.cfg, rows8_join_kernel<TO>, a, plan);
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
