// window_rows8.cuh -- the windowed attention of few new tokens per sequence over pages of 8 bits: one each
// (the decode step) or a handful (drafts).  8 NT rows, (token, query head) of one key head, are a unit; a
// CTA takes a unit, or a part of its page's slots, in rounds that one thread's TMA brings: each of its four
// warps multiplies a quarter of a round's keys, and then a quarter of the channels of all its values.
//
//   z = 2^e (c . q),  o = sum p 2^e c / sum p   with the rows' codes c as fp16 operands, exactly
//
// whatever the call's type.  An operand of the scores is (c + 128) 2^-24, a value without an exponent: an
// exclusive or and a byte permute; the 128 comes off by a product with the queries' sum before.  The values are
// c itself, one subtraction more: with 128 in sums of thousands of values that cancel, what the tensor cores cut
// off would be 1.5e-4 of the result.
// Queries of bf16 are scaled by a power of two per row into fp16's range; the values' 2^e goes into the
// weight, relative to a common e_ref within 4 of the largest so far, so that a weight rounds by 2^-11 of
// itself or by 2^-25 of the weight of the page's largest row.  The new tokens' own keys and values are taken as
// given, in the call's type, straight from global memory, behind the page.
//
// The codes are the products' first operand (16 slots by channels; 16 channels by slots), the rows their
// columns, eight at a time: most calls have four or eight rows.  Keys are read eight channels at a time, in an
// order of the channels that the queries share; values by transposed loads of pairs of channels, which come
// apart in the permutes.  Weights go to all four warps through shared memory, in units of a maximum that all
// share: they are worked out before it is known whether a score passes it by more than 8, and again in the
// rare round where one does, so that a round has one barrier.
//
// Bound by latency: a CTA's first loads and its last sums are a fifth of its time, and in its rounds it waits for
// HBM, whose rate then is what a copy reaches; the three CTAs of an SM begin and end nearly together.  256 tokens
// on 1,028 slots of 4 key heads, 290 bytes a slot and key head: 65 us, 4.7 TB/s of the 6.7 of a copy (without the
// loads 51 us, without the products 60, without both 29); 96 chunks of four tokens on 2,052 slots 60 us.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "tmap.h"
#include "window_join.cuh"
#include "window_packed.cuh"

namespace gla {
namespace rows8 {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int TILES = kDV / 16 / WARPS;  // a warp's channels, 16 each
constexpr uint64_t DRAIN_NS = 4000000000ull;
static_assert(kDV % (16 * WARPS) == 0, "the warps' channels");

// By the groups of 8 rows.  A round of 128 slots (WIDE) has twice the products in flight for the same waits, but with
// more than one group no room is left for three CTAs of an SM with two such rounds beside the queries: two CTAs, or
// rounds of 64 slots in three stages, or in two where the rows take the room of the third.  make_plan
// has the rule.  Chunks of 4 and 8 tokens on 2,052 slots, 4 key heads, by 128 and by 64 slots: 64 chunks 44 and 58,
// 56 and 86 us; 96 76 and 60, 103 and 88; 128 84 and 86, 105 and 131; 200 123 and 115, 156 and 173.  Of 6, by units of
// 24 rows: 48 and 69, 89 and 71, 92 and 104 (by units of 32 96 chunks took 88).  (One group by 64
// slots: 71 us in place of 68 with 256 tokens on 1,028 slots.  With 5, 4 and 3 CTAs of two stages of 64 slots 69, but
// 96 chunks of two and four tokens took 65 and 74 us in place of 48 and 57; four groups in three stages leave
// room for two CTAs: 96 chunks of eight tokens 101 us in place of 94.)
template <int NT, bool WIDE>
struct Shape {
  static constexpr int HOLD = NT > 1 && WIDE ? 2 : 3;          // CTAs that an SM holds
  static constexpr int SB = WIDE ? 32 : 16;                    // slots of a round for each warp
  static constexpr int STAGES = NT < 4 && !WIDE ? 3 : 2;
  static constexpr int ROUND = WARPS * SB;
  static constexpr int KEYS = ROUND * kDV, STAGE = KEYS + ROUND * kDK;  // a stage: values, keys
  static constexpr int EXPS = 2 * SB + 16;               // the exponents of a warp's slots, from a word's start
  // A warp's weights take the place of its keys of the round, [row][slot].
  static constexpr int SLICE = SB * kDK, P_ROW = 2 * SB + 16;
  static_assert(8 * NT * P_ROW <= SLICE, "weights in place of keys");
};

// What the warps of a unit of NT groups of 8 rows share.
template <int NT, bool WIDE>
struct Shared {
  using S = Shape<NT, WIDE>;
  uint64_t full[S::STAGES], behind;    // mbarriers: a stage is there; the rounds are over
  uint8_t exps[WARPS][S::STAGES][S::EXPS];
  union {
    uint2 q[NT][kDK / 16][32];         // the second operand of the scores' products
    struct {
      int upto[THREADS + 1], sums[WARPS];  // before: units before a slice of the sequences
    } find;
  };
  float z0[8 * NT], zs[8 * NT];        // of a row: - q . (code 0), a score's factor
  float top[WARPS][8 * NT], sum[WARPS][8 * NT];  // (top[0] before the rounds: the scores of one token alone)
  int e_top[WARPS];
  int found[4];
};
template <int NT, bool WIDE>
constexpr int smem_bytes() {
  using S = Shape<NT, WIDE>;
  constexpr int bytes = S::STAGES * S::STAGE + (int)sizeof(Shared<NT, WIDE>) + 512;
  static_assert(S::HOLD * (bytes + 1024) <= 228 * 1024, "shared memory");
  return bytes;
}

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
  int whole, parts, part_slots, rows;  // rows of a unit: 8, 16, 24 or 32
  bool wide;                           // rounds of 128 slots with more than 8
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

// Codes c as fp16 values (c + 128) 2^-24, which have no exponent to be put in: codes 0, 2 and 1, 3 of a word.
__device__ __forceinline__ void whole16(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t u = w ^ 0x80808080u;
  even = __byte_perm(u, 0u, 0x4240);
  odd = __byte_perm(u, 0u, 0x4341);
}
constexpr uint32_t kZero16 = 0x00800080u;  // of code 0

// Two or four 8 x 8 matrices of 16 bits to shared memory, transposed; lane l has the address of row l % 8 of the
// (l / 8)-th.
__device__ __forceinline__ void stsm2t(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void stsm4t(uint32_t at, const uint32_t (&x)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3])
               : "memory");
}

template <class T, class TO, int NT, bool WIDE>
__global__ void __launch_bounds__(THREADS, Shape<NT, WIDE>::HOLD)
rows8_kernel(const __grid_constant__ Maps maps, Args a, Plan plan, DevCtl ctl) {
  constexpr int HB = 8 * NT, NR = 2 * NT;  // rows of a unit, and those of a thread
  using Sh = Shape<NT, WIDE>;
  constexpr int SB = Sh::SB, STAGES = Sh::STAGES, ROUND = Sh::ROUND, STAGE = Sh::STAGE, P_ROW = Sh::P_ROW;
  extern __shared__ __align__(512) uint8_t smem_raw[];  // (the swizzle counts from multiples of 512)
  uint8_t* const smem = (uint8_t*)(((uintptr_t)smem_raw + 511) & ~(uintptr_t)511);
  Shared<NT, WIDE>& sh = *reinterpret_cast<Shared<NT, WIDE>*>(smem + STAGES * STAGE);
  const uint32_t sm = smem_u32(smem), bar = smem_u32(sh.full);
  const WindowCache& c = a.cache.c;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int KV = c.KV, G = a.H / KV;
  griddep_launch_dependents();  // the join waits for this whole grid
  const int cut = (int)blockIdx.x - plan.whole;  // < 0: a whole unit
  const int parts = cut < 0 ? 1 : plan.parts, part = cut < 0 ? 0 : cut % parts;
  const int part_slots = cut < 0 ? 1 << 30 : plan.part_slots;
  const int unit = cut < 0 ? (int)blockIdx.x : plan.whole + cut / parts;
  if (tid <= STAGES) {
    mbar_init(tid < STAGES ? bar + 8 * tid : smem_u32(&sh.behind), 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }

  // ---- the unit: sequence b, key head kv, rows 8 NT grp .. of its (token, head) rows
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
    // sums of groups over a slice of the sequences a thread, and a search; the sums stop at the groups that the
    // plan has room for, which sequences that overlap, where `start` decreases, could pass
    const int room = (int)(plan.units / KV);
    int *const upto = sh.find.upto, *const sums = sh.find.sums;
    const int slice = (c.n + THREADS - 1) / THREADS;
    const int lo = min(tid * slice, c.n), hi = min(lo + slice, c.n);
    int mine = 0;
    for (int i = lo; i < hi; ++i) mine = min(mine + (sequence(c, a.tok, i, ctl).tokens * G + HB - 1) / HB, room);
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum = min(sum + y, room);
    }
    if (lane == 31) sums[w] = sum;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < w; ++i) before = min(before + sums[i], room);
    upto[tid + 1] = min(before + sum, room);
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
          sh.found[0] = i;
          sh.found[1] = left / (n / KV);
          sh.found[2] = left % (n / KV);
          break;
        }
        left -= n;
      }
    }
    __syncthreads();
    b = sh.found[0];
    kv = sh.found[1];
    grp = sh.found[2];
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

  // ---- rounds
  const int rounds = hi > lo ? (hi - lo + ROUND - 1) / ROUND : 0;
  int sent = 0;             // (thread 0)
  auto fetch = [&](int i) {  // by one thread: slots lo + i ROUND ..
    if (i >= rounds) return;
    const uint32_t st = sm + i % STAGES * STAGE, full = bar + 8 * (i % STAGES);
    mbar_arrive_expect_tx(full, STAGE);
    tma_load_5d(st, &maps.v, full, 0, 0, kv, lo + i * ROUND, page);
    tma_load_4d(st + Sh::KEYS, &maps.k, full, 0, kv, lo + i * ROUND, page);
    sent = i + 1;
  };
  if (tid == 0)
    for (int i = 0; i < STAGES; ++i) fetch(i);
  auto first_slot = [&](int i) { return lo + i * ROUND + w * SB; };
  const signed char* pe = a.cache.exps + ((long long)page * KV + kv) * seen.slots * 2;
  const int skew = (int)(reinterpret_cast<uintptr_t>(pe) & 2);
  auto fetch_exps = [&](int i) {  // of the warp's slots of round i
    // exponents, two bytes a slot, in words: where the row starts in the middle of one, from there
    const int s0 = first_slot(i);
    if (i < rounds && s0 < hi && lane <= SB / 2) {
      const long long from = 2ll * s0 - skew + 4 * lane;  // byte of the row
      if (from < 2ll * hi)
        copy4(smem_u32(sh.exps[w][i % STAGES]) + 4 * lane, pe + from,
              (int)min(2ll * hi - from, 4ll));
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch_exps(i);

  // ---- queries: step 2 j + h of the product has channels 32 j + 8 t + 4 h .. + 3 of thread t of a row's
  // four.  Each group of eight rows by a warp: scaled into fp16's range by a power of two per row, in the order
  // of the codes' operands (channels 0, 2 and 1, 3 of four).
  const int g = lane >> 2, t = lane & 3, t2 = t * 2;
  auto row_of = [&](int r) { return grp * HB + min(r, rows - 1); };  // (the last one again behind them)
  auto load_q = [&](int n, uint32_t (&qf)[kDK / 16][2]) {
    const int R = row_of(8 * n + g), i = R / G;
    const T* q = static_cast<const T*>(a.q) + ((long long)(s.first + i) * a.H + kv * G + R - i * G) * kDK;
#pragma unroll
    for (int j = 0; j < kDK / 16; ++j) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(q + 32 * (j >> 1) + 8 * t + 4 * (j & 1)));
      qf[j][0] = x.x;
      qf[j][1] = x.y;
    }
  };
  static_assert(NT <= WARPS, "a warp for each group of rows");
  if (w < NT) {
    uint32_t qf[kDK / 16][2];
    load_q(w, qf);
    float up = 16777216.f * kLog2e;
    if constexpr (!__is_same(T, __half)) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j) top = top2<T>(top, top2<T>(qf[j][0], qf[j][1]));
      top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = top2<T>(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float2 f = halves<T>(top);
      // from 2^-126, since a query loses bits where it stays below fp16's 2^-14, to 2^100, since 2^24 log2(e) 2^e has to
      // be finite: rows of up to 2^115 stay within fp16
      const int e = min(max((int)(__float_as_uint(fmaxf(f.x, f.y)) >> 23) - 127, -126), 100);
      const float down = pow2(-e);
      up *= pow2(e);
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 x = halves<T>(qf[j][h]);
          qf[j][h] = pack2<__half>(x.x * down, x.y * down);
        }
    }
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t zero[4] = {kZero16, kZero16, kZero16, kZero16};
#pragma unroll
    for (int j = 0; j < kDK / 16; ++j) {
      const uint2 y = make_uint2(__byte_perm(qf[j][0], qf[j][1], 0x5410), __byte_perm(qf[j][0], qf[j][1], 0x7632));
      sh.q[w][j][lane] = y;
      mma16816<__half>(x, zero, y.x, y.y);
    }
    if (g == 0) *reinterpret_cast<float2*>(sh.z0 + 8 * w + t2) = make_float2(-x[0], -x[1]);
    if (t == 0) sh.zs[8 * w + g] = up;
  }
  const T* nk = static_cast<const T*>(a.k) + ((long long)s.first * KV + kv) * kDK;
  const T* nv = static_cast<const T*>(a.v) + ((long long)s.first * KV + kv) * kDV;
  // One token alone: its score by the last warp, and its values' channels of this thread (16 (TILES w + j) + 2 g, +
  // 1), ahead of the page.  (Behind it, as those of more are, they took 3,300 of a unit's 48,000 cycles; more than
  // one group of rows has no registers for it.)
  const bool one = NT == 1 && part == 0 && i1 == 0;
  [[maybe_unused]] uint32_t own[TILES];
  if constexpr (NT == 1) {
    if (one) {
#pragma unroll
      for (int j = 0; j < TILES; ++j)
        own[j] = __ldg(reinterpret_cast<const uint32_t*>(nv + 16 * (TILES * w + j) + 2 * g));
      if (w == WARPS - 1) {
        uint32_t qf[kDK / 16][2];
        load_q(0, qf);
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < kDK / 16; ++j) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(nk + 32 * (j >> 1) + 8 * t + 4 * (j & 1)));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 u = halves<T>(qf[j][h]), v = halves<T>(h ? x.y : x.x);
            z = fmaf(u.x, v.x, fmaf(u.y, v.y, z));
          }
        }
        z += __shfl_xor_sync(0xffffffffu, z, 1);
        z += __shfl_xor_sync(0xffffffffu, z, 2);
        if (t == 0) sh.top[0][g] = z * kLog2e;
      }
    }
  }
  __syncthreads();

  // A thread's scores are of slots g, g + 8, .. of the warp's and rows 8 n + t2, + 1 (NR of them); its sums of
  // channels 16 (TILES w + c) + 2 g (0, 1) and + 1 (2, 3) and the same rows.
  float z0[NR], zs[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    z0[r] = sh.z0[8 * (r >> 1) + t2 + (r & 1)];
    zs[r] = sh.zs[8 * (r >> 1) + t2 + (r & 1)];
  }
  // (read by all ahead of the first round's barrier, behind which `refer` writes there; without rounds, for one token,
  // nothing does)
  [[maybe_unused]] const float z_own[2] = {sh.top[0][t2], sh.top[0][t2 + 1]};
  auto at = [&](int r) { return s.pos + row_of(8 * (r >> 1) + t2 + (r & 1)) / G; };  // a row's position
  float acc[TILES][NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < TILES; ++j) acc[j][n][k] = 0.f;
  float m[NR], l[NR];  // base 2, the same in all warps; l of this thread's slots
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
  int e_ref = -1000;  // acc is in units of 2^e_ref; -60 at least: what is below 2^-78 in a page is lost

  // The rare round in which a score passes a row's maximum by more than 8, or an exponent e_ref by more than 4
  // (weights of up to 2^12 lose nothing in fp16): new ones for all, and the sums in their units.
  auto refer = [&](float (&top)[NR], int e_top) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
      if (g == 0) sh.top[w][8 * (r >> 1) + t2 + (r & 1)] = top[r];
    }
    if (lane == 0) sh.e_top[w] = e_top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WARPS; ++k) e_top = max(e_top, sh.e_top[k]);
    const float f = e_top > e_ref + 4 ? pow2(max(e_ref - e_top, -126)) : 1.f;
    if (e_top > e_ref + 4) e_ref = e_top;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float all = -INFINITY;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) all = fmaxf(all, sh.top[k][8 * (r >> 1) + t2 + (r & 1)]);
      const float now = all > m[r] + 8.f ? all : m[r];
      const float keep = now == m[r] || m[r] == -INFINITY ? 1.f : ex2(m[r] - now);
      m[r] = now;
      l[r] *= keep;
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        acc[j][r >> 1][r & 1] *= keep * f;
        acc[j][r >> 1][2 + (r & 1)] *= keep * f;
      }
    }
  };

  // ---- the page
  // where the lane's 16 bytes of a transposed load lie: slot `lane` of 32, the warp's channels, swizzled by the
  // address
  uint32_t v_at[TILES];
#pragma unroll
  for (int j = 0; j < TILES; ++j) {
    const int x = lane * kDV + 16 * (TILES * w + j);
    v_at[j] = sm + (x ^ ((x >> 3) & 48));
  }
  // a lane's row of the weights: of the stores (in the warp's slice) and of the loads (32 slots)
  const uint32_t p_to = sm + Sh::KEYS + w * Sh::SLICE + (lane & 7) * P_ROW + (lane >> 3) % (SB / 8) * 16;
  const uint32_t p_from = sm + Sh::KEYS + (lane & 7) * P_ROW +
                          (SB == 32 ? (lane >> 3) * 16 : (lane >> 4) * Sh::SLICE + ((lane >> 3) & 1) * 16);
  bool dead = false;  // a wait ran out: no more loads, and nothing of use comes out
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    const int s0 = first_slot(i);
    if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(bar + 8 * (i % STAGES), (i / STAGES) & 1, ctl));
    if (i == ctl.stall_step && w == 0)  // the give-up path's diagnostic (see chunk_fwd.cu)
      dead = !__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.behind), 0, ctl));
    copy_wait<STAGES - 1>();
    __syncwarp();
    float z[SB / 16][NT][4];  // slots 16 h + g, + 8
    float f[SB / 8];          // the factors of the thread's slots, 8 k + g: of keys,
    uint32_t fv[SB / 8];      // of values, twice
    int ev = -128;
    float ks = 0.f;
    bool up = false;
    if (s0 < hi) {
      const uint8_t* keys = smem + i % STAGES * STAGE + Sh::KEYS + w * Sh::SLICE;
#pragma unroll
      for (int h = 0; h < SB / 16; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[h][n][k] = z0[2 * n + (k & 1)];
#pragma unroll
      for (int j = 0; j < kDK / 32; ++j) {
        uint2 q[2][NT];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) q[k][n] = sh.q[n][2 * j + k][lane];
#pragma unroll
        for (int h = 0; h < SB / 16; ++h) {
          const uint2 x = *reinterpret_cast<const uint2*>(keys + (16 * h + g) * kDK + 32 * j + 8 * t);
          const uint2 y = *reinterpret_cast<const uint2*>(keys + (16 * h + 8 + g) * kDK + 32 * j + 8 * t);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t x4[4];
            whole16(k ? x.y : x.x, x4[0], x4[2]);
            whole16(k ? y.y : y.x, x4[1], x4[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<__half>(z[h][n], x4, q[k][n].x, q[k][n].y);
          }
        }
      }
      // factors of slot `lane`, and from there of this thread's.  (The first row sees what any does.  A slot
      // that none sees may be written meanwhile.)
      const bool all = whole(s0);
      const char2 ex = reinterpret_cast<const char2*>(sh.exps[w][i % STAGES] + skew)[lane & (SB - 1)];
      ev = (signed char)ex.y;
      const uint32_t there = bits_to(min(hi - s0, SB) - 1);
      if (!all && !(((seen.bits(s.pos + i0, s0) & there) >> (lane & (SB - 1))) & 1)) ev = -128;
      ks = scale_of((signed char)ex.x);
#pragma unroll
      for (int k = 0; k < SB / 8; ++k) f[k] = __shfl_sync(0xffffffffu, ks, 8 * k + g);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int k = 0; k < SB / 8; ++k) {
          float& x = z[k >> 1][r >> 1][2 * (k & 1) + (r & 1)];
          x = x * zs[r] * f[k];
        }
      if (!all) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const uint32_t see = (seen.bits(at(r), s0) & there) >> g;
#pragma unroll
          for (int k = 0; k < SB / 8; ++k)
            if (!((see >> (8 * k)) & 1)) z[k >> 1][r >> 1][2 * (k & 1) + (r & 1)] = -INFINITY;
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < SB / 16; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[h][n][k] = -INFINITY;
    }
    __syncwarp();
    fetch_exps(i + STAGES);
    const int e_top = max(__reduce_max_sync(0xffffffffu, ev), -60);
    float top[NR], part_sum[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      top[r] = -INFINITY;
#pragma unroll
      for (int k = 0; k < SB / 8; ++k) top[r] = fmaxf(top[r], z[k >> 1][r >> 1][2 * (k & 1) + (r & 1)]);
      up |= top[r] > m[r] + 8.f;
    }
    up |= e_top > e_ref + 4;
    auto weigh = [&] {
      const __half2 vs = __float2half2_rn(pow2(min(max(ev - e_ref, -126), 8)));
#pragma unroll
      for (int k = 0; k < SB / 8; ++k)
        fv[k] = __shfl_sync(0xffffffffu, reinterpret_cast<const uint32_t&>(vs), 8 * k + g);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float base[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          base[j] = m[2 * n + j] == -INFINITY ? 0.f : m[2 * n + j];
          part_sum[2 * n + j] = 0.f;
        }
        uint32_t pf[SB / 8];
#pragma unroll
        for (int k = 0; k < SB / 8; ++k) {
          // the sum is of the rounded weights: where one outweighs the others, its rounding cancels
          pf[k] = pack2<__half>(ex2(z[k >> 1][n][2 * (k & 1)] - base[0]), ex2(z[k >> 1][n][2 * (k & 1) + 1] - base[1]));
          const float2 p = halves<__half>(pf[k]);
          part_sum[2 * n] += p.x;
          part_sum[2 * n + 1] += p.y;
          const __half2 y = __hmul2(reinterpret_cast<const __half2&>(pf[k]), reinterpret_cast<const __half2&>(fv[k]));
          pf[k] = reinterpret_cast<const uint32_t&>(y);
        }
        const uint32_t to = p_to + i % STAGES * STAGE + n * (8 * P_ROW);
        if constexpr (SB == 32) stsm4t(to, pf);
        else stsm2t(to, pf[0], pf[1]);
      }
    };
    weigh();
    const bool again = __syncthreads_or(up);
    // all warps are done with the round before
    if (tid == 0 && i > 0 && !dead) {
      fence_proxy_async();
      fetch(i - 1 + STAGES);
    }
    if (again) {
      refer(top, e_top);
      weigh();
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] += part_sum[r];
    // codes of slots 2 t, + 1 (x[0]) and + 8, + 9 (x[1]) of the first 16 of 32, x[2], x[3]: of the others
    const uint32_t st = i % STAGES * STAGE, p_at = p_from + st;
    const int left = hi - (lo + i * ROUND);
#pragma unroll
    for (int y = 0; y < ROUND / 32; ++y) {
      if (32 * y >= left) break;
      uint32_t pf[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) ldsm4(pf[n], p_at + n * (8 * P_ROW) + y * (32 / SB) * Sh::SLICE);
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        uint32_t x[4];
        ldsm4t(x, v_at[j] + st + y * (32 * kDV));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x4[4];
          whole_of<__half, true>(x[2 * h], x4[0], x4[1]);
          whole_of<__half, true>(x[2 * h + 1], x4[2], x4[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<__half>(acc[j][n], x4, pf[n][2 * h], pf[n][2 * h + 1]);
        }
      }
    }
  }
  copy_wait<0>();
  if (tid == 0) mbar_arrive(smem_u32(&sh.behind));
  {
    const float unit_of = pow2(min(max(e_ref, -126), 127));
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][n][k] *= unit_of;
  }

  // ---- the new tokens, 16 a warp
  // (their weights where the rounds were, which all warps have left when they have met)
  constexpr int F_ROW = 32 * WARPS + 16;
  if constexpr (NT == 1) {
    if (one) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float now = z_own[r] > m[r] + 8.f ? z_own[r] : m[r];
        const float keep = now == m[r] || m[r] == -INFINITY ? 1.f : ex2(m[r] - now), p = ex2(z_own[r] - now);
        m[r] = now;
        l[r] = l[r] * keep + (w == 0 && g == 0 ? p : 0.f);
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          const float2 v = halves<T>(own[j]);
          acc[j][0][r] = fmaf(p, v.x, acc[j][0][r] * keep);
          acc[j][0][2 + r] = fmaf(p, v.y, acc[j][0][2 + r] * keep);
        }
      }
    }
  }
  if (part == 0 && !one) {
    const int sinks = max(c.sink - s.pos, 0);
#pragma unroll 1
    for (int j0 = 0; j0 <= i1; j0 += 16 * WARPS) {
      if (j0 + 16 * WARPS - 1 <= i0 - c.window && j0 >= sinks) continue;
      const int mine = j0 + 16 * w;
      float z[NT][4], top[NR], part_sum[NR];
      bool up = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) top[r] = -INFINITY;
      if (mine <= i1) {
        uint32_t key[kDK / 16][4];
        const bool in0 = mine + g <= i1, in1 = mine + g + 8 <= i1;
        const T* from = nk + (long long)(mine + g) * KV * kDK + 8 * t;
#pragma unroll
        for (int j = 0; j < kDK / 16; ++j) {
          uint2 x = make_uint2(0u, 0u), y = x;
          if (in0) x = __ldg(reinterpret_cast<const uint2*>(from + 32 * (j >> 1) + 4 * (j & 1)));
          if (in1)
            y = __ldg(reinterpret_cast<const uint2*>(from + 8ll * KV * kDK + 32 * (j >> 1) + 4 * (j & 1)));
          key[j][0] = x.x, key[j][1] = y.x, key[j][2] = x.y, key[j][3] = y.y;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t qf[kDK / 16][2];
          load_q(n, qf);
#pragma unroll
          for (int k = 0; k < 4; ++k) z[n][k] = 0.f;
#pragma unroll
          for (int j = 0; j < kDK / 16; ++j) mma16816<T>(z[n], key[j], qf[j][0], qf[j][1]);
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const uint32_t see = mine <= i1 ? keys_seen(at(r) - s.pos, mine, i1 + 1, c.window, sinks) >> g : 0u;
        float &x = z[r >> 1][r & 1], &y = z[r >> 1][2 + (r & 1)];
        x = see & 1 ? x * kLog2e : -INFINITY;
        y = (see >> 8) & 1 ? y * kLog2e : -INFINITY;
        top[r] = fmaxf(x, y);
        up |= top[r] > m[r] + 8.f;
      }
      auto weigh = [&] {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float base = m[2 * n + j] == -INFINITY ? 0.f : m[2 * n + j];
            z[n][j] = ex2(z[n][j] - base);
            z[n][2 + j] = ex2(z[n][2 + j] - base);
          }
          const uint32_t lo = pack2<T>(z[n][0], z[n][1]), hi = pack2<T>(z[n][2], z[n][3]);
          const float2 x = halves<T>(lo), y = halves<T>(hi);
          part_sum[2 * n] = x.x + y.x;
          part_sum[2 * n + 1] = x.y + y.y;
          stsm2t(sm + (8 * n + (lane & 7)) * F_ROW + (16 * w + ((lane >> 3) & 1) * 8) * 2, lo, hi);
        }
      };
      if (__syncthreads_or(up)) refer(top, -1000);
      weigh();
      __syncthreads();
#pragma unroll
      for (int r = 0; r < NR; ++r) l[r] += part_sum[r];
#pragma unroll 1
      for (int y = 0; y < WARPS && j0 + 16 * y <= i1; ++y) {
        // channels 2 g, + 1 of 16 and tokens t2, + 1 and + 8, + 9
        const int tok = j0 + 16 * y + t2;
        const T* val = nv + (long long)tok * KV * kDV + 16 * TILES * w + 2 * g;
        uint32_t x[TILES][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int d = (k & 1) + 8 * (k >> 1);
#pragma unroll
          for (int j = 0; j < TILES; ++j) {
            x[j][k] = 0u;
            if (tok + d <= i1)
              x[j][k] = __ldg(reinterpret_cast<const uint32_t*>(val + (long long)d * KV * kDV + 16 * j));
          }
        }
        const uint8_t* weights = smem + g * F_ROW + (16 * y + t2) * 2;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t p0 = *reinterpret_cast<const uint32_t*>(weights + n * (8 * F_ROW));
          const uint32_t p1 = *reinterpret_cast<const uint32_t*>(weights + n * (8 * F_ROW) + 16);
#pragma unroll
          for (int j = 0; j < TILES; ++j) {
            const uint32_t x4[4] = {__byte_perm(x[j][0], x[j][1], 0x5410), __byte_perm(x[j][0], x[j][1], 0x7632),
                                    __byte_perm(x[j][2], x[j][3], 0x5410), __byte_perm(x[j][2], x[j][3], 0x7632)};
            mma16816<T>(acc[j][n], x4, p0, p1);
          }
        }
      }
    }
  }

  // ---- the rows' sums of all warps, and the outputs
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
    if (g == 0) sh.sum[w][8 * (r >> 1) + t2 + (r & 1)] = l[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = 8 * (r >> 1) + t2 + (r & 1), ch = 16 * TILES * w + 2 * g;
    if (row >= rows) continue;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) sum += sh.sum[k][row];
    if (parts == 1) {
      const int R = grp * HB + row, i = R / G;
      const float inv = 1.f / sum;  // the token itself is there: sum > 0
      TO* o = static_cast<TO*>(a.o) + ((long long)(s.first + i) * a.H + kv * G + R - i * G) * kDV + ch;
#pragma unroll
      for (int j = 0; j < TILES; ++j)
        store2(o + 16 * j, acc[j][r >> 1][r & 1] * inv, acc[j][r >> 1][2 + (r & 1)] * inv);
    } else {
      const long long cuts = plan.units - plan.whole;
      float* pw = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + table_bytes(cuts)) +
                  (((long long)(unit - plan.whole) * HB + row) * parts + part) * (kDV + 2);
#pragma unroll
      for (int j = 0; j < TILES; ++j)
        *reinterpret_cast<float2*>(pw + ch + 16 * j) =
            make_float2(acc[j][r >> 1][r & 1], acc[j][r >> 1][2 + (r & 1)]);
      if (w == 0 && g == 0) *reinterpret_cast<float2*>(pw + kDV) = make_float2(m[r], sum);
    }
  }
  if (part == 0) {
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
  if (dead && tid == 0)  // the loads on their way land before the CTA may exit
    for (int i = max(sent - STAGES, 0); i < sent; ++i) mbar_wait(bar + 8 * (i % STAGES), (i / STAGES) & 1, ctl, DRAIN_NS);
}

// One block per row of a cut unit.
template <class TO>
__global__ void __launch_bounds__(JOIN_THREADS)
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
  const int KV = a.cache.c.KV, G = a.H / KV, R = u.row0 + row, i = R / G;
  join_row(
      parts, [&](int p) { return *reinterpret_cast<const float2*>(pw + p * (kDV + 2) + kDV); },
      [&](int p) { return pw + p * (kDV + 2); },
      static_cast<TO*>(a.o) + ((long long)(u.first + i) * a.H + u.kv * G + R - i * G) * kDV);
}

// `units` at most, `likely` so many: as many whole ones as fill the device one or more times, and the others in
// as many parts as fill it once more, of at least one round.  (More parts than that, in two turns: 69 us in place of
// 58 with 64 chunks of four tokens on 2,052 slots, 256 units on 456 places.)
inline Plan make_plan(long long units, long long likely, int rows, int slots, int n_sm) {
  // a unit takes three quarters of the time by rounds of 128 slots (16 rows; two thirds with more), two to an SM
  const long long two = (likely + 2 * n_sm - 1) / std::max(2 * n_sm, 1), three = (likely + 3 * n_sm - 1) / std::max(3 * n_sm, 1);
  const bool wide = rows == 8 || (rows == 16 ? 3 * two <= 4 * three : 2 * two <= 3 * three);
  const int ROUND = wide ? Shape<1, true>::ROUND : Shape<2, false>::ROUND;
  static_assert(Shape<1, true>::ROUND == Shape<2, true>::ROUND && Shape<1, true>::ROUND == Shape<4, true>::ROUND &&
                    Shape<2, false>::ROUND == Shape<4, false>::ROUND,
                "rounds");
  const int hold = std::max((rows > 8 && wide ? 2 : 3) * n_sm, 1), rest = (int)(likely % hold);
  const int most = std::min((slots - 1) / ROUND + 1, kMostParts);
  // (where many more units may come than are likely, each of those has room for as many parts)
  const long long room = std::max(4ll * hold / std::max(units - (likely - rest), 1ll), 1ll);
  const int cut = rest ? (int)std::min<long long>(std::min(hold / rest, most), room) : 1;
  if (cut < 2) return Plan{units, (int)units, 1, 0, rows, wide};
  const int part_slots = ((slots + cut - 1) / cut + ROUND - 1) / ROUND * ROUND;
  const int parts = (slots + part_slots - 1) / part_slots;
  if (parts < 2) return Plan{units, (int)units, 1, 0, rows, wide};
  return Plan{units, (int)(likely - rest), parts, part_slots, rows, wide};
}

template <int ROUND>
bool make_maps(Maps* m, const ServeCache& cache) {
  auto fn = encode_tiled_fn();
  if (!fn) return false;
  const WindowCache& c = cache.c;
  const cuuint64_t slots = c.window + c.sink, pages = (cuuint64_t)((long long)c.n_pages * c.pool_layers);
  const cuuint64_t KV = c.KV, k_dims[4] = {kDK, KV, slots, pages};
  const cuuint64_t k_strides[3] = {kDK, kDK * KV, kDK * KV * slots};
  const cuuint64_t v_dims[5] = {64, kDV / 64, KV, slots, pages};
  const cuuint64_t v_strides[4] = {64, kDV, kDV * KV, kDV * KV * slots};
  const cuuint32_t k_box[4] = {kDK, 1, ROUND, 1}, v_box[5] = {64, kDV / 64, 1, ROUND, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn(&m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.k, k_dims, k_strides, k_box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         fn(&m->v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, c.v, v_dims, v_strides, v_box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, class TO, int NT, bool WIDE>
cudaError_t run(const Args& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  Maps m;
  if (!make_maps<Shape<NT, WIDE>::ROUND>(&m, a.cache)) return cudaErrorInvalidValue;
  auto kern = rows8_kernel<T, TO, NT, WIDE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NT, WIDE>());
  if (e != cudaSuccess) return e;
  const long long cut = plan.units - plan.whole;
  kern<<<(unsigned)(plan.whole + cut * plan.parts), THREADS, smem_bytes<NT, WIDE>(), stream>>>(m, a, plan, ctl);
  if ((e = cudaGetLastError()) != cudaSuccess || plan.parts == 1) return e;
  PdlLaunch l(dim3((unsigned)(cut * plan.rows)), dim3(JOIN_THREADS), 0, stream, true);
  return cudaLaunchKernelEx(&l.cfg, rows8_join_kernel<TO>, a, plan);
}

template <class T, class TO>
cudaError_t run(const Args& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  if (plan.rows == 8) return run<T, TO, 1, true>(a, plan, ctl, stream);
  if (plan.rows == 24)
    return plan.wide ? run<T, TO, 3, true>(a, plan, ctl, stream) : run<T, TO, 3, false>(a, plan, ctl, stream);
  if (plan.rows == 32)
    return plan.wide ? run<T, TO, 4, true>(a, plan, ctl, stream) : run<T, TO, 4, false>(a, plan, ctl, stream);
  return plan.wide ? run<T, TO, 2, true>(a, plan, ctl, stream) : run<T, TO, 2, false>(a, plan, ctl, stream);
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
