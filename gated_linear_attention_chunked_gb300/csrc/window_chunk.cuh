// window_chunk.cuh -- the windowed attention (window_fwd.cu) of new tokens over the pages of their
// sequences: token t of a sequence, t = pos + i, sees its page's tokens below pos and the call's own
// from pos to t, of these the last `window` and the first `sink`.  Instantiated for pages of 16 bits
// (window_chunk.cu) and of 8 (window_chunk8.cu).
//
// The roles are window_fwd.cu's (softmax in two groups of four warps that take the key tiles in turn, TMA
// of keys, of values, the tcgen05 issuer, output rows), with its scores two tiles ahead and its rare
// rescaling.  What differs:
//   rows     an item is 128 / G tokens of one sequence with all G query heads of a key head, row = (token,
//            head): keys are read once for the G heads, and a chunk of few tokens still fills rows.  Warps
//            whose rows are all empty only keep step.
//   keys     first the tiles of the page, 128 slots each, then those of the call's own tokens.  A page is
//            read in the order of its slots: what a row sees of it are three runs of slots (the sinks, and the
//            ring in front of and behind its newest token), so a mask is three runs of bits and no key has to
//            be put in order.  Tiles that the item's first row does not see are passed over.
//   items    every CTA finds its own from the sequences' lengths on the device: sums of tiles over
//            slices of the sequences, one slice a thread, then a search for each item, which are put down in
//            shared memory before the roles start.
//   parts    where the items do not fill the device, each one's tiles are cut into parts that leave
//            (o, reference, sum) in fp32 in the workspace, joined in order by a second kernel.
//   codes    come by TMA as they are, and the output warps, idle while an item is walked, turn them into
//            the swizzled 16-bit operands, c 2^e exactly.  They do so for the next item's first two tiles before they take the
//            output rows, so that the scores stay two tiles ahead across items.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "tmap.h"
#include "window_join.cuh"
#include "window_packed.cuh"
#include "window_wait.cuh"

namespace gla {
namespace chunk {

using scan::Cta;
using scan::DRAIN_NS;

constexpr int BM = 128, BN = 128;
constexpr uint32_t K_BOX = 8192, V_BOX = 16384;  // 128 rows x 64 B, x 128 B
constexpr uint32_t K_BYTES = 3 * K_BOX, V_BYTES = 3 * V_BOX;
constexpr int LIST = 48;                         // items of a CTA

// Tokens of one sequence with the query heads of a key head, and the key tiles of one part of them: tile
// i of an item is tile i + d of the page (128 slots each) or of the sequence's new tokens, d by where i
// lies: page tiles below n0, n1 and n2 in the three runs of slots that are seen, then new tokens below nf
// that hold sinks, then the window's.
struct alignas(16) Item {
  int n0, n1, n2, nf;
  int d1, d2, d3, d4;
  int w[8];                       // whole tiles, which every row sees: w[0] .. w[1]-1, w[2] .., w[4] .., w[6] ..
  int row0, i0, n_tok, tokens;    // first packed row; its index and count in the sequence's new tokens
  int pos, page, kv, sink;        // page and layer
  int tb, te;                     // tiles tb .. te-1 are this part's
  int ns, a_lo, a_hi, b_lo, base; // slots seen: 0 .. ns-1, a_lo .. a_hi-1, b_lo .. (all for the first row);
                                  // slot sink + r of the first ring run holds token base + r
  int slots;
};
static_assert(sizeof(Item) == 128, "whole 16-byte accesses");

// As in window_fwd.cu.  RAW, RAW + 1: a tile's codes of keys, of values have come; RAW_FREE: they have been
// read.  K_CODES, V_CODES: they have been turned into operands; the loaders and the output warps arrive
// there for every tile, also for one that asks nothing of them, so that none falls two phases behind a
// barrier that it waits for, which its parity would not show.
enum Bar : uint32_t {
  Q_FULL = 0, K_FULL = 2, V_FULL = 4, S_FULL = 6, O_DONE = 8, P_READY = 10, O_FREE = 12, DRAIN = 13,
  REF = 14, SUM = 22, RAW = 26, RAW_FREE = 28, K_CODES = 30, V_CODES = 32, NBAR = 34
};
constexpr uint32_t RAW_K = BN * kDK, RAW_V = BN * kDV;
// Shared memory.  With codes, whose raw tiles take room, there is one buffer of queries (the next item's come
// when the scores of the one before are done, ahead of its last products), and output rows are staged in
// half the width.
template <bool CODES>
struct Layout {
  static constexpr uint32_t QS = CODES ? 1 : 2;            // buffers of queries
  static constexpr uint32_t STG_ROW = CODES ? 64 : 128;    // bytes of a staged row
  static constexpr uint32_t Q = 0, K = QS * K_BYTES, V = K + 2 * K_BYTES;
  static constexpr uint32_t RAWS = V + 2 * V_BYTES;        // codes of keys, of values
  static constexpr uint32_t STG = RAWS + (CODES ? RAW_K + RAW_V : 0);  // 32 rows per output warp
  static constexpr uint32_t REFS = STG + 4 * 32 * STG_ROW; // float ref[2][128]: each group's reference
  static constexpr uint32_t SUMS = REFS + 1024;            // float2 sum[2][2][128]: (sum, ref), by item
  static constexpr uint32_t ITEM = SUMS + 4096;
  static constexpr uint32_t BAR = ITEM + LIST * sizeof(Item);
  static constexpr uint32_t TMEM = BAR + NBAR * 8;
  static constexpr uint32_t COUNT = TMEM + 4;              // items, their tiles
  static constexpr uint32_t INFO = COUNT + 8;              // uint32 [4]: tiles for the issuer (TileInfo)
  static constexpr uint32_t PLACE = INFO + 16;             // uint32 [LIST]: items' first rows in the workspace
  static constexpr uint32_t ABORT = PLACE + 4 * LIST;
  static constexpr uint32_t USED = ABORT + 4 * kWaitWords, BYTES = USED + 1024;
  static_assert(BYTES <= 232448, "shared memory budget");
  static_assert(BAR % 8 == 0 && STG % 512 == 0 && RAWS % 128 == 0, "alignment");
};

// Columns: S twice 128, O 192.  A tile's P takes the place of its S, from the front.
constexpr uint32_t TM_S = 0, TM_O = 256;

constexpr int GROUP = 128, K_WARP = 8, V_WARP = 9, MMA_WARP = 10, OUT_WARP = 11;
constexpr int THREADS = 15 * 32;

struct Plan {
  int per;        // tokens of an item
  int parts;
  long long units;  // (tile, key head) at most
  unsigned grid;
  // The workspace of cut items: the tiles' rows and tokens, and by part, key head and row (token, query head)
  // (reference, sum) and o: an item's rows lie together, and take no more room than there are.  Its bytes, and where
  // ml and o begin:
  size_t bytes, ml, o;
};
struct Partials {
  int* tiles;   // [0]: how many; [2 + 2 i], [3 + 2 i]: row0, n_tok
  float2* ml;   // [parts][KV][n_tokens][G]
  float* o;     // [parts][KV][n_tokens][G][192]
  __device__ __forceinline__ Partials(void* p, const Plan& plan)
      : tiles(static_cast<int*>(p)), ml(reinterpret_cast<float2*>(static_cast<char*>(p) + plan.ml)),
        o(reinterpret_cast<float*>(static_cast<char*>(p) + plan.o)) {}
};

__device__ __forceinline__ int ceil_tiles(int n) { return n <= 0 ? 0 : (n - 1) / BN + 1; }

// Item of tokens i0 .. of a sequence, part `part` of `parts`.
static __device__ __noinline__ void make_item(Item& it, const WindowCache& c, const Sequence& s, int per, int i0,
                                       int kv, int part, int parts) {
  it.i0 = i0;
  it.n_tok = min(per, s.tokens - i0);
  it.row0 = s.first + i0;
  it.tokens = s.tokens;
  it.pos = s.pos;
  it.page = s.page * c.pool_layers + c.layer;
  it.kv = kv;
  it.sink = c.sink;
  it.slots = c.window + c.sink;
  const int slots = it.slots, p0 = s.pos + i0, i1 = i0 + it.n_tok;
  const int ns = min(c.sink, s.pos);
  int a_lo = 0, a_hi = 0, b_lo = slots, base = 0;
  int a_all = 0, b_all = slots;   // from where the last row sees
  if (s.pos > c.sink) {
    const int last = s.pos - 1 - c.sink, lr = last % c.window;
    base = s.pos - 1 - lr;
    const int x = p0 - base - c.window + 1, y = x + it.n_tok - 1;  // ring place of the oldest token seen
    a_hi = c.sink + lr + 1;
    a_lo = min(c.sink + max(0, x), a_hi);
    a_all = min(c.sink + max(0, y), a_hi);
    // behind the newest token are those of the round before, if there was one
    if (base > c.sink) {
      b_lo = min(max(a_hi, c.sink + x + c.window), slots);
      b_all = min(max(a_hi, c.sink + y + c.window), slots);
    }
  }
  const int n0 = ceil_tiles(ns);
  const int l1 = max(a_lo / BN, n0), h1 = a_lo < a_hi ? max(ceil_tiles(a_hi), l1) : l1;
  const int l2 = max(b_lo / BN, h1), h2 = b_lo < slots ? max(ceil_tiles(slots), l2) : l2;
  const int sinks = max(c.sink - s.pos, 0);  // of the new tokens
  const KeyTiles kt(i0, i1, BN, c.window, sinks);
  it.n0 = n0;
  it.n1 = n0 + h1 - l1;
  it.n2 = it.n1 + h2 - l2;
  it.nf = it.n2 + kt.far;
  it.d1 = l1 - n0;
  it.d2 = l2 - it.n1;
  it.d3 = -it.n2;
  it.d4 = kt.lo - it.nf;
  it.ns = ns;
  it.a_lo = a_lo;
  it.a_hi = a_hi;
  it.b_lo = b_lo;
  it.base = base;
  // slots that all rows see: 0 .. ns-1, a_all .. a_hi-1, b_all .., joined where they meet
  const int s_end = a_all > ns ? ns : b_all > a_hi ? max(a_hi, ns) : slots;
  const int a_end = b_all > a_hi ? a_hi : slots, a_from = a_all > ns ? a_all : 0;
  it.w[0] = 0;
  it.w[1] = min(s_end / BN, n0);
  it.w[2] = n0 + max((a_from + BN - 1) / BN, l1) - l1;
  it.w[3] = n0 + min(a_end / BN, h1) - l1;
  it.w[4] = it.n1 + max(((b_all > a_hi ? b_all : a_from) + BN - 1) / BN, l2) - l2;
  it.w[5] = it.n1 + min(slots / BN, h2) - l2;
  // new tokens: of tiles before the first row, those inside the last row's window
  const int in = max(i1 - c.window, 0), w_lo = max((in + BN - 1) / BN, kt.lo);
  it.w[6] = it.nf + w_lo - kt.lo;
  it.w[7] = it.nf + (i0 + 1) / BN - kt.lo;
  const long long n = it.n2 + kt.n;
  it.tb = (int)(n * part / parts);
  it.te = (int)(n * (part + 1) / parts);
}

// What the roles ask of an item's tiles.  With codes, out of line (Ask<true>): every role asks, and with the
// conversion of codes their code no longer shares the instruction cache (192 us inlined, 159 not); without,
// inlined (Ask<false>: 103 us, 110 not).
struct Tile {
  int s0;         // first slot, or first of the sequence's new tokens
  unsigned bits;
  __device__ __forceinline__ bool fresh() const { return bits & 1; }  // of the new tokens
  __device__ __forceinline__ bool whole() const { return bits & 2; }  // all rows see all its columns
};
__device__ __forceinline__ Tile tile_inline(const Item& it, int i) {
  const int4 n = *reinterpret_cast<const int4*>(&it.n0), d = *reinterpret_cast<const int4*>(&it.d1);
  const int4 u = *reinterpret_cast<const int4*>(it.w), v = *reinterpret_cast<const int4*>(it.w + 4);
  Tile t;
  t.s0 = BN * (i + (i < n.x ? 0 : i < n.y ? d.x : i < n.z ? d.y : i < n.w ? d.z : d.w));
  const bool whole = (i >= u.x && i < u.y) || (i >= u.z && i < u.w) || (i >= v.x && i < v.y) ||
                     (i >= v.z && i < v.w);
  t.bits = (i >= n.z ? 1 : 0) | (whole ? 2 : 0);
  return t;
}
// Columns of tile i that some row may see, rounded to 16.
__device__ __forceinline__ int cols_inline(const Item& it, Tile t, int i) {
  if (t.whole()) return BN;
  int end;
  if (t.fresh()) {
    end = it.i0 + it.n_tok;
    if (i < it.nf) end = min(it.sink - it.pos, end);
  } else {
    end = it.ns;
    if (it.a_lo < min(it.a_hi, t.s0 + BN)) end = max(end, it.a_hi);
    if (it.b_lo < min(it.slots, t.s0 + BN)) end = it.slots;
  }
  return min(BN, (end - t.s0 + 15) & ~15);
}
// The columns c0 .. c0 + 31 of a tile that token i of the sequence's new ones sees.
__device__ __forceinline__ uint32_t seen_inline(const Item& it, bool fresh, int i, int c0) {
  const int window = it.slots - it.sink;
  if (fresh) return keys_seen(i, c0, it.tokens, window, max(it.sink - it.pos, 0));
  const int x = it.pos - it.base + i - window + 1;
  return bits_to(it.ns - 1 - c0) | (bits_to(it.a_hi - 1 - c0) & ~bits_to(it.sink + max(0, x) - 1 - c0)) |
         (it.base > it.sink && it.a_hi > 0
              ? bits_to(it.slots - 1 - c0) & ~bits_to(max(it.a_hi, it.sink + x + window) - 1 - c0)
              : 0u);
}

static __device__ __noinline__ Tile tile_call(const Item& it, int i) { return tile_inline(it, i); }
static __device__ __noinline__ int cols_call(const Item& it, Tile t, int i) { return cols_inline(it, t, i); }
static __device__ __noinline__ uint32_t seen_call(const Item& it, bool fresh, int i, int c0) {
  return seen_inline(it, fresh, i, c0);
}
template <bool CALL>
struct Ask {
  static __device__ __forceinline__ Tile tile(const Item& it, int i) {
    return CALL ? tile_call(it, i) : tile_inline(it, i);
  }
  static __device__ __forceinline__ int cols(const Item& it, Tile t, int i) {
    return CALL ? cols_call(it, t, i) : cols_inline(it, t, i);
  }
  static __device__ __forceinline__ uint32_t seen(const Item& it, bool fresh, int i, int c0) {
    return CALL ? seen_call(it, fresh, i, c0) : seen_inline(it, fresh, i, c0);
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Parities of barriers that complete phases at a pace of their own, a bit each.
struct Parities {
  uint32_t bits = 0;
  // of the next phase of number i
  __device__ __forceinline__ uint32_t take(uint32_t i) {
    const uint32_t p = (bits >> i) & 1;
    bits ^= 1u << i;
    return p;
  }
};

// Eight codes as eight 16-bit values c 2^e, in one 16-byte chunk.
template <class T>
__device__ __forceinline__ uint4 values_of(uint32_t lo, uint32_t hi, float s) {
  uint4 o;
  if constexpr (__is_same(T, __half)) {
    whole_of<T, false>(lo, o.x, o.y);
    whole_of<T, false>(hi, o.z, o.w);
    o = make_uint4(scaled<T>(o.x, s), scaled<T>(o.y, s), scaled<T>(o.z, s), scaled<T>(o.w, s));
  } else {
    // 0x4B000000 | u is 2^23 + u, from which an addition takes 2^23 + 128; the upper half of c s is its bf16 value.
    // All exact.  (One operation, (2^23 + u) s - (2^23 + 128) s, overflows from s = 2^105, which large rows have; four
    // steps in bf16 arithmetic take a third longer than it.  96 x 32 tokens on 2,052 slots: 152 us, with the one 160; 37
    // on 65,552 slots: 3 us more than with it, of 90.)
    const float2 s2 = make_float2(s, s), off = make_float2(-8388736.f, -8388736.f);
    const uint32_t m = 0x4B000000u;
    uint32_t* w = &o.x;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t u = (j ? hi : lo) ^ 0x80808080u;
      const float2 x = mul2(add2(make_float2(__uint_as_float(__byte_perm(u, m, 0x7440)),
                                             __uint_as_float(__byte_perm(u, m, 0x7441))), off), s2);
      const float2 y = mul2(add2(make_float2(__uint_as_float(__byte_perm(u, m, 0x7442)),
                                             __uint_as_float(__byte_perm(u, m, 0x7443))), off), s2);
      w[2 * j] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
      w[2 * j + 1] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
    }
  }
  return o;
}

// The tiles of a CTA's items, one after the other.
struct Walk {
  int x, i;
  __device__ __forceinline__ void settle(const Item* items, int n) {
    while (x < n && i >= items[x].te)
      if (++x < n) i = items[x].tb;
  }
  __device__ __forceinline__ void begin(const Item* items, int n) {
    x = 0;
    i = n ? items[0].tb : 0;
    settle(items, n);
  }
  __device__ __forceinline__ void step(const Item* items, int n) {
    ++i;
    settle(items, n);
  }
};

// Rows 32 q4 .. + 31 of a raw tile of codes as operands, in pieces of 16 codes (two 16-byte chunks).  Two
// lanes take a key row's piece pairs, one of each 32-channel box, in 2 steps of 16 rows; four lanes a value
// row's, one of each 64-channel box, in 4 steps of 8 rows: so the eight lanes that a load or a store serves
// at once fall into different banks.  sc: 2^e of row `lane` (0 where there is none).
// (Rolled, and out of line: its code has to stay in the instruction cache beside the other roles'.)
template <class T, int LANES, uint32_t BOX>
static __device__ __noinline__ void put_rows(const uint8_t* raw, uint8_t* dst, float sc, int row0) {
  const int lane = threadIdx.x & 31, l = lane / LANES, ch = 2 * (lane % LANES);
  const uint8_t* from = raw + (row0 + l) * (LANES * 48) + lane % LANES * 16;
#pragma unroll 1
  for (int h = 0; h < LANES; h += 2) {
    uint4 x[6];  // all loads ahead of the stores, which the compiler takes for writing over them
#pragma unroll
    for (int j = 0; j < 6; ++j)
      x[j] = *(const uint4*)(from + j / 3 * (32 / LANES) * (LANES * 48) + j % 3 * LANES * 16);
    from += 2 * (32 / LANES) * (LANES * 48);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 32 / LANES * (h + j) + l, row = row0 + r;
      const float f = __shfl_sync(0xffffffffu, sc, r);
      uint8_t* const to = dst + swz_off(row, ch, LANES * 32);
      uint8_t* const to1 = dst + swz_off(row, ch + 1, LANES * 32);
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        *(uint4*)(to + b * BOX) = values_of<T>(x[3 * j + b].x, x[3 * j + b].y, f);
        *(uint4*)(to1 + b * BOX) = values_of<T>(x[3 * j + b].z, x[3 * j + b].w, f);
      }
    }
  }
  fence_proxy_async();
}
// The exponents of row `lane` of a tile's rows 32 q4 .. as two bytes; -128 where no token is.
__device__ __forceinline__ int exponents(const Item& it, const Tile& t, const ServeCache& cache, int q4,
                                         int lane) {
  const WindowCache& c = cache.c;
  const int slots = c.window + c.sink, slot = t.s0 + 32 * q4 + lane;
  if (t.fresh() || slot >= min(it.pos, slots)) return 0x8080;
  return __ldg(reinterpret_cast<const unsigned short*>(cache.exps) +
               ((long long)it.page * c.KV + it.kv) * slots + slot);
}

// What the issuer has to know of a tile, from the loader of keys: looked up by the issuer itself it costs a
// tile of 2,100 cycles a thousand.
enum TileInfo : uint32_t { INFO_FRESH = 1, INFO_FIRST = 2, INFO_COLS = ~15u };  // and the columns

struct Maps {
  CUtensorMap q, k, v;    // the call's rows
  CUtensorMap pk, pv;     // the pages: 16-bit rows, or codes
};

// Loads of a tile's keys or values: from the page or the call's rows.
struct Source {
  const CUtensorMap* map;
  int row, outer;
  __device__ __forceinline__ Source(const Item& it, const Tile& t, const CUtensorMap* fresh,
                                    const CUtensorMap* page)
      : map(t.fresh() ? fresh : page),
        row(t.fresh() ? it.row0 - it.i0 + t.s0 : t.s0), outer(t.fresh() ? 0 : it.page) {}
};

template <class T, class TO, bool CODES, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
window_chunk_kernel(const __grid_constant__ Maps maps, ChunkArgs a, Plan plan, DevCtl ctl) {
  constexpr bool BF16 = !__is_same(T, __half), WIDE = sizeof(TO) == 4;
  static_assert(!SPLIT || WIDE, "partial sums are fp32");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Cta cta;
  cta.base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  cta.sb = smem_u32(cta.base);
  using L = Layout<CODES>;
  cta.bar_off = L::BAR;
  cta.abort_off = L::ABORT;
  uint8_t* const base = cta.base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WindowCache& c = a.cache.c;
  const int KV = c.KV, G = a.H / KV;
  uint32_t* tmem_slot = (uint32_t*)(base + L::TMEM);
  Item* const items = (Item*)(base + L::ITEM);
  if (SPLIT) griddep_launch_dependents();  // the join waits for this whole grid
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (tid == K_WARP * 32) {
    for (uint32_t i = 0; i < P_READY; ++i) mbar_init(cta.bar(i), 1);
    mbar_init(cta.bar(P_READY), GROUP);
    mbar_init(cta.bar(P_READY + 1), GROUP);
    mbar_init(cta.bar(O_FREE), GROUP);
    mbar_init(cta.bar(DRAIN), 1);
    for (uint32_t q = REF; q < SUM; ++q) mbar_init(cta.bar(q), 32);
    for (uint32_t q = SUM; q < RAW; ++q) mbar_init(cta.bar(q), 64);
    for (uint32_t q = RAW; q < RAW_FREE; ++q) mbar_init(cta.bar(q), 1);
    for (uint32_t q = RAW_FREE; q < K_CODES; ++q) mbar_init(cta.bar(q), 128);
    for (uint32_t q = K_CODES; q < NBAR; ++q) mbar_init(cta.bar(q), 128 + 1);
    for (uint32_t i = 0; i < kWaitWords; ++i) cta.abort_flag()[i] = 0;
    ((int*)(base + L::COUNT))[1] = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.pk);
    prefetch_tensormap(&maps.pv);
  }
  {
    // ------------------------------------------------------------ the CTA's items
    // Tiles of a thread's slice of the sequences, their sums up to each slice, and a search.  Sums stop at the
    // tiles that the plan and its workspace have room for: of sequences that overlap, where `start`
    // decreases, there may be any number.  (Then a slice's tiles are what is left of it, from its front.)
    const int room = (int)(plan.units / KV);
    int* const upto = (int*)(base + L::STG);
    int* const warps = upto + THREADS + 1;
    const int slice = (c.n + THREADS - 1) / THREADS;
    const int b0 = min(tid * slice, c.n), b1 = min(b0 + slice, c.n);
    int mine = 0;
    for (int b = b0; b < b1; ++b)
      mine = min(mine + (sequence(c, a.tok, b, ctl).tokens + plan.per - 1) / plan.per, room);
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum = min(sum + y, room);
    }
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before = min(before + warps[w], room);
    upto[tid + 1] = min(before + sum, room);
    if (tid == 0) upto[0] = 0;
    __syncthreads();
    const int tiles = upto[THREADS];
    const long long all = (long long)tiles * KV * plan.parts;
    if (tid < LIST) {
      const long long u = blockIdx.x + (long long)tid * gridDim.x;
      if (u < all) {
        const int part = (int)(u % plan.parts), unit = (int)(u / plan.parts), t = unit / KV;
        int x = 0, y = THREADS;  // upto[x] <= t < upto[y]
        while (y - x > 1) {
          const int mid = (x + y) >> 1;
          if (upto[mid] <= t) x = mid;
          else y = mid;
        }
        int left = t - upto[x], b = x * slice;
        Sequence s = sequence(c, a.tok, b, ctl);
        for (;;) {
          const int n = (s.tokens + plan.per - 1) / plan.per;
          if (left < n) break;
          left -= n;
          s = sequence(c, a.tok, ++b, ctl);
        }
        make_item(items[tid], c, s, plan.per, left * plan.per, unit % KV, part, plan.parts);
        atomicAdd((int*)(base + L::COUNT) + 1, items[tid].te - items[tid].tb);
        // (rows and parts together are below 2^31)
        if (SPLIT)
          ((uint32_t*)(base + L::PLACE))[tid] =
              ((uint32_t)(part * KV + unit % KV) * a.tok.n_tokens + items[tid].row0) * G;
        if (SPLIT && part == 0 && unit % KV == 0) {
          const Partials ps(a.workspace, plan);
          ps.tiles[2 + 2 * t] = items[tid].row0;
          ps.tiles[3 + 2 * t] = items[tid].n_tok;
        }
      }
    }
    if (SPLIT && blockIdx.x == 0 && tid == 0) *(int*)a.workspace = tiles;
    if (tid == 0)
      *(int*)(base + L::COUNT) =
          (int)min((long long)LIST, max(0ll, (all - blockIdx.x + gridDim.x - 1) / gridDim.x));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_items = *(const int*)(base + L::COUNT);
  volatile uint32_t* const info = (volatile uint32_t*)(base + L::INFO);

  if (warp == K_WARP) {
    // ------------------------------------------------------------ TMA: queries and keys
    if (lane == 0) {
      const uint32_t q_bytes = 3u * 64u * plan.per * G;
      int n = 0, m = 0, q_armed = 0, raw = 0;  // key tiles and items so far; tiles of codes
      uint32_t armed = 0;                      // stages that a load was sent to
      Parities turn;
      bool ok = true;
      for (int x = 0; ok && x < n_items; ++x) {
        const Item& it = items[x];
        if (it.tb == it.te) continue;
        const uint32_t qs = m++ % L::QS;
        for (int i = it.tb; i < it.te; ++i, ++n) {
          const uint32_t s = n & 1;
          const Tile t = Ask<CODES>::tile(it, i);
          if (CODES && !t.fresh()) {
            // ahead of the stage, into the raw tile's place
            if (raw > 0 && !(ok = await(cta, cta.bar(RAW_FREE), (raw - 1) & 1, ctl))) break;
            ++raw;
            mbar_arrive_expect_tx(cta.bar(RAW), RAW_K);
            tma_load_4d(cta.sb + L::RAWS, &maps.pk, cta.bar(RAW), 0, it.kv, t.s0, it.page);
          }
          if (n >= 2 && !(ok = await(cta, cta.bar(S_FULL + s), ((n >> 1) - 1) & 1, ctl))) break;
          if (i == it.tb) {
            // of two buffers the one is free: with an item between, the scores of two tiles ago are past
            // the item before it; a single one is when the last tile's scores are done
            if (L::QS == 1 && n > 0 && !(ok = await(cta, cta.bar(S_FULL + (s ^ 1)), ((n - 1) >> 1) & 1, ctl)))
              break;
            ++q_armed;
            mbar_arrive_expect_tx(cta.bar(Q_FULL + qs), q_bytes);
            for (int j = 0; j < 3; ++j)
              tma_load_4d(cta.sb + L::Q + qs * K_BYTES + j * K_BOX, &maps.q, cta.bar(Q_FULL + qs),
                          32 * j, it.kv * G, it.row0, 0);
          }
          info[n & 3] = Ask<CODES>::cols(it, t, i) | (t.fresh() ? INFO_FRESH : 0) | (i == it.tb ? INFO_FIRST : 0);
          if (CODES) mbar_arrive(cta.bar(K_CODES + s));
          if (CODES && !t.fresh()) continue;
          const Source src(it, t, &maps.k, &maps.pk);
          armed |= 1u << s;
          turn.take(s);
          mbar_arrive_expect_tx(cta.bar(K_FULL + s), K_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + L::K + s * K_BYTES + j * K_BOX, src.map, cta.bar(K_FULL + s), 32 * j,
                        it.kv, src.row, src.outer);
        }
      }
      // every armed load has landed before the CTA may exit
      if (raw > 0) mbar_wait(cta.bar(RAW), (raw - 1) & 1, ctl, DRAIN_NS);
      for (int s = 0; s < 2; ++s)
        if ((armed >> s) & 1) mbar_wait(cta.bar(K_FULL + s), turn.take(s) ^ 1, ctl, DRAIN_NS);
      for (int s = 0; s < (int)L::QS; ++s)
        if (q_armed > s) mbar_wait(cta.bar(Q_FULL + s), ((q_armed - 1 - s) / L::QS) & 1, ctl, DRAIN_NS);
    }
  } else if (warp == V_WARP) {
    // ------------------------------------------------------------ TMA: values
    if (lane == 0) {
      int n = 0;
      uint32_t armed = 0;
      Parities turn;
      int raw = 0;
      bool ok = true;
      for (int x = 0; ok && x < n_items; ++x) {
        const Item& it = items[x];
        for (int i = it.tb; i < it.te; ++i, ++n) {
          const uint32_t s = n & 1;
          const Tile t = Ask<CODES>::tile(it, i);
          if (CODES && !t.fresh()) {
            if (raw > 0 && !(ok = await(cta, cta.bar(RAW_FREE + 1), (raw - 1) & 1, ctl))) break;
            ++raw;
            mbar_arrive_expect_tx(cta.bar(RAW + 1), RAW_V);
            tma_load_4d(cta.sb + L::RAWS + RAW_K, &maps.pv, cta.bar(RAW + 1), 0, it.kv, t.s0, it.page);
          }
          if (n >= 2 && !(ok = await(cta, cta.bar(O_DONE + s), ((n >> 1) - 1) & 1, ctl))) break;
          if (CODES) mbar_arrive(cta.bar(V_CODES + s));
          if (CODES && !t.fresh()) continue;
          const Source src(it, t, &maps.v, &maps.pv);
          armed |= 1u << s;
          turn.take(s);
          mbar_arrive_expect_tx(cta.bar(V_FULL + s), V_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + L::V + s * V_BYTES + j * V_BOX, src.map, cta.bar(V_FULL + s), 64 * j,
                        it.kv, src.row, src.outer);
        }
      }
      if (raw > 0) mbar_wait(cta.bar(RAW + 1), (raw - 1) & 1, ctl, DRAIN_NS);
      for (int s = 0; s < 2; ++s)
        if ((armed >> s) & 1) mbar_wait(cta.bar(V_FULL + s), turn.take(s) ^ 1, ctl, DRAIN_NS);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t ID_S = idesc_f16(128, 0, BF16, BF16, false, false);
      constexpr uint32_t ID_PV = idesc_f16(128, 192, BF16, BF16, false, true);
      const uint64_t q_desc = smem_desc(cta.sb + L::Q, 16, 512, SW_64);
      const uint64_t k_desc = smem_desc(cta.sb + L::K, 16, 512, SW_64);
      const uint64_t v_desc = smem_desc(cta.sb + L::V, V_BOX, 1024, SW_128);
      // the scores run two tiles ahead of the values
      const int total = ((const int*)(base + L::COUNT))[1];
      int sn = 0, sm = -1, vm = -1;
      uint32_t kept = 0;  // the infos of the tiles whose scores have been asked for, a half word each
      Parities turn;
      // stage s has the CTA's n-th tile: keys (what 0) or values (2)
      auto filled = [&](bool fresh, uint32_t what, uint32_t s, int n) -> bool {
        if (CODES && !await(cta, cta.bar(K_CODES + what + s), (n >> 1) & 1, ctl)) return false;
        return (CODES && !fresh) || await(cta, cta.bar(K_FULL + what + s), turn.take(what + s), ctl);
      };
      auto scores = [&]() -> bool {  // S[sn & 1] = Q K^T
        const uint32_t s = sn & 1;
        // the info comes with the loader's arrival, codes: at the operands' barrier
        if (!CODES && !await(cta, cta.bar(K_FULL + s), turn.take(s), ctl)) return false;
        if (CODES && !await(cta, cta.bar(K_CODES + s), (sn >> 1) & 1, ctl)) return false;
        const uint32_t k1 = info[sn & 3];
        if (CODES && (k1 & INFO_FRESH) && !await(cta, cta.bar(K_FULL + s), turn.take(s), ctl)) return false;
        if (k1 & INFO_FIRST) ++sm;
        const uint32_t qs = sm % L::QS;
        if ((k1 & INFO_FIRST) && !await(cta, cta.bar(Q_FULL + qs), (sm / L::QS) & 1, ctl)) return false;
        const uint32_t id = ID_S | ((k1 & INFO_COLS) << 14);
        kept = s ? (kept & 0xFFFFu) | k1 << 16 : (kept & 0xFFFF0000u) | k1;
        tc_fence_after();
        const uint64_t q = q_desc + (qs * K_BYTES >> 4), k = k_desc + (s * K_BYTES >> 4);
#pragma unroll
        for (int j = 0; j < 6; ++j) {  // (the descriptors count in 16 bytes)
          const uint32_t off = ((j >> 1) * K_BOX + (j & 1) * 32) >> 4;
          mma_f16_ss(tmem + TM_S + 128 * s, q + off, k + off, id, j > 0);
        }
        mma_commit(cta.bar(S_FULL + s));
        ++sn;
        return true;
      };
      bool ok = true;
      for (int i = 0; i < 2 && ok && sn < total; ++i) ok = scores();
      for (int vn = 0; ok && vn < total; ++vn) {
        const uint32_t s = vn & 1;
        if (vn == ctl.stall_step) {  // the give-up path's diagnostic (see chunk_fwd.cu)
          await(cta, cta.bar(DRAIN), 0, ctl);
          break;
        }
        const uint32_t k1 = s ? kept >> 16 : kept & 0xFFFFu;
        const int steps = (int)k1 >> 4;
        const bool first = k1 & INFO_FIRST;
        if (!filled(k1 & INFO_FRESH, 2, s, vn)) break;
        if (first && ++vm > 0 && !await(cta, cta.bar(O_FREE), (vm - 1) & 1, ctl)) break;
        if (!await(cta, cta.bar(P_READY + s), (vn >> 1) & 1, ctl)) break;
        tc_fence_after();
        const uint64_t v = v_desc + (s * V_BYTES >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < steps)
            mma_f16_ts(tmem + TM_O, tmem + TM_S + 128 * s + 8 * j, v + (j * 2048 >> 4), ID_PV,
                       !first || j > 0);
        mma_commit(cta.bar(O_DONE + s));
        made_step(cta, STEP_TILE, vn + 1);
        if (sn < total) ok = scores();
      }
      mma_commit(cta.bar(DRAIN));
      mbar_wait(cta.bar(DRAIN), 0, ctl, DRAIN_NS);
    }
  } else if (warp < K_WARP) {
    // ------------------------------------------------------------ softmax
    // Group g takes the CTA's tiles of parity g, whose scores are in buffer g.  ref and the sums
    // are in base 2.
    const int q4 = warp & 3, g = warp >> 2, row = 32 * q4 + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    const int tok = row / G, tok_a = 32 * q4 / G, tok_b = (32 * q4 + 31) / G;  // of a tile's tokens
    float* refs = (float*)(base + L::REFS);
    float2* sums = (float2*)(base + L::SUMS);
    int n0 = 0, m = 0;      // tiles and items before this one
    uint32_t v_turn = 0;    // parity of the group's next tile of values that comes by TMA
    bool ok = true;
    for (int x = 0; ok && x < n_items; ++x) {
      const Item& it = items[x];
      if (it.tb == it.te) continue;
      // rows past the item's tokens see nothing; a warp of such rows only keeps step
      const bool live = tok < it.n_tok && row < plan.per * G, awake = tok_a < it.n_tok;
      const int at = it.i0 + tok, ends = it.i0 + (lane & 4 ? min(tok_b, it.n_tok - 1) : tok_a);
      float ref = -INFINITY, sum = 0.f;  // this row's, as of the group's last tile
      for (int i = it.tb + ((n0 ^ g) & 1); i < it.te; i += 2) {
        const int n = n0 + i - it.tb;
        const Tile t = Ask<CODES>::tile(it, i);
        // chunks of 32 columns that all rows of the warp see, and that some do: what its first and its
        // last row both see, those between do too; a chunk that neither sees, none does
        uint32_t full = awake ? 15u : 0u, some = full;
        if (!t.whole() && awake) {
          const uint32_t see = Ask<CODES>::seen(it, t.fresh(), ends, t.s0 + 32 * (lane & 3));
          full = __ballot_sync(0xffffffffu, see == ~0u);
          some = __ballot_sync(0xffffffffu, see != 0u);
          full = full & (full >> 4) & 15u;
          some = (some | (some >> 4)) & 15u;
        }
        const int cols = Ask<CODES>::cols(it, t, i);
        if (!(ok = await_warp(cta, cta.bar(S_FULL + g), (n >> 1) & 1, ctl))) break;
        tc_fence_after();
        const uint32_t ts = trow + TM_S + 128 * g;
        auto sees = [&](int j) -> uint32_t {
          return live ? Ask<CODES>::seen(it, t.fresh(), at, t.s0 + 32 * j) : 0u;
        };
        auto hide = [&](uint32_t (&z)[32], int j) {  // the columns that this row does not see
          const uint32_t see = sees(j);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((see >> e) & 1)) z[e] = 0xFF800000u;  // -inf
        };
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto maxima = [&](const uint32_t (&z)[32]) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            m4[j & 3] = max3(m4[j & 3], __uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1]));
        };
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          if (!((some >> j) & 1)) continue;
          uint32_t z[32];
          tmem_ld32(ts + 32 * j, z);
          tmem_wait_ld();
          if (!((full >> j) & 1)) hide(z, j);
          maxima(z);
        }
        // (a row of no token may hold anything, and reaches none but itself)
        const float top = live ? max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * kLog2e : -INFINITY;
        // the other group's reference of the tile before (and, as the item begins, no more
        // than its word that it is past that tile)
        if (n > 0 &&
            !(ok = await_warp(cta, cta.bar(REF + 4 * (g ^ 1) + q4), ((n - 1) >> 1) & 1, ctl)))
          break;
        const float before = i > it.tb ? refs[(g ^ 1) * 128 + row] : -INFINITY;
        // a row that has seen nothing yet has o = 0 and takes any scale
        const float now = top > before + 8.f ? top : before;
        refs[g * 128 + row] = now;
        mbar_arrive(cta.bar(REF + 4 * g + q4));
        const float scale = now == before || before == -INFINITY ? 1.f : ex2(before - now);
        if (now != ref) sum = ref == -INFINITY ? 0.f : sum * ex2(ref - now);
        ref = now;
        if (awake) {
          const float sub = ref == -INFINITY ? 0.f : -ref;
          const float2 sub2 = make_float2(sub, sub), l2e = make_float2(kLog2e, kLog2e);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // P over the columns of S that have been read: weights of 32 columns from their scores, as pairs.
          // (One rolled loop for all tiles: a copy of it for whole ones, unrolled, pushes other roles' code
          // out of the instruction cache.)
#pragma unroll 1
          for (int j = 0; 32 * j < cols; ++j) {
            uint32_t p[16];
            if ((some >> j) & 1) {
              uint32_t z[32];
              tmem_ld32(ts + 32 * j, z);
              tmem_wait_ld();
              if (!((full >> j) & 1)) hide(z, j);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float2 y = fma2(make_float2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])),
                                l2e, sub2);
                y.x = ex2(y.x);
                y.y = ex2(y.y);
                acc[e & 1] = add2(acc[e & 1], y);
                p[e] = pack2<T>(y.x, y.y);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) p[e] = 0u;
            }
            tmem_st16(ts + 16 * j, p);
          }
          acc[0] = add2(acc[0], acc[1]);
          sum += acc[0].x + acc[0].y;
        }
        if (i > it.tb && __any_sync(0xffffffffu, scale != 1.f)) {
          // O once the tile before has been added (and the one before that, whose phase of the
          // barrier this could be taken for, is: this tile's scores came behind it)
          if (!(ok = await_warp(cta, cta.bar(O_DONE + (g ^ 1)), ((n - 1) >> 1) & 1, ctl))) break;
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < 6; ++j) {
            uint32_t o[32];
            tmem_ld32(trow + TM_O + 32 * j, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
            tmem_st32(trow + TM_O + 32 * j, o);
          }
        }
        // values behind the tokens of a page or a sequence may be anything, and 0 x NaN is NaN: zero
        // their rows (codes: the output warps did)
        const int kept = t.fresh() ? it.tokens - t.s0 : CODES ? BN : it.pos - t.s0;
        const uint32_t v_now = v_turn;
        if (!CODES || t.fresh()) v_turn ^= 1;
        if (awake && kept < cols) {
          if (!(ok = await_warp(cta, cta.bar(V_FULL + g), v_now, ctl))) break;
          const int step = 32 * min((min(it.n_tok, plan.per) * G + 31) / 32, 4), cnt = (cols - kept) * 24;
          for (int y = row; y < cnt; y += step)
            *(uint4*)(base + L::V + g * V_BYTES + (y % 24 / 8) * V_BOX + (kept + y / 24) * 128 +
                      (y & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(cta.bar(P_READY + g));
      }
      if (!ok) break;
      n0 += it.te - it.tb;
      // one item at a time: the output warps have taken the sums of the item before
      if (m > 0 && !(ok = await_warp(cta, cta.bar(O_FREE), (m - 1) & 1, ctl))) break;
      sums[(m & 1) * 256 + g * 128 + row] = make_float2(sum, ref);
      mbar_arrive(cta.bar(SUM + q4));
      ++m;
    }
  } else {
    // ------------------------------------------------------------ output rows (and codes)
    const int q4 = warp & 3, row = 32 * q4 + lane;  // the quadrant that the warp may read
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    const float2* sums = (const float2*)(base + L::SUMS);
    constexpr int SR = L::STG_ROW, SUBS = SR / 64, LPR = SR / 16;  // staged rows: 64-byte parts, lanes of a row
    uint8_t* const stg = base + L::STG + q4 * 32 * SR;
    constexpr int CB = WIDE ? 16 : 32;  // channels of 64 bytes
    const uint32_t by_G = (65536 + G - 1) / G;
    int n0 = 0, m = 0, seen = 0, n = 0;  // tiles and items before this one; tiles filled
    bool ok = true;

    // Codes: rows 32 q4 .. + 31 of each tile by this warp.
    [[maybe_unused]] int raw = 0, exps = 0;  // tiles of codes so far; the next tile's exponents
    [[maybe_unused]] bool codes_next = false;
    [[maybe_unused]] Walk at{0, 0};
    [[maybe_unused]] auto look = [&]() {
      if (at.x >= n_items) return;
      const Tile t = Ask<CODES>::tile(items[at.x], at.i);
      codes_next = !t.fresh();
      exps = exponents(items[at.x], t, a.cache, q4, lane);
    };
    if constexpr (CODES) {
      at.begin(items, n_items);
      look();
    }
    // Fills up to tile `stop` of item `upto`.
    [[maybe_unused]] auto fill_to = [&](int upto, int stop) -> bool {
      while (at.x < n_items && (at.x < upto || (at.x == upto && at.i < stop))) {
        const uint32_t s = n & 1;
        const bool codes = codes_next;
        asm volatile("" : "+r"(exps));  // (not taken apart where it is loaded, a tile ahead)
        const int ek = (signed char)(exps & 255), ev = (signed char)(exps >> 8);
        const float sk = ek < -126 ? 0.f : pow2(ek), sv = ev < -126 ? 0.f : pow2(ev);
        at.step(items, n_items);
        look();
        if (n >= 2 && !await_warp(cta, cta.bar(S_FULL + s), ((n >> 1) - 1) & 1, ctl)) return false;
        if (codes) {
          if (!await_warp(cta, cta.bar(RAW), raw & 1, ctl)) return false;
          put_rows<T, 2, K_BOX>(base + L::RAWS, base + L::K + s * K_BYTES, sk, 32 * q4);
          mbar_arrive(cta.bar(RAW_FREE));
        }
        mbar_arrive(cta.bar(K_CODES + s));
        if (n >= 2 && !await_warp(cta, cta.bar(O_DONE + s), ((n >> 1) - 1) & 1, ctl)) return false;
        if (codes) {
          if (!await_warp(cta, cta.bar(RAW + 1), raw & 1, ctl)) return false;
          put_rows<T, 4, V_BOX>(base + L::RAWS + RAW_K, base + L::V + s * V_BYTES, sv, 32 * q4);
          mbar_arrive(cta.bar(RAW_FREE + 1));
          ++raw;
        }
        mbar_arrive(cta.bar(V_CODES + s));
        ++n;
      }
      return true;
    };

    for (int x = 0; x < n_items; ++x) {
      const Item& it = items[x];
      const bool live_item = it.tb < it.te;
      if constexpr (CODES) {
        // all of this item's tiles, and the first two of the next one that has any
        if (!(ok = fill_to(x, it.te))) break;
        if (at.x < n_items && !(ok = fill_to(at.x, items[at.x].tb + 2))) break;
      }
      float ref = -INFINITY, sum = 0.f;
      if (live_item) {
        n0 += it.te - it.tb;
        if (!await_warp(cta, cta.bar(SUM + q4), m & 1, ctl)) break;
        const float2 s0 = sums[(m & 1) * 256 + row], s1 = sums[(m & 1) * 256 + 128 + row];
        ref = fmaxf(s0.y, s1.y);
        if (s0.y != -INFINITY) sum = s0.x * ex2(s0.y - ref);
        if (s1.y != -INFINITY) sum = fmaf(s1.x, ex2(s1.y - ref), sum);
        // the last tile's scores came behind the sums of the tile before the one before it, so this
        // is the last one's phase
        if (!await_warp(cta, cta.bar(O_DONE + ((n0 - 1) & 1)), ((n0 - 1) >> 1) & 1, ctl)) break;
        tc_fence_after();
        ++m;
      }
      const int rows = it.n_tok * G;
      float inv = SPLIT ? 1.f : 1.f / sum;
      TO* out;
      if constexpr (SPLIT) {
        const Partials ps(a.workspace, plan);
        const size_t at = ((const uint32_t*)(base + L::PLACE))[x];
        if (row < rows) ps.ml[at + row] = make_float2(ref, sum);
        out = ps.o + at * kDV;
      } else {
        out = static_cast<TO*>(a.o) + ((long long)it.row0 * a.H + it.kv * G) * kDV;
      }
      if (live_item) {
        const bool awake = 32 * q4 < rows;
        // 32 rows of SR bytes at a time go through shared memory, so that LPR lanes write a row
        auto stage = [&](int e, const uint32_t (&w)[16]) {  // 64 bytes of this lane's row
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            *(uint4*)(stg + swz_off(lane, 4 * e + ch, SR)) =
                make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
        };
        auto emit = [&](int k) {  // channels SUBS CB k ..
          __syncwarp();
#pragma unroll
          for (int ch = 0; ch < LPR; ++ch) {
            const int r = 32 / LPR * ch + lane / LPR, rr = 32 * q4 + r;
            const uint4 y = *(const uint4*)(stg + swz_off(r, lane % LPR, SR));
            if (rr < rows) {
              // row rr's token and head: rr / G by a product, exact for rr, G <= 128
              const int to = SPLIT ? rr : rr + (int)((uint32_t)rr * by_G >> 16) * (a.H - G);
              reinterpret_cast<uint4*>(out + (long long)to * kDV + SUBS * CB * k)[lane % LPR] = y;
            }
          }
          __syncwarp();
        };
        auto rounded = [&](int blk, uint32_t (&y)[16]) {  // 64 bytes of this lane's row
          if constexpr (WIDE) {
            tmem_ld16(trow + TM_O + CB * blk, y);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * inv);
          } else {
            uint32_t o[32];
            tmem_ld32(trow + TM_O + CB * blk, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              y[j] = pack2<TO>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
          }
        };
        if constexpr (WIDE || CODES) {
#pragma unroll 1
          for (int k = 0; k < kDV / (SUBS * CB); ++k) {
            if (awake)
#pragma unroll
              for (int e = 0; e < SUBS; ++e) {
                uint32_t o[16];
                rounded(SUBS * k + e, o);
                stage(e, o);
              }
            if (k == kDV / (SUBS * CB) - 1) {
              tc_fence_before();
              mbar_arrive(cta.bar(O_FREE));
            }
            if (awake) emit(k);
          }
        } else {
          // all of the row is read and rounded before any of it is written, so that the next item's products
          // wait less: blocks of 32 channels, the last ones to the staging, the others in registers
          constexpr int HOLD = kDV / CB - SUBS;
          uint32_t w[HOLD][16], last[16];
          if (awake) {
#pragma unroll
            for (int e = 0; e < SUBS; ++e) {
              rounded(HOLD + e, last);
              stage(e, last);
            }
#pragma unroll
            for (int k = 0; k < HOLD; ++k) rounded(k, w[k]);
          }
          tc_fence_before();
          mbar_arrive(cta.bar(O_FREE));
          if (awake) {
            emit(HOLD / SUBS);
#pragma unroll
            for (int k = 0; k < HOLD / SUBS; ++k) {
#pragma unroll
              for (int e = 0; e < SUBS; ++e) stage(e, w[SUBS * k + e]);
              emit(k);
            }
          }
        }
      }
      if (tid == OUT_WARP * 32) made_step(cta, STEP_ITEM, ++seen);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One block per row of a cut unit.
template <class TO>
__global__ void __launch_bounds__(JOIN_THREADS)
window_chunk_join_kernel(ChunkArgs a, Plan plan) {
  griddep_wait();
  const uint32_t all = (uint32_t)a.tok.n_tokens * a.H;  // (times the parts below 2^31)
  const Partials ps(a.workspace, plan);
  const int KV = a.cache.c.KV, G = a.H / KV;
  const int unit = blockIdx.x, t = unit / KV, kv = unit % KV, row = blockIdx.y;
  if (t >= ps.tiles[0]) return;
  const int row0 = ps.tiles[2 + 2 * t];
  if (row >= ps.tiles[3 + 2 * t] * G) return;
  const uint32_t at = ((uint32_t)kv * a.tok.n_tokens + row0) * G + row;
  join_row(
      plan.parts, [&](int p) { return ps.ml[at + p * all]; }, [&](int p) { return ps.o + (size_t)(at + p * all) * kDV; },
      static_cast<TO*>(a.o) + (((long long)row0 + row / G) * a.H + kv * G + row % G) * kDV);
}

// Rows [outer, rows, heads, d] of 16 bits as boxes of `box_d` channels, `box_h` heads, `box_r` rows.
inline bool make_map(CUtensorMap* map, const void* base, CUtensorMapDataType type, int size, int d, int heads,
                     long long rows, long long outer, int box_d, int box_h, int box_r,
                     CUtensorMapSwizzle sw) {
  auto fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[3] = {(cuuint64_t)d * size, (cuuint64_t)d * size * heads,
                           (cuuint64_t)d * size * heads * rows};
  cuuint32_t box[4] = {(cuuint32_t)box_d, (cuuint32_t)box_h, (cuuint32_t)box_r, 1u};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, type, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, class TO, bool CODES, bool SPLIT>
cudaError_t launch(const Maps& maps, const ChunkArgs& a, const Plan& plan, DevCtl ctl,
                   cudaStream_t stream) {
  auto kern = window_chunk_kernel<T, TO, CODES, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<CODES>::BYTES);
  if (e != cudaSuccess) return e;
  kern<<<plan.grid, THREADS, Layout<CODES>::BYTES, stream>>>(maps, a, plan, ctl);
  return cudaGetLastError();
}

template <class T, bool CODES>
cudaError_t run(const ChunkArgs& a, const Plan& plan, DevCtl ctl, cudaStream_t stream) {
  constexpr bool bf16 = !__is_same(T, __half);
  const auto type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const WindowCache& c = a.cache.c;
  const int G = a.H / c.KV, slots = c.window + c.sink;
  const long long N = a.tok.n_tokens, pages = (long long)c.n_pages * c.pool_layers;
  Maps m;
  bool ok = make_map(&m.q, a.q, type, 2, kDK, a.H, N, 1, 32, G, plan.per, CU_TENSOR_MAP_SWIZZLE_64B) &&
            make_map(&m.k, a.k, type, 2, kDK, c.KV, N, 1, 32, 1, BN, CU_TENSOR_MAP_SWIZZLE_64B) &&
            make_map(&m.v, a.v, type, 2, kDV, c.KV, N, 1, 64, 1, BN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (CODES) {
    const auto code = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    ok = ok && make_map(&m.pk, c.k, code, 1, kDK, c.KV, slots, pages, kDK, 1, BN, CU_TENSOR_MAP_SWIZZLE_NONE) &&
         make_map(&m.pv, c.v, code, 1, kDV, c.KV, slots, pages, kDV, 1, BN, CU_TENSOR_MAP_SWIZZLE_NONE);
  } else {
    ok = ok &&
         make_map(&m.pk, c.k, type, 2, kDK, c.KV, slots, pages, 32, 1, BN, CU_TENSOR_MAP_SWIZZLE_64B) &&
         make_map(&m.pv, c.v, type, 2, kDV, c.KV, slots, pages, 64, 1, BN, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (plan.parts > 1) return launch<T, float, CODES, true>(m, a, plan, ctl, stream);
  if (a.out_type == GLA_FP32) return launch<T, float, CODES, false>(m, a, plan, ctl, stream);
  return launch<T, T, CODES, false>(m, a, plan, ctl, stream);
}

cudaError_t launch8(const ChunkArgs& a, const Plan& plan, DevCtl ctl, cudaStream_t stream);

}  // namespace chunk
}  // namespace gla
