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
//   codes    the output warps, idle while an item is walked, turn the 8-bit rows of a page's tile into
//            the swizzled 16-bit operands, c 2^e exactly; rows come from L2, where TMA prefetches have
//            put them four tiles ahead.  They do so for the next item's first two tiles before they take the
//            output rows, so that the scores stay two tiles ahead across items.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "tmap.h"
#include "window_packed.cuh"
#include "window_wait.cuh"

namespace gla {
namespace chunk {

using scan::Cta;
using scan::DRAIN_NS;

constexpr int BM = 128, BN = 128;
constexpr uint32_t K_BOX = 8192, V_BOX = 16384;  // 128 rows x 64 B, x 128 B
constexpr uint32_t K_BYTES = 3 * K_BOX, V_BYTES = 3 * V_BOX;
constexpr int LIST = 64;                         // items of a CTA
constexpr int AHEAD = 4;                         // tiles that codes are prefetched ahead

// The sequence's keys that an item walks, and which of them are its part's.
struct Item {
  int row0, i0, n_tok;            // first packed row; first token of the sequence's new ones; tokens
  int tokens, pos, page, kv;      // of the sequence
  int unit;                       // (tile, key head), part: where its partial results go
  int n0, l1, h1, l2, h2;         // tiles of the page: 0 .. n0-1, l1 .. h1-1, l2 .. h2-1
  int far, lo;                    // of the new tokens: 0 .. far-1, lo ..
  int tb, te;                     // tiles tb .. te-1 of all these are this part's
  int ns, a_lo, a_hi, b_lo, base; // slots seen: 0 .. ns-1, a_lo .. a_hi-1, b_lo .. (all for the first row);
                                  // slot sink + r of the first ring run holds token base + r
};
static_assert(sizeof(Item) == 22 * 4, "words");

constexpr uint32_t OFF_Q = 0, OFF_K = 2 * K_BYTES, OFF_V = 4 * K_BYTES;
constexpr uint32_t OFF_STG = OFF_V + 2 * V_BYTES;  // output staging, 4 KB per output warp
constexpr uint32_t OFF_REF = OFF_STG + 4 * 4096;   // float ref[2][128]: each group's reference
constexpr uint32_t OFF_SUM = OFF_REF + 1024;       // float2 sum[2][2][128]: (sum, ref), by item
constexpr uint32_t OFF_ITEM = OFF_SUM + 4096;
constexpr uint32_t OFF_BAR = OFF_ITEM + LIST * sizeof(Item);
static_assert(OFF_BAR % 8 == 0, "barriers");
// As in window_fwd.cu.  K_CODES, V_CODES: a tile's codes have been turned into operands; the loaders and
// the output warps arrive there for every tile, also for one that asks nothing of them, so that none falls
// two phases behind a barrier that it waits for, which its parity would not show.
enum Bar : uint32_t {
  Q_FULL = 0, K_FULL = 2, V_FULL = 4, S_FULL = 6, O_DONE = 8, P_READY = 10, O_FREE = 12, DRAIN = 13,
  REF = 14, SUM = 22, K_CODES = 26, V_CODES = 28, NBAR = 30
};
constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_COUNT = OFF_TMEM + 4;
constexpr uint32_t OFF_ABORT = OFF_COUNT + 4;
constexpr uint32_t SMEM_USED = OFF_ABORT + 4 * kWaitWords, SMEM_BYTES = SMEM_USED + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

// Columns: S twice 128, O 192.  A tile's P takes the place of its S, from the front.
constexpr uint32_t TM_S = 0, TM_O = 256;

constexpr int GROUP = 128, K_WARP = 8, V_WARP = 9, MMA_WARP = 10, OUT_WARP = 11;
constexpr int THREADS = 15 * 32;

struct Plan {
  int per;        // tokens of an item
  int parts;
  long long units;  // (tile, key head) at most
  unsigned grid;
};
// The workspace of cut items: the tiles' rows and tokens, (reference, sum) and o of each unit's parts.
struct Partials {
  int* tiles;   // [0]: how many; [2 + 2 i], [3 + 2 i]: row0, n_tok
  float2* ml;   // [units][parts][128]
  float* o;     // [units][parts][128][192]
  static __host__ __device__ size_t head(long long units) { return ((units + 1) * 8 + 255) / 256 * 256; }
  static __host__ __device__ size_t bytes(long long units, int parts) {
    return head(units) + (size_t)units * parts * BM * (8 + kDV * 4);
  }
  __host__ __device__ Partials(void* p, long long units, int parts) {
    tiles = static_cast<int*>(p);
    ml = reinterpret_cast<float2*>(static_cast<char*>(p) + head(units));
    o = reinterpret_cast<float*>(ml + (size_t)units * parts * BM);
  }
};

__device__ __forceinline__ int ceil_tiles(int n) { return n <= 0 ? 0 : (n - 1) / BN + 1; }

// Item of tokens i0 .. of a sequence, part `part` of `parts`.
__device__ __forceinline__ Item make_item(const WindowCache& c, const Sequence& s, int per, int i0, int kv,
                                          int unit, int part, int parts) {
  Item it;
  it.i0 = i0;
  it.n_tok = min(per, s.tokens - i0);
  it.row0 = s.first + i0;
  it.tokens = s.tokens;
  it.pos = s.pos;
  it.page = s.page * c.pool_layers + c.layer;
  it.kv = kv;
  it.unit = unit;
  const int slots = c.window + c.sink, p0 = s.pos + i0, i1 = i0 + it.n_tok;
  it.ns = min(c.sink, s.pos);
  it.a_lo = it.a_hi = 0;
  it.b_lo = slots;
  it.base = 0;
  if (s.pos > c.sink) {
    const int last = s.pos - 1 - c.sink, lr = last % c.window;
    it.base = s.pos - 1 - lr;
    const int x = p0 - it.base - c.window + 1;  // ring place of the oldest token seen
    it.a_lo = c.sink + max(0, x);
    it.a_hi = c.sink + lr + 1;
    if (it.a_lo >= it.a_hi) it.a_lo = it.a_hi;
    // behind the newest token are those of the round before, if there was one
    if (it.base > c.sink) it.b_lo = min(max(it.a_hi, c.sink + x + c.window), slots);
  }
  it.n0 = ceil_tiles(it.ns);
  it.l1 = max(it.a_lo / BN, it.n0);
  it.h1 = it.a_lo < it.a_hi ? max(ceil_tiles(it.a_hi), it.l1) : it.l1;
  it.l2 = max(it.b_lo / BN, it.h1);
  it.h2 = it.b_lo < slots ? max(ceil_tiles(slots), it.l2) : it.l2;
  const KeyTiles kt(i0, i1, BN, c.window, max(c.sink - s.pos, 0));
  it.far = kt.far;
  it.lo = kt.lo;
  const long long n = it.n0 + it.h1 - it.l1 + it.h2 - it.l2 + kt.n;
  it.tb = (int)(n * part / parts);
  it.te = (int)(n * (part + 1) / parts);
  return it;
}

struct Tile {
  bool fresh;   // of the new tokens
  int s0;       // first slot, or first of the sequence's new tokens
  int cols;     // columns that some row may see, rounded to 16
};
__device__ __forceinline__ Tile tile_of(const Item& it, const WindowCache& c, int i) {
  Tile t;
  const int n1 = it.n0 + it.h1 - it.l1, n2 = n1 + it.h2 - it.l2;
  t.fresh = i >= n2;
  int end;
  if (t.fresh) {
    const int j = i - n2;
    t.s0 = BN * (j < it.far ? j : it.lo + j - it.far);
    end = j < it.far && t.s0 / BN < it.lo ? min(c.sink - it.pos, it.i0 + it.n_tok) : it.i0 + it.n_tok;
  } else {
    t.s0 = BN * (i < it.n0 ? i : i < n1 ? it.l1 + i - it.n0 : it.l2 + i - n1);
    const int slots = c.window + c.sink;
    end = it.ns;
    if (it.a_lo < min(it.a_hi, t.s0 + BN)) end = max(end, it.a_hi);
    if (it.b_lo < min(slots, t.s0 + BN)) end = slots;
  }
  t.cols = min(BN, (end - t.s0 + 15) & ~15);
  return t;
}
// The columns c0 .. c0 + 31 of a tile that token i of the sequence's new ones sees.
__device__ __forceinline__ uint32_t columns_seen(const Item& it, const WindowCache& c, bool fresh, int i,
                                                 int c0) {
  if (fresh) return keys_seen(i, c0, it.tokens, c.window, max(c.sink - it.pos, 0));
  const int x = it.pos - it.base + i - c.window + 1, slots = c.window + c.sink;
  return bits_to(it.ns - 1 - c0) | (bits_to(it.a_hi - 1 - c0) & ~bits_to(c.sink + max(0, x) - 1 - c0)) |
         (it.base > c.sink && it.a_hi > 0
              ? bits_to(slots - 1 - c0) & ~bits_to(max(it.a_hi, c.sink + x + c.window) - 1 - c0)
              : 0u);
}

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
    // (2^23 + u) s - (2^23 + 128) s, exact in one fp32 operation
    const float2 s2 = make_float2(s, s), off = make_float2(-8388736.f * s, -8388736.f * s);
    const uint32_t m = 0x4B000000u;
    uint32_t* w = &o.x;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t u = (j ? hi : lo) ^ 0x80808080u;
      const float2 x = fma2(make_float2(__uint_as_float(__byte_perm(u, m, 0x7440)),
                                        __uint_as_float(__byte_perm(u, m, 0x7441))), s2, off);
      const float2 y = fma2(make_float2(__uint_as_float(__byte_perm(u, m, 0x7442)),
                                        __uint_as_float(__byte_perm(u, m, 0x7443))), s2, off);
      w[2 * j] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
      w[2 * j + 1] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
    }
  }
  return o;
}

struct Maps {
  CUtensorMap q, k, v;    // the call's rows
  CUtensorMap pk, pv;     // the pages: 16-bit rows, or codes (for prefetches)
};

// Loads of a tile's keys or values: from the page or the call's rows.
struct Source {
  const CUtensorMap* map;
  int row, outer;
  __device__ __forceinline__ Source(const Item& it, const Tile& t, const CUtensorMap* fresh,
                                    const CUtensorMap* page)
      : map(t.fresh ? fresh : page),
        row(t.fresh ? it.row0 - it.i0 + t.s0 : t.s0), outer(t.fresh ? 0 : it.page) {}
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
  cta.bar_off = OFF_BAR;
  cta.abort_off = OFF_ABORT;
  uint8_t* const base = cta.base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WindowCache& c = a.cache.c;
  const int KV = c.KV, G = a.H / KV;
  uint32_t* tmem_slot = (uint32_t*)(base + OFF_TMEM);
  Item* const items = (Item*)(base + OFF_ITEM);
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
    for (uint32_t q = SUM; q < K_CODES; ++q) mbar_init(cta.bar(q), 64);
    for (uint32_t q = K_CODES; q < NBAR; ++q) mbar_init(cta.bar(q), 128 + 1);
    for (uint32_t i = 0; i < kWaitWords; ++i) cta.abort_flag()[i] = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.pk);
    prefetch_tensormap(&maps.pv);
  }
  {
    // ------------------------------------------------------------ the CTA's items
    // Tiles of a thread's slice of the sequences, their sums up to each slice, and a search.
    int* const upto = (int*)(base + OFF_STG);
    int* const warps = upto + THREADS + 1;
    const int slice = (c.n + THREADS - 1) / THREADS;
    const int b0 = min(tid * slice, c.n), b1 = min(b0 + slice, c.n);
    int mine = 0;
    for (int b = b0; b < b1; ++b)
      mine += (sequence(c, a.tok, b, ctl).tokens + plan.per - 1) / plan.per;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += y;
    }
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warps[w];
    upto[tid + 1] = before + sum;
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
        items[tid] = make_item(c, s, plan.per, left * plan.per, unit % KV, unit, part, plan.parts);
        if (SPLIT && part == 0 && unit % KV == 0) {
          const Partials ps(a.workspace, plan.units, plan.parts);
          ps.tiles[2 + 2 * t] = items[tid].row0;
          ps.tiles[3 + 2 * t] = items[tid].n_tok;
        }
      }
    }
    if (SPLIT && blockIdx.x == 0 && tid == 0) *(int*)a.workspace = tiles;
    if (tid == 0)
      *(int*)(base + OFF_COUNT) =
          (int)min((long long)LIST, max(0ll, (all - blockIdx.x + gridDim.x - 1) / gridDim.x));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_items = *(const int*)(base + OFF_COUNT);

  if (warp == K_WARP) {
    // ------------------------------------------------------------ TMA: queries and keys
    if (lane == 0) {
      const uint32_t q_bytes = 3u * 64u * plan.per * G;
      int n = 0, m = 0, q_armed = 0;  // key tiles and items so far
      uint32_t armed = 0;             // stages that a load was sent to
      Parities turn;
      bool ok = true;
      for (int x = 0; ok && x < n_items; ++x) {
        const Item& it = items[x];
        if (it.tb == it.te) continue;
        const uint32_t qs = m++ & 1;
        for (int i = it.tb; i < it.te; ++i, ++n) {
          const uint32_t s = n & 1;
          if (n >= 2 && !(ok = await(cta, cta.bar(S_FULL + s), ((n >> 1) - 1) & 1, ctl))) break;
          // with an item between, the scores of two tiles ago are past the item before it: its
          // queries' buffer is free
          if (i == it.tb) {
            ++q_armed;
            mbar_arrive_expect_tx(cta.bar(Q_FULL + qs), q_bytes);
            for (int j = 0; j < 3; ++j)
              tma_load_4d(cta.sb + OFF_Q + qs * K_BYTES + j * K_BOX, &maps.q, cta.bar(Q_FULL + qs),
                          32 * j, it.kv * G, it.row0, 0);
          }
          const Tile t = tile_of(it, c, i);
          if (CODES) mbar_arrive(cta.bar(K_CODES + s));
          if (CODES && !t.fresh) continue;
          const Source src(it, t, &maps.k, &maps.pk);
          armed |= 1u << s;
          turn.take(s);
          mbar_arrive_expect_tx(cta.bar(K_FULL + s), K_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + OFF_K + s * K_BYTES + j * K_BOX, src.map, cta.bar(K_FULL + s), 32 * j,
                        it.kv, src.row, src.outer);
        }
      }
      // every armed load has landed before the CTA may exit
      for (int s = 0; s < 2; ++s) {
        if ((armed >> s) & 1) mbar_wait(cta.bar(K_FULL + s), turn.take(s) ^ 1, ctl, DRAIN_NS);
        if (q_armed > s) mbar_wait(cta.bar(Q_FULL + s), ((q_armed - 1 - s) >> 1) & 1, ctl, DRAIN_NS);
      }
    }
  } else if (warp == V_WARP) {
    // ------------------------------------------------------------ TMA: values
    if (lane == 0) {
      int n = 0;
      uint32_t armed = 0;
      Parities turn;
      [[maybe_unused]] int px = 0, pi = n_items ? items[0].tb : 0, pn = 0;  // the prefetches' walk
      bool ok = true;
      for (int x = 0; ok && x < n_items; ++x) {
        const Item& it = items[x];
        for (int i = it.tb; i < it.te; ++i, ++n) {
          const uint32_t s = n & 1;
          if constexpr (CODES) {
            while (px < n_items && pn <= n + AHEAD) {
              if (pi >= items[px].te) {
                if (++px < n_items) pi = items[px].tb;
                continue;
              }
              const Tile t = tile_of(items[px], c, pi);
              if (!t.fresh) {
                tma_prefetch_4d(&maps.pk, 0, items[px].kv, t.s0, items[px].page);
                tma_prefetch_4d(&maps.pv, 0, items[px].kv, t.s0, items[px].page);
              }
              ++pi;
              ++pn;
            }
          }
          if (n >= 2 && !(ok = await(cta, cta.bar(O_DONE + s), ((n >> 1) - 1) & 1, ctl))) break;
          const Tile t = tile_of(it, c, i);
          if (CODES) mbar_arrive(cta.bar(V_CODES + s));
          if (CODES && !t.fresh) continue;
          const Source src(it, t, &maps.v, &maps.pv);
          armed |= 1u << s;
          turn.take(s);
          mbar_arrive_expect_tx(cta.bar(V_FULL + s), V_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + OFF_V + s * V_BYTES + j * V_BOX, src.map, cta.bar(V_FULL + s), 64 * j,
                        it.kv, src.row, src.outer);
        }
      }
      for (int s = 0; s < 2; ++s)
        if ((armed >> s) & 1) mbar_wait(cta.bar(V_FULL + s), turn.take(s) ^ 1, ctl, DRAIN_NS);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t ID_S = idesc_f16(128, 0, BF16, BF16, false, false);
      constexpr uint32_t ID_PV = idesc_f16(128, 192, BF16, BF16, false, true);
      const uint64_t q_desc = smem_desc(cta.sb + OFF_Q, 16, 512, SW_64);
      const uint64_t k_desc = smem_desc(cta.sb + OFF_K, 16, 512, SW_64);
      const uint64_t v_desc = smem_desc(cta.sb + OFF_V, V_BOX, 1024, SW_128);
      // the scores' walk (two tiles ahead) and the values'
      int sx = -1, sn = 0, sm = -1, s_at = 0, vn = 0, vm = -1;
      auto next_item = [&]() -> bool {
        while (++sx < n_items)
          if (items[sx].tb < items[sx].te) {
            ++sm;
            s_at = items[sx].tb;
            return true;
          }
        return false;
      };
      bool s_live = next_item();
      Parities turn;
      // stage s has tile t, the CTA's n-th: keys (what 0) or values (2)
      auto filled = [&](const Tile& t, uint32_t what, uint32_t s, int n) -> bool {
        if (CODES && !await(cta, cta.bar(K_CODES + what + s), (n >> 1) & 1, ctl)) return false;
        return (CODES && !t.fresh) || await(cta, cta.bar(K_FULL + what + s), turn.take(what + s), ctl);
      };
      auto scores = [&]() -> bool {  // S[sn & 1] = Q K^T
        const uint32_t s = sn & 1, qs = sm & 1;
        const Item& it = items[sx];
        if (s_at == it.tb && !await(cta, cta.bar(Q_FULL + qs), (sm >> 1) & 1, ctl)) return false;
        const Tile t = tile_of(it, c, s_at);
        const uint32_t id = ID_S | ((uint32_t)(t.cols >> 3) << 17);
        if (!filled(t, 0, s, sn)) return false;
        tc_fence_after();
        const uint64_t q = q_desc + (qs * K_BYTES >> 4), k = k_desc + (s * K_BYTES >> 4);
#pragma unroll
        for (int j = 0; j < 6; ++j) {  // (the descriptors count in 16 bytes)
          const uint32_t off = ((j >> 1) * K_BOX + (j & 1) * 32) >> 4;
          mma_f16_ss(tmem + TM_S + 128 * s, q + off, k + off, id, j > 0);
        }
        mma_commit(cta.bar(S_FULL + s));
        ++sn;
        if (++s_at == it.te) s_live = next_item();
        return true;
      };
      bool ok = true;
      for (int i = 0; i < 2 && ok && s_live; ++i) ok = scores();
      for (int x = 0; ok && x < n_items; ++x) {
        const Item& it = items[x];
        if (it.tb == it.te) continue;
        ++vm;
        for (int i = it.tb; i < it.te; ++i, ++vn) {
          const uint32_t s = vn & 1;
          if (vn == ctl.stall_step) {  // the give-up path's diagnostic (see chunk_fwd.cu)
            await(cta, cta.bar(DRAIN), 0, ctl);
            ok = false;
            break;
          }
          const Tile t = tile_of(it, c, i);
          const int steps = t.cols >> 4;
          if (!(ok = filled(t, 2, s, vn))) break;
          if (i == it.tb && vm > 0 && !(ok = await(cta, cta.bar(O_FREE), (vm - 1) & 1, ctl))) break;
          if (!(ok = await(cta, cta.bar(P_READY + s), (vn >> 1) & 1, ctl))) break;
          tc_fence_after();
          const uint64_t v = v_desc + (s * V_BYTES >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < steps)
              mma_f16_ts(tmem + TM_O, tmem + TM_S + 128 * s + 8 * j, v + (j * 2048 >> 4), ID_PV,
                         i > it.tb || j > 0);
          mma_commit(cta.bar(O_DONE + s));
          made_step(cta, STEP_TILE, vn + 1);
          if (s_live && !(ok = scores())) break;
        }
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
    float* refs = (float*)(base + OFF_REF);
    float2* sums = (float2*)(base + OFF_SUM);
    int n0 = 0, m = 0;      // tiles and items before this one
    uint32_t v_turn = 0;    // parity of the group's next tile of values that comes by TMA
    bool ok = true;
    for (int x = 0; ok && x < n_items; ++x) {
      const Item& it = items[x];
      if (it.tb == it.te) continue;
      // rows past the item's tokens see nothing; a warp of such rows only keeps step
      const bool live = tok < it.n_tok && row < plan.per * G, awake = tok_a < it.n_tok;
      const bool all_live = tok_b < it.n_tok && 32 * q4 + 31 < plan.per * G;
      const int at = it.i0 + tok, ends = it.i0 + (lane & 4 ? min(tok_b, it.n_tok - 1) : tok_a);
      float ref = -INFINITY, sum = 0.f;  // this row's, as of the group's last tile
      for (int i = it.tb + ((n0 ^ g) & 1); i < it.te; i += 2) {
        const int n = n0 + i - it.tb;
        const Tile t = tile_of(it, c, i);
        // chunks of 32 columns that all rows of the warp see, and that some do: what its first and its
        // last row both see, those between do too; a chunk that neither sees, none does
        uint32_t full = 0, some = 0;
        if (awake) {
          const uint32_t see = columns_seen(it, c, t.fresh, ends, t.s0 + 32 * (lane & 3));
          full = __ballot_sync(0xffffffffu, see == ~0u);
          some = __ballot_sync(0xffffffffu, see != 0u);
          full = all_live ? full & (full >> 4) & 15u : 0u;
          some = (some | (some >> 4)) & 15u;
        }
        if (!(ok = await_warp(cta, cta.bar(S_FULL + g), (n >> 1) & 1, ctl))) break;
        tc_fence_after();
        const uint32_t ts = trow + TM_S + 128 * g;
        auto sees = [&](int j) -> uint32_t {
          return live ? columns_seen(it, c, t.fresh, at, t.s0 + 32 * j) : 0u;
        };
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto maxima = [&](const uint32_t (&z)[32]) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            m4[j & 3] = max3(m4[j & 3], __uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1]));
        };
        if (full == 15u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t z[32];
            tmem_ld32(ts + 32 * j, z);
            tmem_wait_ld();
            maxima(z);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            if (!((some >> j) & 1)) continue;
            uint32_t z[32];
            tmem_ld32(ts + 32 * j, z);
            tmem_wait_ld();
            if (!((full >> j) & 1)) {
              const uint32_t see = sees(j);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see >> e) & 1)) z[e] = 0xFF800000u;  // -inf
            }
            maxima(z);
          }
        }
        const float top = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * kLog2e;
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
          // weights of 32 columns from their scores, as pairs, and their sum
          auto weights = [&](const uint32_t (&z)[32], uint32_t (&p)[16], uint32_t see, bool masked) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 y = fma2(make_float2(__uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1])),
                              l2e, sub2);
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              if (masked) {
                y.x = (see >> (2 * j)) & 1 ? y.x : 0.f;
                y.y = (see >> (2 * j + 1)) & 1 ? y.y : 0.f;
              }
              acc[j & 1] = add2(acc[j & 1], y);
              p[j] = pack2<T>(y.x, y.y);
            }
          };
          // P over the columns of S that have been read
          if (full == 15u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t z[32], p[16];
              tmem_ld32(ts + 32 * j, z);
              tmem_wait_ld();
              weights(z, p, 0u, false);
              tmem_st16(ts + 16 * j, p);
            }
          } else {
#pragma unroll 1
            for (int j = 0; 32 * j < t.cols; ++j) {
              uint32_t p[16];
              if ((some >> j) & 1) {
                uint32_t z[32];
                tmem_ld32(ts + 32 * j, z);
                tmem_wait_ld();
                if ((full >> j) & 1) weights(z, p, 0u, false);
                else weights(z, p, sees(j), true);
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] = 0u;
              }
              tmem_st16(ts + 16 * j, p);
            }
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
        const int kept = t.fresh ? it.tokens - t.s0 : CODES ? BN : it.pos - t.s0;
        const uint32_t v_now = v_turn;
        if (!CODES || t.fresh) v_turn ^= 1;
        if (awake && kept < t.cols) {
          if (!(ok = await_warp(cta, cta.bar(V_FULL + g), v_now, ctl))) break;
          const int step = 32 * min((min(it.n_tok, plan.per) * G + 31) / 32, 4), cnt = (t.cols - kept) * 24;
          for (int y = row; y < cnt; y += step)
            *(uint4*)(base + OFF_V + g * V_BYTES + (y % 24 / 8) * V_BOX + (kept + y / 24) * 128 +
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
    const float2* sums = (const float2*)(base + OFF_SUM);
    uint8_t* const stg = base + OFF_STG + q4 * 4096;
    constexpr int CB = WIDE ? 16 : 32;  // channels of 64 bytes
    int n0 = 0, m = 0, seen = 0, n = 0;  // tiles and items before this one; tiles filled
    bool ok = true;

    // Tile n of the CTA, i of item `it`, if it is one of codes: rows 32 q4 .. + 31 by this warp, a row's
    // 16-byte pieces by adjacent lanes.
    [[maybe_unused]] auto fill = [&](const Item& it, int i) -> bool {
      const uint32_t s = n & 1;
      const Tile t = tile_of(it, c, i);
      const int slots = c.window + c.sink, r0 = t.s0 + 32 * q4, kept = min(it.pos, slots) - r0;
      const long long first = ((long long)it.page * slots + r0) * KV + it.kv;
      uint4 w[6], w2[6];
      float2 sc = make_float2(1.f, 1.f);  // row `lane`: 2^e of its key and value
      auto load = [&](uint4 (&d)[6], const void* p, int pieces, int from) {
#pragma unroll
        for (int j = 0; j < 6; ++j) {
          const int z = (from + j) * 32 + lane, r = z / pieces;
          d[j] = make_uint4(0u, 0u, 0u, 0u);
          if (r < kept)
            d[j] = __ldg(static_cast<const uint4*>(p) + (first + (long long)r * KV) * pieces + z % pieces);
        }
      };
      auto put = [&](const uint4 (&x)[6], uint8_t* dst, int pieces, int from, uint32_t box, int per_box,
                     float scale) {
#pragma unroll
        for (int j = 0; j < 6; ++j) {
          const int z = (from + j) * 32 + lane, r = z / pieces, ch = 2 * (z % pieces);
          const float f = __shfl_sync(0xffffffffu, scale, r);
          uint8_t* const to = dst + ch / per_box * box;
          const int e = ch % per_box, bytes = per_box * 16;
          *(uint4*)(to + swz_off(32 * q4 + r, e, bytes)) = values_of<T>(x[j].x, x[j].y, f);
          *(uint4*)(to + swz_off(32 * q4 + r, e + 1, bytes)) = values_of<T>(x[j].z, x[j].w, f);
        }
        fence_proxy_async();
      };
      if (!t.fresh) {
        load(w, c.k, 6, 0);
        load(w2, c.v, 12, 0);
        if (lane < kept) {
          const unsigned short e = __ldg(reinterpret_cast<const unsigned short*>(a.cache.exps) +
                                         ((long long)it.page * KV + it.kv) * slots + r0 + lane);
          sc = make_float2(scale_of((signed char)(e & 255)), scale_of((signed char)(e >> 8)));
        }
      }
      if (n >= 2 && !await_warp(cta, cta.bar(S_FULL + s), ((n >> 1) - 1) & 1, ctl)) return false;
      if (!t.fresh) put(w, base + OFF_K + s * K_BYTES, 6, 0, K_BOX, 4, sc.x);
      mbar_arrive(cta.bar(K_CODES + s));
      if (!t.fresh) load(w, c.v, 12, 6);
      if (n >= 2 && !await_warp(cta, cta.bar(O_DONE + s), ((n >> 1) - 1) & 1, ctl)) return false;
      if (!t.fresh) {
        put(w2, base + OFF_V + s * V_BYTES, 12, 0, V_BOX, 8, sc.y);
        put(w, base + OFF_V + s * V_BYTES, 12, 6, V_BOX, 8, sc.y);
      }
      mbar_arrive(cta.bar(V_CODES + s));
      ++n;
      return true;
    };
    [[maybe_unused]] int fx = 0, fi = n_items ? items[0].tb : 0;  // the next tile to fill
    // Fills up to tile `stop` of item `upto`.
    [[maybe_unused]] auto fill_to = [&](int upto, int stop) -> bool {
      while (fx < n_items && fx <= upto) {
        const int end = fx < upto ? items[fx].te : min(stop, items[fx].te);
        for (; fi < end; ++fi)
          if (!fill(items[fx], fi)) return false;
        if (fx == upto) break;
        if (++fx < n_items) fi = items[fx].tb;
      }
      return true;
    };

    for (int x = 0; x < n_items; ++x) {
      const Item& it = items[x];
      const bool live_item = it.tb < it.te;
      if constexpr (CODES) {
        // all of this item's tiles, and the first two of the next one that has any
        int next = x + 1;
        while (next < n_items && items[next].tb == items[next].te) ++next;
        if (!(ok = fill_to(x, it.te))) break;
        if (next < n_items && !(ok = fill_to(next, items[next].tb + 2))) break;
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
        const Partials ps(a.workspace, plan.units, plan.parts);
        // this part's place: the CTA's items are blockIdx.x, + gridDim.x, ..
        const long long at = (blockIdx.x + (long long)x * gridDim.x) * BM;
        if (row < rows) ps.ml[at + row] = make_float2(ref, sum);
        out = ps.o + at * kDV;
      } else {
        out = static_cast<TO*>(a.o) + ((long long)it.row0 * a.H + it.kv * G) * kDV;
      }
      if (live_item) {
        const bool awake = 32 * q4 < rows;
        // 32 rows of 128 bytes at a time go through shared memory, so that eight lanes write a row
#pragma unroll 1
        for (int k = 0; k < kDV / (2 * CB); ++k) {
          if (awake) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t o[CB];
              if constexpr (WIDE) tmem_ld16(trow + TM_O + CB * (2 * k + e), o);
              else tmem_ld32(trow + TM_O + CB * (2 * k + e), o);
              tmem_wait_ld();
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if constexpr (WIDE) {
                    w[j] = __float_as_uint(__uint_as_float(o[4 * ch + j]) * inv);
                  } else {
                    const float lo = __uint_as_float(o[8 * ch + 2 * j]) * inv;
                    const float hi = __uint_as_float(o[8 * ch + 2 * j + 1]) * inv;
                    w[j] = pack2<TO>(lo, hi);
                  }
                }
                *(uint4*)(stg + swz_off(lane, 4 * e + ch, 128)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          if (k == kDV / (2 * CB) - 1) {
            tc_fence_before();
            mbar_arrive(cta.bar(O_FREE));
          }
          if (awake) {
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              const int r = 4 * ch + (lane >> 3), rr = 32 * q4 + r;
              const uint4 y = *(const uint4*)(stg + swz_off(r, lane & 7, 128));
              if (rr < rows) {
                const long long to = SPLIT ? rr : (long long)(rr / G) * a.H + rr % G;
                reinterpret_cast<uint4*>(out + to * kDV + 2 * CB * k)[lane & 7] = y;
              }
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

// One warp per row of a cut unit: o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p, in order.
template <class TO>
__global__ void __launch_bounds__(256)
window_chunk_join_kernel(ChunkArgs a, Plan plan) {
  griddep_wait();
  const Partials ps(a.workspace, plan.units, plan.parts);
  const int KV = a.cache.c.KV, G = a.H / KV, lane = threadIdx.x & 31;
  const int unit = blockIdx.x, t = unit / KV, kv = unit % KV, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (t >= ps.tiles[0]) return;
  const int row0 = ps.tiles[2 + 2 * t];
  if (row >= ps.tiles[3 + 2 * t] * G) return;
  const long long at = (long long)unit * plan.parts * BM + row;
  float top = -INFINITY;
  for (int p = 0; p < plan.parts; ++p) top = fmaxf(top, ps.ml[at + (long long)p * BM].x);
  float sum = 0.f, o[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < plan.parts; ++p) {
    const float2 ml = ps.ml[at + (long long)p * BM];
    if (ml.x == -INFINITY) continue;  // a part that this row sees nothing of
    const float f = ex2(ml.x - top);
    sum = fmaf(f, ml.y, sum);
    const float2* src = reinterpret_cast<const float2*>(ps.o + (at + (long long)p * BM) * kDV);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const float2 y = src[32 * j + lane];
      o[2 * j] = fmaf(f, y.x, o[2 * j]);
      o[2 * j + 1] = fmaf(f, y.y, o[2 * j + 1]);
    }
  }
  const float inv = 1.f / sum;  // the token itself is in one of the parts: sum > 0
  TO* out = static_cast<TO*>(a.o) + (((long long)row0 + row / G) * a.H + kv * G + row % G) * kDV;
#pragma unroll
  for (int j = 0; j < 3; ++j) store2(out + 64 * j + 2 * lane, o[2 * j] * inv, o[2 * j + 1] * inv);
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
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  kern<<<plan.grid, THREADS, SMEM_BYTES, stream>>>(maps, a, plan, ctl);
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
  if (CODES)
    ok = ok &&
         make_map(&m.pk, c.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kDK, c.KV, slots, pages, kDK, 1, BN,
                  CU_TENSOR_MAP_SWIZZLE_NONE) &&
         make_map(&m.pv, c.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kDV, c.KV, slots, pages, kDV, 1, BN,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
  else
    ok = ok &&
         make_map(&m.pk, c.k, type, 2, kDK, c.KV, slots, pages, 32, 1, BN, CU_TENSOR_MAP_SWIZZLE_64B) &&
         make_map(&m.pv, c.v, type, 2, kDV, c.KV, slots, pages, 64, 1, BN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  if (plan.parts > 1) return launch<T, float, CODES, true>(m, a, plan, ctl, stream);
  if (a.out_type == GLA_FP32) return launch<T, float, CODES, false>(m, a, plan, ctl, stream);
  return launch<T, T, CODES, false>(m, a, plan, ctl, stream);
}

cudaError_t launch8(const ChunkArgs& a, const Plan& plan, DevCtl ctl, cudaStream_t stream);

}  // namespace chunk
}  // namespace gla
