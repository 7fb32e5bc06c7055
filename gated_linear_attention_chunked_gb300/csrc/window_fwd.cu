// window_fwd.cu -- causal softmax attention over the last `window` tokens and the first `sink`
// ones, 96 key and 192 value channels per head, H query heads on KV key heads:
//
//   z_ts = q_t . k_s,   lse_t = ln sum_s exp(z_ts),   o_t = sum_s exp(z_ts - lse_t) v_s
//
// over the s <= t with t - s < window or s < sink.  One pass over the keys: a row keeps a
// reference m and the sum l of exp(z - m), and what was summed is rescaled only when a tile's
// maximum passes m by more than 8 in base 2 (weights up to 2^8 lose nothing in either 16-bit
// type, and l and o are fp32), so the rescaling of o in tensor memory is rare.
//
// A persistent grid of one CTA per SM; an item is 128 queries of one head, walked in tiles of 128
// keys: first the ones that hold sinks (only as many columns as there are sinks, rounded to 16),
// then the window's.
//   warps 0..7   softmax, two groups of four warps that take the tiles in turn (thread = row, one
//                warp per 32 queries): mask, maximum, exp2, weights as 16-bit pairs into tensor
//                memory.  The reference goes from group to group as soon as a tile's maximum is
//                known, so that the two work on two tiles at once
//   warp 8       TMA loads of queries and keys (3 boxes of 32 channels, 64-byte swizzle)
//   warp 9       TMA loads of values (3 boxes of 64 channels, 128-byte swizzle)
//   warp 10      tcgen05 issuer and TMEM owner: S = Q K^T into one of two score buffers, O += P V
//                with P from tensor memory
//   warps 11..14 the output rows of an item, while the softmax is on the next one
// The scores run two tiles ahead of the values (and across items), so that the tensor cores go
// from P V of a tile to the scores of the next but one while the softmax works on the tile
// between.  P takes the place of the scores it came from: products run in the order of their
// issue, so the next scores there come behind the P V that reads it, and a group writes P without
// waiting for the P V of the tile before.  A tile's scores and sums are each one commit, which also
// frees the key and value buffers.
//
// Bound by a tile's chain: its P V (770 cycles), the scores two tiles on behind it (380), their
// softmax (1,800) and the hand-overs take 3,550 cycles for two tiles, 1,775 a tile where the products
// take 1,150; between items, by the wait for the output rows.  Measured, bf16, B=8 T=2048, 16 heads,
// window 512, 4 sinks: 107.5 us, 2.4 times the copy of its bytes (110.4 before the waits of
// window_wait.cuh, with which fewer registers spill); then 126 with P in columns of its own, 117 with
// masks decided by votes of the warp instead of by the tile's position.  No faster: the
// next scores ahead of P V (120), output rows held in registers (spills, 127), tiles of a sequence
// from the last (130: the keys' tiles then leave the L2 between their readers).
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

constexpr int BM = 128, BN = 128;
constexpr uint32_t K_BOX = 8192, V_BOX = 16384;  // 128 rows x 64 B, x 128 B
constexpr uint32_t K_BYTES = 3 * K_BOX, V_BYTES = 3 * V_BOX;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * K_BYTES, OFF_V = 4 * K_BYTES;
constexpr uint32_t OFF_STG = OFF_V + 2 * V_BYTES;  // output staging, 4 KB per output warp
constexpr uint32_t OFF_REF = OFF_STG + 4 * 4096;   // float ref[2][128]: each group's reference
constexpr uint32_t OFF_SUM = OFF_REF + 1024;       // float2 sum[2][2][128]: (sum, ref), by item
constexpr uint32_t OFF_BAR = OFF_SUM + 4096;
enum Bar : uint32_t {  // +stage (+4 group + quadrant, + quadrant) where there are several
  Q_FULL = 0, K_FULL = 2, V_FULL = 4,
  S_FULL = 6,    // a tile's scores are in tensor memory (and its keys have been read)
  O_DONE = 8,    // O += P V has run: P, V and O are free to touch
  P_READY = 10,  // +group: P has been written (over its S)
  O_FREE = 12,   // the output rows have been read
  DRAIN = 13,
  REF = 14,      // a group's references of a tile are known
  SUM = 22,      // both groups' sums of an item are known
  NBAR = 26
};
constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t SMEM_USED = OFF_ABORT + 4 * kWaitWords, SMEM_BYTES = SMEM_USED + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

// Columns: S twice 128, O 192.  A tile's P takes the place of its S, from the front.
constexpr uint32_t TM_S = 0, TM_O = 256;

constexpr int GROUP = 128, K_WARP = 8, V_WARP = 9, MMA_WARP = 10, OUT_WARP = 11;
constexpr int THREADS = 15 * 32;

// The items of a CTA, blockIdx.x, + gridDim.x, ...: heads fastest, then tiles of a sequence.  The
// step is added digit by digit, so that an item costs no division.
struct Items {
  const WindowArgs& a;
  int tiles, dh, dj, db;   // tiles of a sequence; the step's heads, tiles and sequences
  int b, h, j, q0, len;    // (the host keeps the count of items below 2^30)
  __device__ Items(const WindowArgs& a_) : a(a_) {
    tiles = (a.T + BM - 1) / BM;
    const int s = gridDim.x / a.H, i = blockIdx.x / a.H;
    dh = gridDim.x - s * a.H;
    db = s / tiles;
    dj = s - db * tiles;
    // one step ahead of the first
    h = (int)blockIdx.x - i * a.H - dh;
    b = i / tiles - db;
    j = i % tiles - dj;
  }
  __device__ bool next() {
    h += dh;
    j += dj;
    b += db;
    if (h >= a.H) { h -= a.H; ++j; }
    if (j >= tiles) { j -= tiles; ++b; }
    if (b >= a.B) return false;
    q0 = j * BM;
    len = a.T;
    if (a.lens) len = min(max(__ldg(a.lens + b), 0), a.T);
    return true;
  }
  // the next item that has a live query
  __device__ bool next_live() {
    while (next())
      if (q0 < len) return true;
    return false;
  }
  __device__ KeyTiles keys() const { return KeyTiles(q0, min(q0 + BM, len), BN, a.window, a.sink); }
};
// Columns of key tile i: all, or of a tile in front of the window only those that hold sinks.
__device__ __forceinline__ int tile_cols(const KeyTiles& kt, int i, int sink) {
  return i < kt.far ? min(BN, (sink - kt.tile(i) * BN + 15) & ~15) : BN;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <class T, class TO>
__global__ void __launch_bounds__(THREADS, 1)
window_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, WindowArgs a, DevCtl ctl) {
  constexpr bool BF16 = !__is_same(T, __half), WIDE = sizeof(TO) == 4;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Cta cta;
  cta.base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  cta.sb = smem_u32(cta.base);
  cta.bar_off = OFF_BAR;
  cta.abort_off = OFF_ABORT;
  uint8_t* const base = cta.base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* tmem_slot = (uint32_t*)(base + OFF_TMEM);
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
    for (uint32_t q = SUM; q < NBAR; ++q) mbar_init(cta.bar(q), 64);
    for (uint32_t i = 0; i < kWaitWords; ++i) cta.abort_flag()[i] = 0;
    fence_barrier_init();
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = a.H / a.KV;

  if (warp == K_WARP) {
    // ------------------------------------------------------------ TMA: queries and keys
    if (lane == 0) {
      Items it(a);
      int n = 0, m = 0, q_armed = 0;  // key tiles and items so far
      bool ok = true;
      for (; ok && it.next_live(); ++m) {
        const uint32_t qs = m & 1;
        const KeyTiles kt = it.keys();
        for (int i = 0; i < kt.n; ++i, ++n) {
          const uint32_t s = n & 1;
          if (n >= 2 && !(ok = await(cta, cta.bar(S_FULL + s), ((n >> 1) - 1) & 1, ctl))) break;
          // with an item between, the scores of two tiles ago are past the item before it: its
          // queries' buffer is free
          if (i == 0) {
            ++q_armed;
            mbar_arrive_expect_tx(cta.bar(Q_FULL + qs), K_BYTES);
            for (int j = 0; j < 3; ++j)
              tma_load_4d(cta.sb + OFF_Q + qs * K_BYTES + j * K_BOX, &map_q, cta.bar(Q_FULL + qs),
                          32 * j, it.h, it.q0, it.b);
          }
          mbar_arrive_expect_tx(cta.bar(K_FULL + s), K_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + OFF_K + s * K_BYTES + j * K_BOX, &map_k, cta.bar(K_FULL + s),
                        32 * j, it.h / G, kt.tile(i) * BN, it.b);
        }
      }
      // every armed load has landed before the CTA may exit
      for (int s = 0; s < 2; ++s) {
        if (n > s) mbar_wait(cta.bar(K_FULL + s), ((n - 1 - s) >> 1) & 1, ctl, DRAIN_NS);
        if (q_armed > s) mbar_wait(cta.bar(Q_FULL + s), ((q_armed - 1 - s) >> 1) & 1, ctl, DRAIN_NS);
      }
    }
  } else if (warp == V_WARP) {
    // ------------------------------------------------------------ TMA: values
    if (lane == 0) {
      Items it(a);
      int n = 0;
      bool ok = true;
      while (ok && it.next_live()) {
        const KeyTiles kt = it.keys();
        for (int i = 0; i < kt.n; ++i, ++n) {
          const uint32_t s = n & 1;
          if (n >= 2 && !(ok = await(cta, cta.bar(O_DONE + s), ((n >> 1) - 1) & 1, ctl))) break;
          mbar_arrive_expect_tx(cta.bar(V_FULL + s), V_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + OFF_V + s * V_BYTES + j * V_BOX, &map_v, cta.bar(V_FULL + s),
                        64 * j, it.h / G, kt.tile(i) * BN, it.b);
        }
      }
      for (int s = 0; s < 2; ++s)
        if (n > s) mbar_wait(cta.bar(V_FULL + s), ((n - 1 - s) >> 1) & 1, ctl, DRAIN_NS);
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
      Items si(a), vi(a);
      KeyTiles sk(0, 1, BN, 1, 0), vk(0, 1, BN, 1, 0);
      int sn = 0, sm = -1, s_at = 0, vn = 0, vm = -1, v_at = 0;
      bool s_live = si.next_live();
      if (s_live) { sk = si.keys(); ++sm; }
      auto scores = [&]() -> bool {  // S[sn & 1] = Q K^T
        const uint32_t s = sn & 1, qs = sm & 1;
        if (s_at == 0 && !await(cta, cta.bar(Q_FULL + qs), (sm >> 1) & 1, ctl)) return false;
        if (!await(cta, cta.bar(K_FULL + s), (sn >> 1) & 1, ctl)) return false;
        tc_fence_after();
        const uint32_t id = ID_S | ((uint32_t)(tile_cols(sk, s_at, a.sink) >> 3) << 17);
        const uint64_t q = q_desc + (qs * K_BYTES >> 4), k = k_desc + (s * K_BYTES >> 4);
#pragma unroll
        for (int c = 0; c < 6; ++c) {  // (the descriptors count in 16 bytes)
          const uint32_t off = ((c >> 1) * K_BOX + (c & 1) * 32) >> 4;
          mma_f16_ss(tmem + TM_S + 128 * s, q + off, k + off, id, c > 0);
        }
        mma_commit(cta.bar(S_FULL + s));
        ++sn;
        if (++s_at == sk.n) {
          s_at = 0;
          if ((s_live = si.next_live())) { sk = si.keys(); ++sm; }
        }
        return true;
      };
      bool ok = true;
      for (int i = 0; i < 2 && ok && s_live; ++i) ok = scores();
      while (ok && vi.next_live()) {
        vk = vi.keys();
        ++vm;
        for (v_at = 0; v_at < vk.n; ++v_at, ++vn) {
          const uint32_t s = vn & 1;
          if (vn == ctl.stall_step) {  // the give-up path's diagnostic (see chunk_fwd.cu)
            await(cta, cta.bar(DRAIN), 0, ctl);
            ok = false;
            break;
          }
          if (!(ok = await(cta, cta.bar(V_FULL + s), (vn >> 1) & 1, ctl))) break;
          if (v_at == 0 && vm > 0 &&
              !(ok = await(cta, cta.bar(O_FREE), (vm - 1) & 1, ctl))) break;
          if (!(ok = await(cta, cta.bar(P_READY + s), (vn >> 1) & 1, ctl))) break;
          tc_fence_after();
          const uint64_t v = v_desc + (s * V_BYTES >> 4);
          const int steps = tile_cols(vk, v_at, a.sink) >> 4;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < steps)
              mma_f16_ts(tmem + TM_O, tmem + TM_S + 128 * s + 8 * c, v + (c * 2048 >> 4), ID_PV,
                         v_at > 0 || c > 0);
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
    float* refs = (float*)(base + OFF_REF);
    float2* sums = (float2*)(base + OFF_SUM);
    Items it(a);
    int n0 = 0;  // tiles before this item
    bool ok = true;
    for (int m = 0; ok && it.next_live(); ++m) {
      const int t = it.q0 + row, len = it.len;
      float ref = -INFINITY, sum = 0.f;  // this row's, as of the group's last tile
      const KeyTiles kt = it.keys();
      for (int i = (n0 ^ g) & 1; i < kt.n; i += 2) {
        const int n = n0 + i, s0 = kt.tile(i) * BN;
        const bool whole = s0 + BN - 1 <= it.q0 && s0 + BN <= len &&
                           (it.q0 + BM - 1 - s0 < a.window || s0 + BN <= a.sink);
        // The columns of the tile that some row of the warp sees lie in chunks (of 32) ca .. cb - 1;
        // chunk c is seen by all if full(c).  Chunks from `cols` on are not multiplied.
        const int t0 = it.q0 + 32 * q4, cols = tile_cols(kt, i, a.sink);
        const int ca = s0 < a.sink ? 0 : max(0, t0 - a.window + 1 - s0) >> 5;
        const int cb = (min(min(t0 + 31, len - 1) - s0, cols - 1) >> 5) + 1;
        auto full = [&](int c) {
          const int c0 = s0 + 32 * c;
          return c0 + 31 <= min(t0, len - 1) && (t0 + 31 - c0 < a.window || c0 + 31 < a.sink);
        };
        // the columns 32 c .. that this row sees
        auto sees = [&](int c) -> uint32_t {
          return keys_seen(t, s0 + 32 * c, len, a.window, a.sink);
        };
        if (!(ok = await_warp(cta, cta.bar(S_FULL + g), (n >> 1) & 1, ctl))) break;
        tc_fence_after();
        const uint32_t ts = trow + TM_S + 128 * g;
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto maxima = [&](const uint32_t (&z)[32]) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            m4[j & 3] = max3(m4[j & 3], __uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1]));
        };
        if (whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t z[32];
            tmem_ld32(ts + 32 * c, z);
            tmem_wait_ld();
            maxima(z);
          }
        } else {
#pragma unroll 1
          for (int c = ca; c < cb; ++c) {
            uint32_t z[32];
            tmem_ld32(ts + 32 * c, z);
            tmem_wait_ld();
            if (!full(c)) {
              const uint32_t see = sees(c);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((see >> j) & 1)) z[j] = 0xFF800000u;  // -inf
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
        const float before = i > 0 ? refs[(g ^ 1) * 128 + row] : -INFINITY;
        // a row that has seen nothing yet has o = 0 and takes any scale
        const float now = top > before + 8.f ? top : before;
        refs[g * 128 + row] = now;
        mbar_arrive(cta.bar(REF + 4 * g + q4));
        const float scale = now == before || before == -INFINITY ? 1.f : ex2(before - now);
        if (now != ref) sum = ref == -INFINITY ? 0.f : sum * ex2(ref - now);
        ref = now;
        const float sub = ref == -INFINITY ? 0.f : -ref;
        const float2 sub2 = make_float2(sub, sub), l2e = make_float2(kLog2e, kLog2e);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // weights of 32 columns from their scores, as pairs, and their sum
        auto weights = [&](const uint32_t (&z)[32], uint32_t (&p)[16], uint32_t see, bool masked) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 x = fma2(make_float2(__uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1])),
                            l2e, sub2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            if (masked) {
              x.x = (see >> (2 * j)) & 1 ? x.x : 0.f;
              x.y = (see >> (2 * j + 1)) & 1 ? x.y : 0.f;
            }
            acc[j & 1] = add2(acc[j & 1], x);
            p[j] = pack2<T>(x.x, x.y);
          }
        };
        // P over the columns of S that have been read
        if (whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t z[32], p[16];
            tmem_ld32(ts + 32 * c, z);
            tmem_wait_ld();
            weights(z, p, 0u, false);
            tmem_st16(ts + 16 * c, p);
          }
        } else {
#pragma unroll 1
          for (int c = 0; 32 * c < cols; ++c) {
            uint32_t p[16];
            if (c >= ca && c < cb) {
              uint32_t z[32];
              tmem_ld32(ts + 32 * c, z);
              tmem_wait_ld();
              if (full(c)) weights(z, p, 0u, false);
              else weights(z, p, sees(c), true);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) p[j] = 0u;
            }
            tmem_st16(ts + 16 * c, p);
          }
        }
        acc[0] = add2(acc[0], acc[1]);
        sum += acc[0].x + acc[0].y;
        if (i > 0 && __any_sync(0xffffffffu, scale != 1.f)) {
          // O once the tile before has been added (and the one before that, whose phase of the
          // barrier this could be taken for, is: this tile's scores came behind it)
          if (!(ok = await_warp(cta, cta.bar(O_DONE + (g ^ 1)), ((n - 1) >> 1) & 1, ctl))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 6; ++c) {
            uint32_t o[32];
            tmem_ld32(trow + TM_O + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * scale);
            tmem_st32(trow + TM_O + 32 * c, o);
          }
        }
        if (s0 + BN > len && len < a.T) {
          // values of padding may be anything, and 0 x NaN is NaN: zero their rows
          if (!(ok = await_warp(cta, cta.bar(V_FULL + g), (n >> 1) & 1, ctl))) break;
          const int r0 = len - s0, cnt = (BN - r0) * 24;
          for (int x = row; x < cnt; x += GROUP)
            *(uint4*)(base + OFF_V + g * V_BYTES + (x % 24 / 8) * V_BOX + (r0 + x / 24) * 128 +
                      (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(cta.bar(P_READY + g));
      }
      if (!ok) break;
      n0 += kt.n;
      // one item at a time: the output warps have taken the sums of the item before
      if (m > 0 && !(ok = await_warp(cta, cta.bar(O_FREE), (m - 1) & 1, ctl))) break;
      sums[(m & 1) * 256 + g * 128 + row] = make_float2(sum, ref);
      mbar_arrive(cta.bar(SUM + q4));
    }
  } else {
    // ------------------------------------------------------------ output rows
    const int q4 = warp & 3, row = 32 * q4 + lane;  // the quadrant that the warp may read
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    const float2* sums = (const float2*)(base + OFF_SUM);
    uint8_t* const stg = base + OFF_STG + q4 * 4096;
    constexpr int CB = WIDE ? 16 : 32;  // channels of 64 bytes
    Items it(a);
    int n0 = 0, m = 0, seen = 0;
    while (it.next()) {
      const int t = it.q0 + row;
      const bool live_item = it.q0 < it.len, live = t < it.len;
      if (a.lens && it.q0 == 0 && it.h == 0 && tid == OUT_WARP * 32 &&
          __ldg(a.lens + it.b) != it.len)
        record_error(ctl, DEV_RANGE);  // outside [0, T]: read as the nearer end
      float ref = -INFINITY, sum = 0.f;
      if (live_item) {
        n0 += it.keys().n;
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
      const float inv = live ? 1.f / sum : 0.f;
      TO* const out =
          static_cast<TO*>(a.o) + (((long long)it.b * a.T + it.q0 + 32 * q4) * a.H + it.h) * kDV;
      // 32 rows of 128 bytes at a time go through shared memory, so that eight lanes write a row
#pragma unroll 1
      for (int k = 0; k < kDV / (2 * CB); ++k) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t o[CB];
          if (live_item) {
            if constexpr (WIDE) tmem_ld16(trow + TM_O + CB * (2 * k + e), o);
            else tmem_ld32(trow + TM_O + CB * (2 * k + e), o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (WIDE) {
                w[j] = live ? __float_as_uint(__uint_as_float(o[4 * c + j]) * inv) : 0u;
              } else {
                const float lo = __uint_as_float(o[8 * c + 2 * j]) * inv;
                const float hi = __uint_as_float(o[8 * c + 2 * j + 1]) * inv;
                w[j] = live ? pack2<TO>(lo, hi) : 0u;
              }
            }
            *(uint4*)(stg + swz_off(lane, 4 * e + c, 128)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (k == kDV / (2 * CB) - 1 && live_item) {
          tc_fence_before();
          mbar_arrive(cta.bar(O_FREE));
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int r = 4 * c + (lane >> 3);
          const uint4 x = *(const uint4*)(stg + swz_off(r, lane & 7, 128));
          if (it.q0 + 32 * q4 + r < a.T)
            reinterpret_cast<uint4*>(out + (long long)r * a.H * kDV + 2 * CB * k)[lane & 7] = x;
        }
      }
      if (a.lse && t < a.T)
        a.lse[((long long)it.b * a.H + it.h) * a.T + t] =
            live ? (ref + log2f(sum)) * kLn2 : -INFINITY;
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

template <class T, class TO>
cudaError_t run(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  constexpr bool bf16 = !__is_same(T, __half);
  CUtensorMap mq, mk, mv;
  if (!make_tmap_seq_16bit(&mq, a.q, kDK, a.H, a.T, a.B, 32, BM, CU_TENSOR_MAP_SWIZZLE_64B, bf16) ||
      !make_tmap_seq_16bit(&mk, a.k, kDK, a.KV, a.T, a.B, 32, BN, CU_TENSOR_MAP_SWIZZLE_64B, bf16) ||
      !make_tmap_seq_16bit(&mv, a.v, kDV, a.KV, a.T, a.B, 64, BN, CU_TENSOR_MAP_SWIZZLE_128B, bf16))
    return cudaErrorInvalidValue;
  auto kern = window_fwd_kernel<T, TO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.B * a.H * ((a.T + BM - 1) / BM);
  kern<<<(unsigned)std::min<long long>(items, n_sm), THREADS, SMEM_BYTES, stream>>>(
      mq, mk, mv, a, ctl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const bool wide = a.out_type == GLA_FP32;
  if (a.in_type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, n_sm, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, n_sm, ctl, stream);
  return wide ? run<__half, float>(a, n_sm, ctl, stream) : run<__half, __half>(a, n_sm, ctl, stream);
}

}  // namespace gla
