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
//   warps 0..7   softmax, two per row quadrant of 32 queries, each with 64 of the 128 columns of
//                a tile of scores (thread = row): mask, maximum (joined by the two through shared
//                memory), exp2, weights as 16-bit pairs into tensor memory; after the item's last
//                tile the output rows, TMA-stored
//   warp 8       TMA loads of queries and keys (3 boxes of 32 channels, 64-byte swizzle)
//   warp 9       TMA loads of values (3 boxes of 64 channels, 128-byte swizzle)
//   warp 10      tcgen05 issuer and TMEM owner: S = Q K^T into one of two score buffers, O += P V
//                with P from tensor memory
// The scores run two tiles ahead of the values (and across items), so that the tensor cores go
// from P V of a tile to the scores of the next but one while the softmax works on the tile
// between; P has columns of its own, so neither waits for the other's reads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "scan_common.cuh"
#include "tmap.h"
#include "window_common.cuh"

namespace gla {
namespace {

using scan::Cta;
using scan::DRAIN_NS;
using scan::wait;
using scan::wait_warp;

constexpr int BM = 128, BN = 128;
constexpr uint32_t K_BOX = 8192, V_BOX = 16384;  // 128 rows x 64 B, x 128 B
constexpr uint32_t K_BYTES = 3 * K_BOX, V_BYTES = 3 * V_BOX;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * K_BYTES, OFF_V = 4 * K_BYTES;
constexpr uint32_t OFF_STG = OFF_V + 2 * V_BYTES;  // output staging, 2 KB per softmax warp
constexpr uint32_t OFF_EX = OFF_STG + 8 * 2048;    // float ex[2][2][128]: halves' row maxima
constexpr uint32_t OFF_EL = OFF_EX + 2048;         // float el[2][128]: halves' row sums
constexpr uint32_t OFF_BAR = OFF_EL + 1024;
constexpr uint32_t NBAR = 27;
constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t SMEM_USED = OFF_ABORT + 4, SMEM_BYTES = SMEM_USED + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

constexpr uint32_t TM_S = 0, TM_O = 256, TM_P = 448;  // columns: S 2 x 128, O 192, P 64

enum Bar : uint32_t {  // +stage where two
  Q_FULL = 0, Q_EMPTY = 2, K_FULL = 4, K_EMPTY = 6, V_FULL = 8, V_EMPTY = 10, S_FULL = 12,
  P_READY = 14,  // the softmax group has written P (and read S)
  O_DONE = 15,   // O += P V has run (P, V and O are free to touch)
  O_FREE = 16,   // the output rows have been read
  DRAIN = 17,
  PX = 18,       // 18..21: quadrant's two warps have their row maxima
  PL = 22,       // 22..25: ... their row sums
};
constexpr int SM_WARPS = 8, K_WARP = 8, V_WARP = 9, MMA_WARP = 10, THREADS = 11 * 32;

// The items of a CTA, blockIdx.x, + gridDim.x, ...: heads fastest, then tiles of a sequence.
struct Items {
  const WindowArgs& a;
  const DevCtl& ctl;
  long long at, total;
  int tiles;
  int b, h, q0, len;
  __device__ Items(const WindowArgs& a_, const DevCtl& c) : a(a_), ctl(c) {
    tiles = (a.T + BM - 1) / BM;
    total = (long long)a.B * tiles * a.H;
    at = (long long)blockIdx.x - gridDim.x;
  }
  __device__ bool next() {
    at += gridDim.x;
    if (at >= total) return false;
    h = (int)(at % a.H);
    const long long r = at / a.H;
    b = (int)(r / tiles);
    q0 = (int)(r % tiles) * BM;
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
// Bits 0 .. n of a 64-bit word (none for n < 0).
__device__ __forceinline__ uint64_t bits_to(int n) {
  return n < 0 ? 0ull : n >= 63 ? ~0ull : (2ull << n) - 1;
}

template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(THREADS, 1)
window_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ CUtensorMap map_o, WindowArgs a, DevCtl ctl) {
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
    mbar_init(cta.bar(P_READY), SM_WARPS * 32);
    mbar_init(cta.bar(O_DONE), 1);
    mbar_init(cta.bar(O_FREE), SM_WARPS * 32);
    mbar_init(cta.bar(DRAIN), 1);
    for (uint32_t q = 0; q < 4; ++q) {
      mbar_init(cta.bar(PX + q), 64);
      mbar_init(cta.bar(PL + q), 64);
    }
    *cta.abort_flag() = 0;
    fence_barrier_init();
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
    prefetch_tensormap(&map_o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = a.H / a.KV;

  if (warp == K_WARP) {
    // ------------------------------------------------------------ TMA: queries and keys
    if (lane == 0) {
      Items it(a, ctl);
      int n = 0, m = 0;  // key tiles and items so far
      bool ok = true;
      for (; ok && it.next_live(); ++m) {
        const uint32_t qs = m & 1;
        if (m >= 2 && !wait(cta, cta.bar(Q_EMPTY + qs), ((m >> 1) - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(cta.bar(Q_FULL + qs), K_BYTES);
        for (int j = 0; j < 3; ++j)
          tma_load_4d(cta.sb + OFF_Q + qs * K_BYTES + j * K_BOX, &map_q, cta.bar(Q_FULL + qs),
                      32 * j, it.h, it.q0, it.b);
        const KeyTiles kt = it.keys();
        for (int i = 0; i < kt.n; ++i, ++n) {
          const uint32_t s = n & 1;
          if (n >= 2 && !(ok = wait(cta, cta.bar(K_EMPTY + s), ((n >> 1) - 1) & 1, ctl))) break;
          mbar_arrive_expect_tx(cta.bar(K_FULL + s), K_BYTES);
          for (int j = 0; j < 3; ++j)
            tma_load_4d(cta.sb + OFF_K + s * K_BYTES + j * K_BOX, &map_k, cta.bar(K_FULL + s),
                        32 * j, it.h / G, kt.tile(i) * BN, it.b);
        }
      }
      // every armed load has landed before the CTA may exit
      for (int s = 0; s < 2; ++s) {
        if (n > s) mbar_wait(cta.bar(K_FULL + s), ((n - 1 - s) >> 1) & 1, ctl, DRAIN_NS);
        if (m > s) mbar_wait(cta.bar(Q_FULL + s), ((m - 1 - s) >> 1) & 1, ctl, DRAIN_NS);
      }
    }
  } else if (warp == V_WARP) {
    // ------------------------------------------------------------ TMA: values
    if (lane == 0) {
      Items it(a, ctl);
      int n = 0;
      bool ok = true;
      while (ok && it.next_live()) {
        const KeyTiles kt = it.keys();
        for (int i = 0; i < kt.n; ++i, ++n) {
          const uint32_t s = n & 1;
          if (n >= 2 && !(ok = wait(cta, cta.bar(V_EMPTY + s), ((n >> 1) - 1) & 1, ctl))) break;
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
    if (lane == 0) {
      constexpr uint32_t ID_PV = idesc_f16(128, 192, BF16, BF16, false, true);
      // the scores' walk (two tiles ahead) and the values'
      Items si(a, ctl), vi(a, ctl);
      KeyTiles sk(0, 1, BN, 1, 0), vk(0, 1, BN, 1, 0);
      int sn = 0, sm = -1, s_at = 0, vn = 0, vm = -1, v_at = 0;
      bool s_live = si.next_live();
      if (s_live) { sk = si.keys(); ++sm; }
      auto scores = [&]() -> bool {  // S[sn & 1] = Q K^T
        const uint32_t s = sn & 1, qs = sm & 1;
        if (s_at == 0 && !wait(cta, cta.bar(Q_FULL + qs), (sm >> 1) & 1, ctl)) return false;
        if (!wait(cta, cta.bar(K_FULL + s), (sn >> 1) & 1, ctl)) return false;
        tc_fence_after();
        const uint32_t id = idesc_f16(128, 128, BF16, BF16, false, false) & ~(0x3Fu << 17);
        const uint32_t cols = (uint32_t)(tile_cols(sk, s_at, a.sink) >> 3) << 17;
        const uint32_t q = cta.sb + OFF_Q + qs * K_BYTES, k = cta.sb + OFF_K + s * K_BYTES;
#pragma unroll
        for (int c = 0; c < 6; ++c) {
          const uint32_t off = (c >> 1) * K_BOX + (c & 1) * 32;
          mma_f16_ss(tmem + TM_S + 128 * s, smem_desc(q + off, 16, 512, SW_64),
                     smem_desc(k + off, 16, 512, SW_64), id | cols, c > 0);
        }
        mma_commit(cta.bar(S_FULL + s));
        mma_commit(cta.bar(K_EMPTY + s));
        ++sn;
        if (++s_at == sk.n) {
          mma_commit(cta.bar(Q_EMPTY + qs));
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
            wait(cta, cta.bar(DRAIN), 0, ctl);
            ok = false;
            break;
          }
          if (!(ok = wait(cta, cta.bar(V_FULL + s), (vn >> 1) & 1, ctl))) break;
          if (v_at == 0 && vm > 0 &&
              !(ok = wait(cta, cta.bar(O_FREE), (vm - 1) & 1, ctl))) break;
          if (!(ok = wait(cta, cta.bar(P_READY), vn & 1, ctl))) break;
          tc_fence_after();
          const uint32_t v = cta.sb + OFF_V + s * V_BYTES;
          const int steps = tile_cols(vk, v_at, a.sink) >> 4;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < steps)
              mma_f16_ts(tmem + TM_O, tmem + TM_P + 8 * c,
                         smem_desc(v + c * 2048, V_BOX, 1024, SW_128), ID_PV, v_at > 0 || c > 0);
          mma_commit(cta.bar(O_DONE));
          mma_commit(cta.bar(V_EMPTY + s));
          if (s_live && !(ok = scores())) break;
        }
      }
      mma_commit(cta.bar(DRAIN));
      mbar_wait(cta.bar(DRAIN), 0, ctl, DRAIN_NS);
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    const int q4 = warp & 3, hv = warp >> 2, row = 32 * q4 + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * q4) << 16);
    float* ex = (float*)(base + OFF_EX);
    float* el = (float*)(base + OFF_EL);
    uint8_t* const stg = base + OFF_STG + warp * 2048;
    Items it(a, ctl);
    int n = 0, m = 0;
    bool ok = true;
    while (ok && it.next()) {
      const int t = it.q0 + row, len = it.len;
      if (a.lens && it.q0 == 0 && it.h == 0 && tid == 0 && __ldg(a.lens + it.b) != len)
        record_error(ctl, DEV_RANGE);  // outside [0, T]: read as the nearer end
      const bool live_item = it.q0 < len;
      float ref = -INFINITY, sum = 0.f;
      if (live_item) {
        const KeyTiles kt = it.keys();
        for (int i = 0; i < kt.n; ++i, ++n) {
          const uint32_t s = n & 1;
          const int s0 = kt.tile(i) * BN;
          if (!(ok = wait_warp(cta, cta.bar(S_FULL + s), (n >> 1) & 1, ctl))) break;
          tc_fence_after();
          uint32_t z[2][32];
          tmem_ld32(trow + TM_S + 128 * s + 64 * hv, z[0]);
          tmem_ld32(trow + TM_S + 128 * s + 64 * hv + 32, z[1]);
          tmem_wait_ld();
          const bool whole = s0 + BN - 1 <= it.q0 && s0 + BN <= len &&
                             (it.q0 + BM - 1 - s0 < a.window || s0 + BN <= a.sink);
          if (!whole) {
            const int c0 = s0 + 64 * hv;
            const uint64_t see = bits_to(min(t, len - 1) - c0) &
                                 (~bits_to(t - a.window - c0) | bits_to(a.sink - 1 - c0));
            const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if (!((lo >> c) & 1)) z[0][c] = 0xFF800000u;  // -inf
              if (!((hi >> c) & 1)) z[1][c] = 0xFF800000u;
            }
          }
          float t4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            t4[j] = fmaxf(__uint_as_float(z[j & 1][j]), __uint_as_float(z[j & 1][j + 4]));
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            t4[c & 3] = fmaxf(t4[c & 3], __uint_as_float(z[0][c]));
            t4[(c + 2) & 3] = fmaxf(t4[(c + 2) & 3], __uint_as_float(z[1][c]));
          }
          float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          ex[(n & 1) * 256 + hv * 128 + row] = top;
          mbar_arrive(cta.bar(PX + q4));
          if (!(ok = wait_warp(cta, cta.bar(PX + q4), n & 1, ctl))) break;
          top = fmaxf(top, ex[(n & 1) * 256 + (hv ^ 1) * 128 + row]) * kLog2e;
          // ref, sum: in base 2; a row that has seen nothing yet has o = 0 and takes any scale
          float scale = 1.f;
          if (top > ref + 8.f) {
            if (ref != -INFINITY) scale = ex2(ref - top);
            ref = top;
          }
          const float sub = ref == -INFINITY ? 0.f : ref;
          sum *= scale;
          uint32_t p[32];
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float x = ex2(fmaf(__uint_as_float(z[c >> 4][(2 * c) & 31]), kLog2e, -sub));
            const float y = ex2(fmaf(__uint_as_float(z[c >> 4][(2 * c + 1) & 31]), kLog2e, -sub));
            s4[c & 1] += x;
            s4[2 + (c & 1)] += y;
            p[c] = BF16 ? pack2<__nv_bfloat16>(x, y) : pack2<__half>(x, y);
          }
          sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          // P's columns and, for the rescaling, O are free once the tile before has been added
          if (n > 0 && !(ok = wait_warp(cta, cta.bar(O_DONE), (n - 1) & 1, ctl))) break;
          tc_fence_after();
          if (i > 0 && __any_sync(0xffffffffu, scale != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 3; ++c) {
              uint32_t o[32];
              tmem_ld32(trow + TM_O + 96 * hv + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * scale);
              tmem_st32(trow + TM_O + 96 * hv + 32 * c, o);
            }
          }
          tmem_st32(trow + TM_P + 32 * hv, p);
          if (s0 + BN > len && len < a.T) {
            // values of padding may be anything, and 0 x NaN is NaN: zero their rows
            if (!(ok = wait_warp(cta, cta.bar(V_FULL + s), (n >> 1) & 1, ctl))) break;
            const int r0 = len - s0, cnt = (BN - r0) * 24;
            for (int x = tid; x < cnt; x += SM_WARPS * 32)
              *(uint4*)(base + OFF_V + s * V_BYTES + (x % 24 / 8) * V_BOX + (r0 + x / 24) * 128 +
                        (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async();
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(cta.bar(P_READY));
        }
        if (!ok) break;
        // the row's sum: both halves'
        el[hv * 128 + row] = sum;
        mbar_arrive(cta.bar(PL + q4));
        if (!(ok = wait_warp(cta, cta.bar(PL + q4), m & 1, ctl))) break;
        sum += el[(hv ^ 1) * 128 + row];
        if (!(ok = wait_warp(cta, cta.bar(O_DONE), (n - 1) & 1, ctl))) break;
        tc_fence_after();
        ++m;
      }
      const bool live = t < len;
      const float inv = live ? 1.f / sum : 0.f;
      const int t0 = it.q0 + 32 * q4;
      constexpr int CB = WIDE ? 16 : 32;  // channels of a 64-byte staged row
#pragma unroll 1
      for (int k = 0; k < 96 / CB; ++k) {
        uint32_t o[CB];
        if (live_item) {
          if constexpr (WIDE) tmem_ld16(trow + TM_O + 96 * hv + CB * k, o);
          else tmem_ld32(trow + TM_O + 96 * hv + CB * k, o);
          tmem_wait_ld();
        }
        if (lane == 0) bulk_wait_read<0>();  // the store before has read the staging
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 u;
          uint32_t* w = &u.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (WIDE) {
              w[e] = live ? __float_as_uint(__uint_as_float(o[4 * c + e]) * inv) : 0u;
            } else {
              const float x = __uint_as_float(o[8 * c + 2 * e]) * inv;
              const float y = __uint_as_float(o[8 * c + 2 * e + 1]) * inv;
              w[e] = !live ? 0u : BF16 ? pack2<__nv_bfloat16>(x, y) : pack2<__half>(x, y);
            }
          }
          *(uint4*)(stg + swz_off(lane, c, 64)) = u;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && t0 < a.T) {
          tma_store_4d(&map_o, smem_u32(stg), 96 * hv + CB * k, it.h, t0, it.b);
          bulk_commit();
        }
      }
      if (live_item) {
        tc_fence_before();
        mbar_arrive(cta.bar(O_FREE));
      }
      if (a.lse && hv == 0 && t < a.T)
        a.lse[((long long)it.b * a.H + it.h) * a.T + t] =
            live ? (ref + log2f(sum)) * kLn2 : -INFINITY;
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_window_fwd(const WindowArgs& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const bool bf16 = a.in_type == GLA_BF16, wide = a.out_type == GLA_FP32;
  CUtensorMap mq, mk, mv, mo;
  if (!make_tmap_seq_16bit(&mq, a.q, kDK, a.H, a.T, a.B, 32, BM, CU_TENSOR_MAP_SWIZZLE_64B, bf16) ||
      !make_tmap_seq_16bit(&mk, a.k, kDK, a.KV, a.T, a.B, 32, BN, CU_TENSOR_MAP_SWIZZLE_64B, bf16) ||
      !make_tmap_seq_16bit(&mv, a.v, kDV, a.KV, a.T, a.B, 64, BN, CU_TENSOR_MAP_SWIZZLE_128B, bf16) ||
      !(wide ? make_tmap_seq_out_f32(&mo, a.o, kDV, a.H, a.T, a.B)
             : make_tmap_seq_16bit(&mo, a.o, kDV, a.H, a.T, a.B, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                                   bf16)))
    return cudaErrorInvalidValue;
  auto kern = bf16 ? (wide ? window_fwd_kernel<true, true> : window_fwd_kernel<true, false>)
                   : (wide ? window_fwd_kernel<false, true> : window_fwd_kernel<false, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.B * a.H * ((a.T + BM - 1) / BM);
  kern<<<(unsigned)std::min<long long>(items, n_sm), THREADS, SMEM_BYTES, stream>>>(mq, mk, mv, mo,
                                                                                   a, ctl);
  return cudaGetLastError();
}

}  // namespace gla
