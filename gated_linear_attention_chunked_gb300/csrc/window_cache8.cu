// window_cache8.cu -- packed tokens into their pages, as 16-bit rows or as codes of 8 bits (code8.cuh),
// and pages of codes read back as 16-bit rows.
//
// Bound by HBM.  Append: a warp has eight rows (a row: one token's key and value of one head) and their
// nine accesses of 16 bytes a lane in flight at once: the keys by 4 lanes a row, the values by 8, in two
// halves.  The maximum of a row goes between those lanes by shuffles.  Only tokens that are still in the page
// at the call's end are read: the last `window`, and the sinks, so that no slot is written twice.
#include <cuda_runtime.h>

#include <algorithm>

#include "code8.cuh"
#include "window_packed.cuh"

namespace gla {
namespace {

constexpr int THREADS = 256, ROWS = 8;  // rows of a warp

// Where one row goes; slot < 0: nowhere.
struct Target {
  int slot;
  long long page;  // page and layer
};

__device__ __forceinline__ Target target(const AppendArgs& a, int token, const DevCtl& ctl) {
  const WindowCache& c = a.cache.c;
  const Target none{-1, 0};
  if (token >= a.tok.n_tokens) return none;
  const int b = sequence_of(a.tok.start, c.n, token);
  if (b < 0 || b >= c.n) return none;  // a row of no sequence
  const Sequence s = sequence(c, a.tok, b, ctl);
  const int i = token - s.first;
  if (i < 0 || i >= s.tokens) return none;
  int count = s.tokens;
  if (a.count) {
    const int given = __ldg(a.count + b);
    if (given < 0 || given > count) record_error(ctl, DEV_RANGE);
    count = min(max(given, 0), count);
  }
  const int t = s.pos + i;
  if (i >= count || (t >= c.sink && i < count - c.window)) return none;
  return Target{slot_at(t, c.window, c.sink), (long long)s.page * c.pool_layers + c.layer};
}

template <class T, bool CODES>
__global__ void __launch_bounds__(THREADS)
append_kernel(AppendArgs a, long long rows, DevCtl ctl) {
  const int lane = threadIdx.x & 31;
  const WindowCache& c = a.cache.c;
  const int slots = c.window + c.sink, KV = c.KV;
  const long long row0 = ((long long)blockIdx.x * THREADS + threadIdx.x) / 32 * ROWS;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    // sequences whose tokens no row belongs to are checked here
    for (int b = lane; b < c.n; b += 32) {
      sequence(c, a.tok, b, ctl);
      if (a.count && __ldg(a.count + b) != 0 &&
          (__ldg(a.count + b) < 0 || __ldg(a.count + b) > __ldg(a.tok.start + b + 1) - __ldg(a.tok.start + b)))
        record_error(ctl, DEV_RANGE);
    }
  }
  if (row0 >= rows) return;
  const uint4* ks = static_cast<const uint4*>(a.k);
  const uint4* vs = static_cast<const uint4*>(a.v);
  // lane l looks up row l / 4; the values' lanes take theirs from it
  const long long mine = row0 + (lane >> 2);
  // (rows below 2^31 have a token by one 32-bit division)
  const int token = rows >> 31 ? (int)(mine / KV) : (int)((unsigned)mine / (unsigned)KV);
  const Target at = mine < rows ? target(a, token, ctl) : Target{-1, 0};
  const int kv = (int)(mine - (long long)token * KV);
  if (!__any_sync(0xffffffffu, at.slot >= 0)) return;
  uint4 x[3][3];
  int slot[3], head[3];
  long long page[3];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    // p 0: keys, a row per 4 lanes; p 1, 2: values of rows 4 (p - 1) .., a row per 8 lanes
    const int from = p == 0 ? lane : 4 * (4 * (p - 1) + (lane >> 3));
    slot[p] = __shfl_sync(0xffffffffu, at.slot, from);
    page[p] = __shfl_sync(0xffffffffu, at.page, from);
    head[p] = __shfl_sync(0xffffffffu, kv, from);
    const long long row = row0 + (from >> 2);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      x[p][i] = make_uint4(0u, 0u, 0u, 0u);
      if (slot[p] >= 0)
        x[p][i] = p == 0 ? __ldcs(ks + row * kCK + 4 * i + (lane & 3))
                         : __ldcs(vs + row * kCV + 8 * i + (lane & 7));
    }
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const long long dst = (page[p] * slots + slot[p]) * KV + head[p];
    if constexpr (CODES) {
      uint2 o[3];
      const int e = p == 0 ? code_row<T, 4>(x[p], o) : code_row<T, 8>(x[p], o);
      if (slot[p] >= 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          if (p == 0) static_cast<uint2*>(c.k)[dst * kCK + 4 * i + (lane & 3)] = o[i];
          else static_cast<uint2*>(c.v)[dst * kCV + 8 * i + (lane & 7)] = o[i];
        }
        if ((lane & (p == 0 ? 3 : 7)) == 0)
          a.cache.exps[((page[p] * KV + head[p]) * slots + slot[p]) * 2 + (p > 0)] =
              (signed char)e;
      }
    } else if (slot[p] >= 0) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (p == 0) static_cast<uint4*>(c.k)[dst * kCK + 4 * i + (lane & 3)] = x[p][i];
        else static_cast<uint4*>(c.v)[dst * kCV + 8 * i + (lane & 7)] = x[p][i];
      }
    }
  }
}

// One thread per 16 codes.  Rows: [n, slots, KV], of 6 (keys) and 12 (values) such pieces.  pos: only slots
// that hold a token; copies: where page n went, n or (its own out of range) -1.
// I: a type that holds the number of pieces.  (With 64-bit divisions the kernel was bound by instructions.)
template <class T, class I>
__global__ void __launch_bounds__(THREADS)
read8_kernel(ServeCache cache, uint4* __restrict__ k, uint4* __restrict__ v, long long rows,
             const int* __restrict__ pos, int* __restrict__ copies, DevCtl ctl) {
  const WindowCache& c = cache.c;
  const int slots = c.window + c.sink;
  const I x = (I)blockIdx.x * THREADS + threadIdx.x, row = x / 18;
  if (row >= (I)rows) return;
  const int piece = (int)(x - row * 18);
  const I ns = row / (I)c.KV;
  const int kv = (int)(row - ns * (I)c.KV), n = (int)(ns / (I)slots), s = (int)(ns - (I)n * (I)slots);
  const int page = __ldg(c.page + n);
  const bool there = page >= 0 && page < c.n_pages;
  if (copies && s == 0 && kv == 0 && piece == 0) copies[n] = there ? n : -1;
  if (!there) {
    if (s == 0 && piece == 0) record_error(ctl, DEV_RANGE);
    return;
  }
  if (pos && s >= __ldg(pos + n)) return;
  const long long at = (long long)page * c.pool_layers + c.layer, src = (at * slots + s) * c.KV + kv;
  const bool key = piece < 6;
  const uint4 w = key ? __ldcs(static_cast<const uint4*>(c.k) + src * 6 + piece)
                      : __ldcs(static_cast<const uint4*>(c.v) + src * 12 + piece - 6);
  const float sc = scale_of(cache.exps[((at * c.KV + kv) * slots + s) * 2 + !key]);
  uint32_t o[8];
  const uint32_t* in = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    whole_of<T, false>(in[i], o[2 * i], o[2 * i + 1]);
    o[2 * i] = scaled<T>(o[2 * i], sc);
    o[2 * i + 1] = scaled<T>(o[2 * i + 1], sc);
  }
  uint4* dst = key ? k + (size_t)row * kCK + 2 * piece : v + (size_t)row * kCV + 2 * (piece - 6);
  __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
}

}  // namespace

cudaError_t launch_window_append(const AppendArgs& a, DevCtl ctl, cudaStream_t stream) {
  const long long rows = (long long)a.tok.n_tokens * a.cache.c.KV;
  const unsigned grid = (unsigned)((rows + ROWS * THREADS / 32 - 1) / (ROWS * THREADS / 32));
  const bool bf16 = a.cache.c.type == GLA_BF16;
  if (!a.cache.exps) append_kernel<__half, false><<<grid, THREADS, 0, stream>>>(a, rows, ctl);
  else if (bf16) append_kernel<__nv_bfloat16, true><<<grid, THREADS, 0, stream>>>(a, rows, ctl);
  else append_kernel<__half, true><<<grid, THREADS, 0, stream>>>(a, rows, ctl);
  return cudaGetLastError();
}

cudaError_t launch_window_read8(const ServeCache& cache, void* k, void* v, const int* pos, int* copies,
                                DevCtl ctl, cudaStream_t stream) {
  const WindowCache& c = cache.c;
  const long long rows = (long long)c.n * (c.window + c.sink) * c.KV;
  const unsigned grid = (unsigned)((rows * 18 + THREADS - 1) / THREADS);
  auto run = [&](auto kern) {
    kern<<<grid, THREADS, 0, stream>>>(cache, static_cast<uint4*>(k), static_cast<uint4*>(v), rows, pos, copies, ctl);
  };
  const bool wide = (long long)grid * THREADS >> 32;
  if (c.type == GLA_BF16) {
    if (wide) run(read8_kernel<__nv_bfloat16, unsigned long long>);
    else run(read8_kernel<__nv_bfloat16, unsigned>);
  } else {
    if (wide) run(read8_kernel<__half, unsigned long long>);
    else run(read8_kernel<__half, unsigned>);
  }
  return cudaGetLastError();
}

}  // namespace gla
