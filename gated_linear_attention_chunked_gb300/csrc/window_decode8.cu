// window_decode8.cu -- the windowed attention one token at a time (window_decode.cu) over pages whose
// rows are codes of 8 bits (code8.cuh).  A page's row is c 2^e, and z = 2^e (q . c) with the codes as
// 16-bit operands, exactly; the values' 2^e goes into their operand (fp16) or into the weight (bf16, whose
// range holds it).  The token's own key and value are taken as given, not as they are rounded for the page.
//
// Bound by HBM: 290 bytes a key and value, half of the 16-bit pages'.  Split and join are those of
// window_decode.cu; a warp's tile has 32 slots, as many bytes as 16 there.  A code becomes an operand by
// byte permutes and one subtraction (fp16: 0x6400 | u is 1024 + u; bf16 by way of fp32), about 1.2 and
// 2.3 instructions each.  Keys are read eight channels at a time, in an order of the channels that
// the query's registers share; values by transposed loads of pairs of channels, which come apart in the
// same permutes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "code8.cuh"
#include "window_packed.cuh"
#include "window_parts.cuh"

namespace gla {
namespace {

constexpr int WARPS = 4, THREADS = 32 * WARPS, SB = 32, STAGES = 3, HB = kPartRows;
constexpr int K8 = kDK / 16, V8 = kDV / 16;       // 16-byte chunks of a row's codes
constexpr int OFF_KV8 = SB * kDK;                 // a stage: keys, values, exponents
constexpr int OFF_EXP = SB * (kDK + kDV);
constexpr int STAGE = OFF_EXP + 2 * SB + 16;      // 9,296 bytes
constexpr int RING = WARPS * STAGES * STAGE;
constexpr int SMEM = RING + HB * 4;               // and the token's own scores

// Four bytes global -> shared, of which `bytes` are read and the others zeros.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

template <class T, class TO>
__global__ void __launch_bounds__(THREADS)
window_decode8_kernel(Decode8Args a, DecodePlan plan, int groups, DevCtl ctl) {
  constexpr bool BF16 = !__is_same(T, __half);
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const WindowCache& c = a.cache.c;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int KV = c.KV, G = a.H / KV;
  griddep_launch_dependents();  // the join waits for this whole grid
  const int cut = (int)blockIdx.x - plan.whole;  // < 0: a whole unit
  const int parts = cut < 0 ? 1 : plan.parts, part = cut < 0 ? 0 : cut % parts;
  const int part_slots = cut < 0 ? 1 << 30 : plan.part_slots;
  const int unit = cut < 0 ? (int)blockIdx.x : plan.whole + cut / parts;
  const int grp = unit % groups, nk = unit / groups;
  const int kv = nk % KV, n = nk / KV;
  const int h0 = grp * HB, heads = min(HB, G - h0);  // of this key head's query heads
  const int page = __ldg(c.page + n), pos = __ldg(a.pos + n);
  const bool ok = page >= 0 && page < c.n_pages && pos >= 0;  // the same for the whole CTA
  if (!ok && tid == 0) record_error(ctl, DEV_RANGE);
  if (!ok && parts == 1) return;

  const int slots = c.window + c.sink;
  const int held = ok ? min(pos, slots) : 0;
  const int lo = part * part_slots, hi = min(held, lo + part_slots);
  const int mine = ok ? slot_at(pos, c.window, c.sink) : 0;
  const long long layer = (long long)(ok ? page : 0) * c.pool_layers + c.layer, at = layer * slots;
  uint8_t* pk = static_cast<uint8_t*>(c.k) + (at * KV + kv) * kDK;
  uint8_t* pv = static_cast<uint8_t*>(c.v) + (at * KV + kv) * kDV;
  signed char* pe = a.cache.exps + (layer * KV + kv) * slots * 2;
  const T* nk_ = static_cast<const T*>(a.k) + ((long long)n * KV + kv) * kDK;
  const T* nv_ = static_cast<const T*>(a.v) + ((long long)n * KV + kv) * kDV;
  const T* q = static_cast<const T*>(a.q) + ((long long)n * a.H + kv * G + h0) * kDK;

  const uint32_t ring = sm + w * STAGES * STAGE;
  const int skew = (int)(reinterpret_cast<uintptr_t>(pe) & 2);
  const int tiles = hi > lo ? (hi - lo + SB * WARPS - 1) / (SB * WARPS) : 0;
  auto fetch = [&](int i) {  // warp w's tile i: slots lo + (i WARPS + w) SB ..
    if (i < tiles) {
      const int s0 = lo + (i * WARPS + w) * SB;
      const uint32_t st = ring + (i % STAGES) * STAGE;
#pragma unroll
      for (int e = 0; e < SB * K8 / 32; ++e) {
        const int x = e * 32 + lane, r = x / K8, ch = x % K8, s = s0 + r;
        copy16(st + r * kDK + ch * 16, pk + (long long)(s < hi ? s : lo) * KV * kDK + ch * 16, s < hi);
      }
#pragma unroll
      for (int e = 0; e < SB * V8 / 32; ++e) {
        const int x = e * 32 + lane, r = x / V8, ch = x % V8, s = s0 + r;
        copy16(st + OFF_KV8 + tile_off<V8>(r, ch),
               pv + (long long)(s < hi ? s : lo) * KV * kDV + ch * 16, s < hi);
      }
      // exponents, two bytes a slot, in words: where the row starts in the middle of one, from there
      if (lane <= SB / 2) {
        const long long from = 2ll * s0 - skew + 4 * lane;  // byte of the row
        copy4(st + OFF_EXP + 4 * lane, pe + (from < 2ll * hi ? from : 2ll * lo - skew),
              (int)min(max(2ll * hi - from, 0ll), 4ll));
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);

  // queries: rows g and g + 8 of 16, zeros behind the group's heads; step 2 c + h of the product has
  // channels 32 c + 8 t + 4 h .. + 3 of thread t of a row's four
  const int g = lane >> 2, t = lane & 3, t2 = t * 2;
  uint32_t qf[kDK / 16][4];
#pragma unroll
  for (int j = 0; j < kDK / 16; ++j) {
    const int ch = 32 * (j >> 1) + 8 * t + 4 * (j & 1);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint2 x = make_uint2(0u, 0u);
      if (g + 8 * r < heads) x = __ldg(reinterpret_cast<const uint2*>(q + (g + 8 * r) * kDK + ch));
      qf[j][r] = x.x;
      qf[j][2 + r] = x.y;
    }
  }
  float* own = reinterpret_cast<float*>(smem + RING);
  if (part == 0 && ok) {
    // the token's own score for each head, eight threads a row
    const int row = tid >> 3, l = tid & 7;
    float z = 0.f;
    if (row < heads)
#pragma unroll
      for (int j = 0; j < kDK / 16; ++j) {
        const float2 x = halves<T>(__ldg(reinterpret_cast<const uint32_t*>(q + row * kDK) + l + 8 * j));
        const float2 y = halves<T>(__ldg(reinterpret_cast<const uint32_t*>(nk_) + l + 8 * j));
        z = fmaf(x.x, y.x, fmaf(x.y, y.y, z));
      }
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    if (l == 0) own[row] = z;
    // and its codes into its slot (the others' rows of that slot are out of the window or not there)
    if (grp == 0 && w == 0) {
      uint4 x[3];
      uint2 o[3];
      const bool key = lane < 4, value = lane >= 8 && lane < 16;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        x[i] = key     ? __ldg(reinterpret_cast<const uint4*>(nk_) + 4 * i + lane)
               : value ? __ldg(reinterpret_cast<const uint4*>(nv_) + 8 * i + lane - 8)
                       : make_uint4(0u, 0u, 0u, 0u);
      const int e = code_row<T, 8>(x, o);  // lanes 4 .. 7 are zeros
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (key) reinterpret_cast<uint2*>(pk + (long long)mine * KV * kDK)[4 * i + lane] = o[i];
        if (value) reinterpret_cast<uint2*>(pv + (long long)mine * KV * kDV)[8 * i + lane - 8] = o[i];
      }
      if (lane == 0) pe[2ll * mine] = (signed char)e;
      if (lane == 8) pe[2ll * mine + 1] = (signed char)e;
    }
  }

  float acc[kDV / 8][4];
#pragma unroll
  for (int j = 0; j < kDV / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int i = 0; i < tiles; ++i) {
    fetch(i + STAGES - 1);
    copy_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t so = w * STAGES * STAGE + (i % STAGES) * STAGE;
    const uint8_t* st = smem + so;
    const uint32_t vs = sm + so + OFF_KV8;
    const int s0 = lo + (i * WARPS + w) * SB;
    float z[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // slots 8 b ..
#pragma unroll
      for (int j = 0; j < 4; ++j) z[b][j] = 0.f;
#pragma unroll
      for (int j = 0; j < kDK / 32; ++j) {
        const uint2 x = *reinterpret_cast<const uint2*>(st + (8 * b + g) * kDK + 32 * j + 8 * t);
        uint32_t b0, b1;
        whole_of<T, false>(x.x, b0, b1);
        mma16816<T>(z[b], qf[2 * j], b0, b1);
        whole_of<T, false>(x.y, b0, b1);
        mma16816<T>(z[b], qf[2 * j + 1], b0, b1);
      }
    }
    // this thread's columns: slots 8 b + t2, + 1
    float sv[4][2];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const char2* ex = reinterpret_cast<const char2*>(st + OFF_EXP + skew) + 8 * b + t2;
      const char2 e0 = ex[0], e1 = ex[1];
      const float k0 = scale_of((signed char)e0.x), k1 = scale_of((signed char)e1.x);
      sv[b][0] = scale_of((signed char)e0.y);
      sv[b][1] = scale_of((signed char)e1.y);
      const int s = s0 + 8 * b + t2;
      const bool in0 = s < hi && s != mine, in1 = s + 1 < hi && s + 1 != mine;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        z[b][2 * r] = in0 ? z[b][2 * r] * k0 : -INFINITY;
        z[b][2 * r + 1] = in1 ? z[b][2 * r + 1] * k1 : -INFINITY;
      }
    }
    uint32_t pf[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < 4; ++b) top = fmaxf(top, fmaxf(z[b][2 * r], z[b][2 * r + 1]));
      top = fmaxf(m[r], quad_max(top));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = ex2((m[r] - base) * kLog2e);
      m[r] = top;
      l[r] *= keep;
#pragma unroll
      for (int j = 0; j < kDV / 8; ++j) {
        acc[j][2 * r] *= keep;
        acc[j][2 * r + 1] *= keep;
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float p0 = ex2((z[b][2 * r] - base) * kLog2e), p1 = ex2((z[b][2 * r + 1] - base) * kLog2e);
        l[r] += p0 + p1;
        if constexpr (BF16) {
          p0 *= sv[b][0];
          p1 *= sv[b][1];
        }
        pf[b >> 1][2 * (b & 1) + r] = pack2<T>(p0, p1);
      }
    }
    [[maybe_unused]] uint32_t s2[4];  // fp16: the scales of the thread's pairs of slots
    if constexpr (!BF16)
#pragma unroll
      for (int b = 0; b < 4; ++b) s2[b] = pack2<__half>(sv[b][0], sv[b][1]);
#pragma unroll
    for (int h = 0; h < 2; ++h)  // slots 16 h ..
#pragma unroll
      for (int ch = 0; ch < V8; ch += 2) {
        // codes of slots 16 h + t2, + 1 (x[0]) and + 8, + 9 (x[1]), channels 16 ch + 2 g, + 1; x[2],
        // x[3]: channels 16 ch + 16 + ..
        uint32_t x[4];
        ldsm4t(x, vs + tile_off<V8>(16 * h + (lane & 15), ch + (lane >> 4)));
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t e0, o0, e1, o1;
          whole_of<T, true>(x[2 * y], e0, o0);
          whole_of<T, true>(x[2 * y + 1], e1, o1);
          if constexpr (!BF16) {
            const __half2 f0 = reinterpret_cast<const __half2&>(s2[2 * h]);
            const __half2 f1 = reinterpret_cast<const __half2&>(s2[2 * h + 1]);
            reinterpret_cast<__half2&>(e0) = __hmul2(reinterpret_cast<__half2&>(e0), f0);
            reinterpret_cast<__half2&>(o0) = __hmul2(reinterpret_cast<__half2&>(o0), f0);
            reinterpret_cast<__half2&>(e1) = __hmul2(reinterpret_cast<__half2&>(e1), f1);
            reinterpret_cast<__half2&>(o1) = __hmul2(reinterpret_cast<__half2&>(o1), f1);
          }
          mma16816<T>(acc[2 * (ch + y)], pf[h], e0, e1);
          mma16816<T>(acc[2 * (ch + y) + 1], pf[h], o0, o1);
        }
      }
    __syncwarp();  // the stage is free for the copy of the next round
  }
  copy_wait<0>();
  __syncthreads();

  // join the warps and the token itself: o, m and l of each row through shared memory
  float* so = reinterpret_cast<float*>(smem);              // [WARPS][HB][kDV]
  float* sml = so + WARPS * HB * kDV;                      // [WARPS][HB][2]
  static_assert(WARPS * HB * (kDV + 2) * 4 <= RING, "the join fits the ring");
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
    for (int j = 0; j < V8; ++j)
      *reinterpret_cast<float4*>(so + (w * HB + row) * kDV + 16 * j + 4 * t) =
          make_float4(acc[2 * j][2 * r], acc[2 * j + 1][2 * r], acc[2 * j][2 * r + 1],
                      acc[2 * j + 1][2 * r + 1]);
  }
  __syncthreads();
  const long long head = (long long)n * a.H + kv * G + h0;
  for (int x = tid; x < heads * (kDV / 2); x += THREADS) {
    const int row = x / (kDV / 2), ch = x % (kDV / 2) * 2;
    const float self = part == 0 && ok ? own[row] : -INFINITY;
    float top = self;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) top = fmaxf(top, sml[(k * HB + row) * 2]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = ex2((self - base) * kLog2e), o0 = 0.f, o1 = 0.f;
    if (part == 0 && ok) {
      const float2 v = halves<T>(__ldg(reinterpret_cast<const uint32_t*>(nv_ + ch)));
      o0 = sum * v.x;
      o1 = sum * v.y;
    }
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float f = ex2((sml[(k * HB + row) * 2] - base) * kLog2e);
      const float2 o = *reinterpret_cast<const float2*>(so + (k * HB + row) * kDV + ch);
      sum = fmaf(f, sml[(k * HB + row) * 2 + 1], sum);
      o0 = fmaf(f, o.x, o0);
      o1 = fmaf(f, o.y, o1);
    }
    if (parts == 1) {
      const float inv = 1.f / sum;  // the token itself is there: sum > 0
      store2(static_cast<TO*>(a.o) + (head + row) * kDV + ch, o0 * inv, o1 * inv);
    } else {
      float* pw = static_cast<float*>(a.workspace) +
                  ((long long)(unit - plan.whole) * HB + row) * parts * (kDV + 2) + part * (kDV + 2);
      *reinterpret_cast<float2*>(pw + ch) = make_float2(o0, o1);
      if (ch == 0) *reinterpret_cast<float2*>(pw + kDV) = make_float2(top, sum);
    }
  }
}

DecodePlan make_plan(int n, int KV, int H, int slots, int n_sm) {
  return make_decode_plan((long long)n * KV * decode_groups(KV, H), slots, SB * WARPS, n_sm);
}

template <class T, class TO>
cudaError_t run(const Decode8Args& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const WindowCache& c = a.cache.c;
  const DecodePlan plan = make_plan(c.n, c.KV, a.H, c.window + c.sink, n_sm);
  auto kern = window_decode8_kernel<T, TO>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(plan.whole + plan.cut * plan.parts), THREADS, SMEM, stream>>>(
      a, plan, decode_groups(c.KV, a.H), ctl);
  if ((e = cudaGetLastError()) != cudaSuccess || !plan.cut) return e;
  WindowDecodeArgs j;
  j.c = c; j.pos = a.pos; j.q = a.q; j.k = a.k; j.v = a.v; j.o = a.o; j.out_type = a.out_type;
  j.H = a.H; j.workspace = a.workspace;
  return launch_window_join(j, plan, stream);
}

}  // namespace

size_t window_decode8_workspace_bytes(int n, int KV, int H, int slots, int n_sm) {
  return decode_plan_bytes(make_plan(n, KV, H, slots, n_sm));
}

cudaError_t launch_window_decode8(const Decode8Args& a, int n_sm, DevCtl ctl, cudaStream_t stream) {
  const bool wide = a.out_type == GLA_FP32;
  if (a.cache.c.type == GLA_BF16)
    return wide ? run<__nv_bfloat16, float>(a, n_sm, ctl, stream)
                : run<__nv_bfloat16, __nv_bfloat16>(a, n_sm, ctl, stream);
  return wide ? run<__half, float>(a, n_sm, ctl, stream) : run<__half, __half>(a, n_sm, ctl, stream);
}

}  // namespace gla
