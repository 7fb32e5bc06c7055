// window_packed.cuh -- packed sequences and their slots, shared by the kernels of window_serve.h.
#pragma once
#include "window_common.cuh"
#include "window_serve.h"

namespace gla {

__device__ __forceinline__ int slot_at(int t, int window, int sink) {
  return t < sink ? t : sink + (int)((unsigned)(t - sink) % (unsigned)window);
}

// The sequence whose tokens hold row i: the last b with start[b] <= i (-1: none; n: rows behind all).
__device__ __forceinline__ int sequence_of(const int* start, int n, int i) {
  int lo = 0, hi = n + 1;  // start[lo - 1] <= i < start[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(start + mid) <= i) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

// One sequence of a call, checked.  Something outside its range is recorded, and the sequence left as it
// is (`tokens` 0).
struct Sequence {
  int first, tokens, pos, page;
};
__device__ __forceinline__ Sequence sequence(const WindowCache& c, const Packed& t, int b,
                                             const DevCtl& ctl) {
  Sequence s;
  s.first = __ldg(t.start + b);
  const int end = __ldg(t.start + b + 1);
  s.tokens = end - s.first;
  s.pos = __ldg(t.pos + b);
  s.page = __ldg(c.page + b);
  const bool rows = s.first >= 0 && end >= s.first && end <= t.n_tokens;
  if (!rows || s.page < 0 || s.page >= c.n_pages || s.pos < 0 ||
      (long long)s.pos + s.tokens > 0x7FFFFFFFll) {
    record_error(ctl, DEV_RANGE);
    s.tokens = 0;
    s.page = 0;
    s.pos = 0;
    s.first = 0;
  }
  return s;
}

}  // namespace gla
