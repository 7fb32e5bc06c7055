// window_parts.cuh -- how the decode steps of the windowed attention cut few units into parts, and the
// join of those.
#pragma once
#include <algorithm>

#include "window_common.cuh"

namespace gla {

constexpr int kPartRows = 16;  // query heads of a unit

// CTAs: a unit each for the first `whole` units, `parts` for each of the `cut` others.
struct DecodePlan {
  int whole, cut, parts, part_slots;
};

// Parts of at least one round of a CTA's tiles (`unit` slots) each; nothing is cut where two do not fit
// into the last round.
inline DecodePlan make_decode_plan(long long units, int slots, int unit, int n_sm) {
  const int hold = std::max(2 * n_sm, 1), rest = (int)(units % hold);
  const int most = std::min((slots + unit - 1) / unit, 64);
  const int parts = rest ? std::min(hold / rest, most) : 1;
  if (parts < 2) return DecodePlan{(int)units, 0, 1, 0};
  const int part_slots = ((slots + parts - 1) / parts + unit - 1) / unit * unit;
  return DecodePlan{(int)(units - rest), rest, parts, part_slots};
}
inline int decode_groups(int KV, int H) { return (H / KV + kPartRows - 1) / kPartRows; }
inline size_t decode_plan_bytes(const DecodePlan& p) {
  return (size_t)p.cut * kPartRows * p.parts * (kDV + 2) * sizeof(float);
}

// The second kernel of a cut step (window_decode.cu), behind the first on the stream.
cudaError_t launch_window_join(const WindowDecodeArgs& a, const DecodePlan& plan,
                               cudaStream_t stream);

}  // namespace gla
