// What the attention kernels over a block cache share (gfx950).
#ifndef ETS_ATTEND_ROWS_H
#define ETS_ATTEND_ROWS_H

#include "ets_attend.h"

namespace ets {

// How far the token t of a live row sees: positions before *upto, and bits of a
// tree's tokens from spot.begin on.
__device__ __forceinline__ void attend_sight(const AttendBlocksParams& p, const AttendSpot& spot, bool live, int t, int* upto,
                                             uint64_t* bits) {
  const ets_attend_args& a = p.a;
  *upto = INT32_MAX, *bits = 0;
  if (!p.first) return;
  const bool alive = live && spot.begin + t < min(a.seq_lens[spot.b], a.L);
  const int64_t to = spot.begin + (a.tree_mask ? 0 : t + 1);
  *upto = alive ? static_cast<int>(min(max(to, static_cast<int64_t>(0)), static_cast<int64_t>(INT32_MAX))) : 0;
  if (a.tree_mask && alive) {
    *bits = static_cast<uint64_t>(a.tree_mask[spot.b * a.mask_b + t]);
    if (a.T < 64) *bits &= (1ull << a.T) - 1;
  }
}

// Rows of padding are masked only where other rows are: what they gather before is thrown away at the end.
__device__ __forceinline__ bool attend_blind(int upto, uint64_t bits) { return upto == 0 && bits == 0; }

// The 32 keys from position `at` on, one bit each, that such a row sees.
__device__ __forceinline__ uint32_t attend_seen_by(const AttendSpot& spot, int upto, uint64_t bits, int at) {
  const int ahead = upto - at;
  uint32_t vis = ahead >= 32 ? ~0u : ahead > 0 ? (1u << ahead) - 1 : 0;
  const int64_t to = spot.begin - at;
  if (to >= 0) {
    vis |= to < 32 ? static_cast<uint32_t>(bits << to) : 0;
  } else {
    vis |= to > -64 ? static_cast<uint32_t>(bits >> -to) : 0;
  }
  return vis;
}

// What the kernel for many rows (ets_attend_rows.hip) takes of them: a workgroup's waves, a wave's tiles of 16.
struct RowsShape {
  int width;  // 64-channel steps: 1 to 4
  int waves, tiles;
};
// Workgroups of a compute unit, by LDS and registers.
constexpr int rows_per_unit(int width, int waves) { return waves == 4 && width <= 2 ? 2 : 1; }

inline int64_t attend_rows_groups(const AttendBlocksParams& p) {
  const int64_t lists = static_cast<int64_t>(p.units) * p.splits;
  return p.dealt == 0 ? attend_groups(p) : (p.dealt == 1 ? (lists + 7) / 8 * 8 : lists) * p.row_groups;
}

void launch_attend_rows(const AttendBlocksParams& p, const RowsShape& r, hipStream_t s);

}  // namespace ets

#endif  // ETS_ATTEND_ROWS_H
