// ets_attend.hip -- attention of one or a few tokens a sequence over an 8-bit
// cache: over selected slots or over whole paged sequences, plus a tree of
// drafted tokens (gfx950).
#include "ets_attend_narrow.h"

namespace ets {
namespace {

constexpr int kThreads = kAttendThreads;
constexpr int kWaves = kAttendWaves;
constexpr int kTile = kAttendTile;

// ---------------------------------------------------------------- host

struct Plan {
  AttendParams p;
  int width;  // 64-channel pairs of the instance: 1, 2, 3, 4 or 9
  int mt;
  bool shared;
  size_t bytes;
};

ets_status make_plan(const ets_attend_args* a, Plan* plan) {
  if (!a || a->B < 0 || a->T < 0 || a->Hkv < 1 || a->Hq < 1 || a->Hq % a->Hkv) return ETS_ERR_INVALID_ARG;
  if (a->D < kCacheBlock || a->D % kCacheBlock || a->D > ETS_MAX_HEAD_DIM || a->Dv < kCacheBlock ||
      a->Dv % kCacheBlock || a->Dv > ETS_MAX_HEAD_DIM)
    return ETS_ERR_INVALID_ARG;
  if ((a->dtype != ETS_BF16 && a->dtype != ETS_FP16) || a->S < 0 || a->S > INT32_MAX) return ETS_ERR_INVALID_ARG;
  const bool paged = a->slots == nullptr;
  // positions are 32-bit numbers in the kernels, and stand up to 3 chunks of slots behind a list's end
  if (paged ? (a->L < 0 || a->L > ETS_MAX_LENGTH || a->page_size < 1) : (a->K < 0 || a->K > ETS_MAX_LENGTH)) return ETS_ERR_INVALID_ARG;
  if (a->tree_slots && a->T > ETS_MAX_TREE) return ETS_ERR_INVALID_ARG;
  // row strides are 32-bit numbers in the kernels; 4 GiB from slot to slot is no cache
  if (a->k_s < 0 || a->ks_s < 0 || a->v_s < 0 || a->vs_s < 0 || (a->k_s | a->ks_s | a->v_s | a->vs_s) > UINT32_MAX)
    return ETS_ERR_INVALID_ARG;
  *plan = Plan{};
  AttendParams& p = plan->p;
  p.a = *a;
  if (a->B == 0 || a->T == 0) return ETS_OK;
  if (static_cast<int64_t>(a->B) * a->T * a->Hq > INT32_MAX) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int wide = (a->D > a->Dv ? a->D : a->Dv) + 63;
  plan->width = wide / 64 <= 4 ? wide / 64 : 9;
  plan->shared = plan->width == 9 && a->Dv <= 512 && a->Dv <= a->D && a->v_codes == a->k_codes && a->v_scales == a->k_scales &&
                 a->v_s == a->k_s && a->v_h == a->k_h && a->vs_s == a->ks_s && a->vs_h == a->ks_h;
  p.G = a->Hq / a->Hkv;
  p.rows = paged ? a->T * p.G : p.G;
  p.units = a->B * a->Hkv * (paged ? 1 : a->T);
  // 16-row tiles of a workgroup: four leave a wave a SIMD (8 heads of 7 sequences of 10296, 40 rows each, probabilities of
  // one part: 73 us against 64), and so do two of 192 channels (14 us against 9.5 for 40 rows of 160 channels)
  const int most = plan->width == 3 ? 1 : 2;
  plan->mt = 1;
  while (plan->mt < most && 16 * plan->mt < p.rows) plan->mt *= 2;
  if (plan->width == 9) plan->mt = attend_wide_rows(p.rows, plan->shared, a->dtype == ETS_BF16);
  p.group_rows = 16 * plan->mt;
  p.row_groups = (p.rows + p.group_rows - 1) / p.group_rows;
  p.tree_tiles = a->tree_slots ? (a->T + kTile - 1) / kTile : 0;
  const int tiles = ((paged ? a->L : a->K) + kTile - 1) / kTile + p.tree_tiles;
  const int64_t lists = static_cast<int64_t>(p.units) * p.row_groups;
  // workgroups to fill the device with: a compute unit holds one of the wide kernel's and up to three of the
  // narrow one's, but two read faster than three (8 sequences of 32768: 118 us against 124)
  const int fits = plan->width == 9 ? 1 : attend_per_unit(plan->width, plan->mt);
  const int64_t room = static_cast<int64_t>(cu) * (fits < 2 ? fits : 2);
  // Heads of one slot lie next to each other in memory: a workgroup of the narrow
  // kernel takes up to 4, a wave each, so that a slot's lines are read together (16
  // sequences of 7 tokens, 1024 slots: 69 us against 80 with one).  Where a wave has
  // few tiles, the 4 times as many splits cost more at their join (one sequence of
  // 32771: 29.6 us against 27).
  p.heads = plan->width == 9 || tiles * lists <= 8 * room * kWaves ? 1 : a->Hkv % 4 == 0 ? 4 : a->Hkv % 2 == 0 ? 2 : 1;
  const int64_t groups = lists / p.heads;
  // each wave with a tile at least
  int64_t splits = (room + groups - 1) / groups;
  // more than the device holds at once would wait for a second turn
  if (groups * splits > static_cast<int64_t>(cu) * fits && splits > 1) splits = static_cast<int64_t>(cu) * fits / groups;
  const int64_t cap = plan->width == 9 ? (tiles + 3) / 4 : (tiles + kWaves / p.heads - 1) / (kWaves / p.heads);
  splits = splits > cap ? cap : splits;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits);
  if (lists * (p.splits + 8) > INT32_MAX / 16) return ETS_ERR_INVALID_ARG;
  // one launch, of fewer than 2^32 lanes
  if (attend_groups(p) * (plan->width == 9 ? 2 * kThreads : kThreads) > UINT32_MAX) return ETS_ERR_INVALID_ARG;
  p.scale_log2 = static_cast<float>(1.4426950408889634074 / __builtin_sqrt(static_cast<double>(a->D)));
  p.by_page = fast_div(paged ? a->page_size : 1);
  p.by_heads = fast_div(a->Hkv);
  p.by_tokens = fast_div(a->T);
  p.by_groups = fast_div(p.row_groups);
  p.by_splits = fast_div(p.splits);
  p.by_G = fast_div(p.G);
  p.by_inner = fast_div(a->Hkv / p.heads * p.row_groups);
  p.by_rows = fast_div(p.group_rows);
  // the join: whole rows to a workgroup, or 32-channel parts where there are few rows with many splits
  p.join_lanes = static_cast<int64_t>(p.units) * p.rows < 2 * cu && p.splits > 16 ? 8 : a->Dv / 4;
  const int most_groups = kThreads / p.join_lanes;
  p.join_groups = p.splits / 4 < most_groups ? (p.splits / 4 > 1 ? p.splits / 4 : 1) : most_groups;
  p.join_parts = kThreads / (p.join_lanes * p.join_groups);
  p.by_lanes = fast_div(p.join_lanes);
  p.by_parts = fast_div(a->Dv / 4 / p.join_lanes);
  p.by_unit_rows = fast_div(p.rows);
  if (p.splits > 1) plan->bytes = static_cast<size_t>(lists) * p.splits * 16 * plan->mt * (a->Dv * 4 + 8);
  return ETS_OK;
}

template <class T, int N, int MT>
void launch_attend(const AttendParams& p, hipStream_t s) {
  const size_t lds = kWaves * kTile * (2 * value_plane(N) + 16) + kWaves * (MT + 1) * 16 * sizeof(f32x2) + 3 * kChunk * kTile * 4;
  const uint32_t grid = attend_grid(p);
  if (p.a.D == 64 * N && p.a.Dv == 64 * N) {
    hipLaunchKernelGGL((attend_kernel<T, N, N, MT, true>), dim3(grid), dim3(kThreads), lds, s, p);
  } else {
    hipLaunchKernelGGL((attend_kernel<T, N, N, MT, false>), dim3(grid), dim3(kThreads), lds, s, p);
  }
}

template <class T, int N>
void launch_width(const Plan& plan, hipStream_t s) {
  if (plan.mt == 1) {
    launch_attend<T, N, 1>(plan.p, s);
  } else if constexpr (N != 3) {
    launch_attend<T, N, 2>(plan.p, s);
  }
}

template <class T>
void launch_type(const Plan& plan, hipStream_t s) {
  const AttendParams& p = plan.p;
  switch (plan.width) {
    case 1: launch_width<T, 1>(plan, s); break;
    case 2: launch_width<T, 2>(plan, s); break;
    case 3: launch_width<T, 3>(plan, s); break;
    case 4: launch_width<T, 4>(plan, s); break;
    default: launch_attend_wide(p, plan.mt, plan.shared, s);
  }
  if (p.splits > 1) {
    const int64_t parts = static_cast<int64_t>(p.units) * p.rows * p.by_parts.d;
    hipLaunchKernelGGL(join_kernel<T>, dim3(static_cast<uint32_t>((parts + p.join_parts - 1) / p.join_parts)), dim3(kThreads), 0, s, p);
  }
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_attend_workspace_size(const ets_attend_args* args, size_t* bytes) {
  if (!bytes) return ETS_ERR_INVALID_ARG;
  ets::Plan plan;
  if (ets_status st = ets::make_plan(args, &plan); st != ETS_OK) return st;
  *bytes = plan.bytes;
  return ETS_OK;
}

ets_status ets_attend(const ets_attend_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ets;
  Plan plan;
  if (ets_status st = make_plan(args, &plan); st != ETS_OK) return st;
  const ets_attend_args& a = plan.p.a;
  if (a.B == 0 || a.T == 0) return ETS_OK;
  if (!a.q || !a.out || !a.lse || (a.S && (!a.k_codes || !a.k_scales || !a.v_codes || !a.v_scales)) ||
      (!a.slots && (!a.seq_lens || (a.L && !a.page_table))) || (a.tree_slots && !a.tree_mask))
    return ETS_ERR_INVALID_ARG;
  if (plan.bytes) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || workspace_bytes < plan.bytes) return ETS_ERR_WORKSPACE;
    plan.p.part = static_cast<float*>(workspace);
    const int64_t rows = static_cast<int64_t>(plan.p.units) * plan.p.row_groups * plan.p.splits * 16 * plan.mt;
    plan.p.stat = reinterpret_cast<f32x2*>(plan.p.part + rows * a.Dv);
  }
  auto s = static_cast<hipStream_t>(stream);
  if (a.dtype == ETS_BF16) {
    launch_type<__bf16>(plan, s);
  } else {
    launch_type<_Float16>(plan, s);
  }
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"
