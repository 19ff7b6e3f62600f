// ets_attend_blocks.hip -- attention over an 8-bit cache with one scale for a
// block of tokens and a head: single tokens, trees of drafted tokens and
// pieces of prompts (gfx950).
#include "ets_speculate.h"

#include "ets_attend_narrow.h"

namespace ets {
namespace {

constexpr int kLongList = 8192;  // positions from which eight waves pay
constexpr int kManyRows = 32;  // the narrow kernel's rows of a workgroup: more would decode each key again

struct BlocksPlan {
  AttendBlocksParams p;
  int width;  // 64-channel steps of the instance: 1 to 4
  int mt;     // tiles of 16 query rows of a wave
  bool many;  // rows for the kernel of ets_attend_rows.hip
  RowsShape shape;
  size_t bytes;
};

ets_status make_plan(const ets_attend_blocks_args* a, BlocksPlan* plan) {
  if (!a || a->B < 0 || a->T < 0 || a->Hkv < 1 || a->Hq < 1 || a->Hq % a->Hkv) return ETS_ERR_INVALID_ARG;
  if (a->D < kCacheBlock || a->D % kCacheBlock || a->D > ETS_MAX_BLOCK_DIM || a->Dv < kCacheBlock || a->Dv % kCacheBlock ||
      a->Dv > ETS_MAX_BLOCK_DIM)
    return ETS_ERR_INVALID_ARG;
  if ((a->dtype != ETS_BF16 && a->dtype != ETS_FP16) || a->S < 0 || a->S > INT32_MAX) return ETS_ERR_INVALID_ARG;
  if (a->L < 0 || a->L > ETS_MAX_LENGTH || a->block < 1 || a->page_size < 1 || a->page_size % a->block || a->S % a->block)
    return ETS_ERR_INVALID_ARG;
  if (a->tree_mask && (!a->first || a->T > ETS_MAX_TREE)) return ETS_ERR_INVALID_ARG;
  // strides from slot to slot and block to block are 32-bit numbers in the kernels
  if (a->k_s < 0 || a->ks_s < 0 || a->v_s < 0 || a->vs_s < 0 || (a->k_s | a->ks_s | a->v_s | a->vs_s) > UINT32_MAX)
    return ETS_ERR_INVALID_ARG;
  *plan = BlocksPlan{};
  AttendBlocksParams& p = plan->p;
  ets_attend_args& to = p.a;
  to.B = a->B, to.T = a->T, to.Hq = a->Hq, to.Hkv = a->Hkv, to.D = a->D, to.Dv = a->Dv, to.dtype = a->dtype;
  to.L = a->L, to.page_size = a->page_size;
  to.S = a->S / a->page_size * a->page_size;  // whole pages
  to.q = a->q, to.q_b = a->q_b, to.q_t = a->q_t, to.q_h = a->q_h;
  to.k_codes = a->k_codes, to.k_s = a->k_s, to.k_h = a->k_h, to.k_scales = a->k_scales, to.ks_s = a->ks_s, to.ks_h = a->ks_h;
  to.v_codes = a->v_codes, to.v_s = a->v_s, to.v_h = a->v_h, to.v_scales = a->v_scales, to.vs_s = a->vs_s, to.vs_h = a->vs_h;
  to.page_table = a->page_table, to.pt_b = a->pt_b, to.seq_lens = a->seq_lens;
  to.tree_mask = a->tree_mask, to.mask_b = a->mask_b, to.out = a->out, to.lse = a->lse;
  p.first = a->first;
  if (a->B == 0 || a->T == 0) return ETS_OK;
  if (static_cast<int64_t>(a->B) * a->T * a->Hq > INT32_MAX) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  plan->width = ((a->D > a->Dv ? a->D : a->Dv) + 63) / 64;
  p.G = a->Hq / a->Hkv;
  p.rows = a->T * p.G;
  p.units = a->B * a->Hkv;
  plan->many = p.rows > kManyRows;
  const int tiles = (a->L + kAttendTile - 1) / kAttendTile;
  int fits = 1, waves_rows = 1;
  if (plan->many) {
    // Two workgroups of four waves share a compute unit, and one works while the other waits at its barrier.  Eight waves
    // decode each key for twice the rows, which pays for 65 to 128 channels and 256 rows and more where no group's second
    // half is empty, lists are long, and there are workgroups for several turns of the device.  Their times over those of
    // four waves, 300 random batches and some that are not:
    //   within the rule      0.99 in the mean of 72, 0.92 to 1.11 (8 full sequences of 8192, 1024 tokens each: 1363 us
    //                        against 1438; 4: 687 against 736; 5 of uneven length: 740 against 741)
    //   129 to 255 rows      1.01, 0.92 to 1.12
    //   lists under 8192     1.04, to 1.15 (16 of 1000, all tokens: 323 us against 300)
    //   empty second halves  1.13, to 1.33 (64 x 300 rows over 4096: 768 us against 595)
    //   fewer workgroups     1.01, 0.91 to 1.23
    //   64 channels          1.20, 1.08 to 1.30
    const int64_t wide = (p.rows + 255) / 256, narrow = (p.rows + 127) / 128;
    const bool eight = plan->width == 2 && p.rows >= 256 && 2 * wide == narrow && a->L >= kLongList && p.units * wide >= 2 * cu;
    plan->shape = {plan->width, eight ? 8 : 4, p.rows > 64 || plan->width > 2 ? 2 : 1};
    plan->mt = plan->shape.tiles;
    waves_rows = plan->shape.waves;
    fits = rows_per_unit(plan->width, waves_rows);
  } else {
    const int most = plan->width == 3 ? 1 : 2;
    plan->mt = 1;
    while (plan->mt < most && 16 * plan->mt < p.rows) plan->mt *= 2;
    fits = attend_per_unit(plan->width, plan->mt);
  }
  p.group_rows = 16 * plan->mt * waves_rows;
  p.row_groups = (p.rows + p.group_rows - 1) / p.group_rows;
  const int64_t lists = static_cast<int64_t>(p.units) * p.row_groups;
  const int64_t room = static_cast<int64_t>(cu) * (fits < 2 ? fits : 2);
  p.heads = plan->many || tiles * lists <= 8 * room * kAttendWaves ? 1 : a->Hkv % 4 == 0 ? 4 : a->Hkv % 2 == 0 ? 2 : 1;
  const int64_t groups = lists / p.heads;
  int64_t splits = (room + groups - 1) / groups;
  if (groups * splits > static_cast<int64_t>(cu) * fits && splits > 1) splits = static_cast<int64_t>(cu) * fits / groups;
  const int64_t cap = plan->many ? (tiles + 3) / 4 : (tiles + kAttendWaves / p.heads - 1) / (kAttendWaves / p.heads);
  splits = splits > cap ? cap : splits;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits);
  // With many rows XCDs are dealt whole lists where they get equally many, or at least 8 (one more does no harm then),
  // else workgroups.  Workgroups' times over lists', 220 random batches: 1.01 for 8 to 63 lists that 8 divides (one
  // prompt of 8192, 8 lists: 959 us against 857), 1.03 from 64 lists on; 0.94 for 1 to 63 others, down to 0.44.
  // With one row group nothing is read twice, and heads of a slot, which lie side by side in memory, are read on one XCD
  // where there are shares for all 8: 0.99 of lists' time for even numbers of heads (12 trees of 13, 4 heads of 96
  // channels: 69 us against 70), 1.02 for others.  With more row groups that was 1.02 where 8 divided the shares or there
  // were 64, to 1.14 (8 sequences of uneven length, 512 tokens each: 698 us against 620).
  const int64_t shares = static_cast<int64_t>(a->B) * p.splits, all = shares * a->Hkv;
  const bool together = p.row_groups == 1 && a->Hkv % 2 == 0 && (shares % 8 == 0 || shares >= 64);
  p.dealt = together ? 0 : all % 8 == 0 || all >= 64 ? 1 : 2;
  if (lists * (p.splits + 8) > INT32_MAX / 16) return ETS_ERR_INVALID_ARG;
  // one launch, of fewer than 2^32 lanes
  if ((plan->many ? attend_rows_groups(p) * 64 * waves_rows : attend_groups(p) * kAttendThreads) > UINT32_MAX) return ETS_ERR_INVALID_ARG;
  p.scale_log2 = static_cast<float>(1.4426950408889634074 / __builtin_sqrt(static_cast<double>(a->D)));
  p.by_page = fast_div(a->page_size);
  p.by_block = fast_div(a->block);
  p.by_heads = fast_div(a->Hkv);
  p.by_tokens = fast_div(a->T);
  p.by_groups = fast_div(p.row_groups);
  p.by_splits = fast_div(p.splits);
  p.by_G = fast_div(p.G);
  p.by_inner = fast_div(a->Hkv / p.heads * p.row_groups);
  p.by_rows = fast_div(p.group_rows);
  p.join_lanes = static_cast<int64_t>(p.units) * p.rows < 2 * cu && p.splits > 16 ? 8 : a->Dv / 4;
  const int most_groups = kAttendThreads / p.join_lanes;
  p.join_groups = p.splits / 4 < most_groups ? (p.splits / 4 > 1 ? p.splits / 4 : 1) : most_groups;
  p.join_parts = kAttendThreads / (p.join_lanes * p.join_groups);
  p.by_lanes = fast_div(p.join_lanes);
  p.by_parts = fast_div(a->Dv / 4 / p.join_lanes);
  p.by_unit_rows = fast_div(p.rows);
  if (p.splits > 1) plan->bytes = static_cast<size_t>(lists) * p.splits * p.group_rows * (a->Dv * 4 + 8);
  return ETS_OK;
}

template <class T, int N, int MT>
void launch_blocks(const AttendBlocksParams& p, hipStream_t s) {
  const size_t lds = kAttendWaves * kAttendTile * (2 * value_plane(N) + 16) + kAttendWaves * (MT + 1) * 16 * sizeof(f32x2) +
                     3 * kChunk * kAttendTile * 4;
  const uint32_t grid = attend_grid(p);
  if (p.a.D == 64 * N && p.a.Dv == 64 * N) {
    hipLaunchKernelGGL((attend_kernel<T, N, N, MT, true, true>), dim3(grid), dim3(kAttendThreads), lds, s, p);
  } else {
    hipLaunchKernelGGL((attend_kernel<T, N, N, MT, false, true>), dim3(grid), dim3(kAttendThreads), lds, s, p);
  }
}

template <class T, int N>
void launch_width(const BlocksPlan& plan, hipStream_t s) {
  if (plan.mt == 1) {
    launch_blocks<T, N, 1>(plan.p, s);
  } else if constexpr (N != 3) {
    launch_blocks<T, N, 2>(plan.p, s);
  }
}

template <class T>
void launch_type(const BlocksPlan& plan, hipStream_t s) {
  const AttendBlocksParams& p = plan.p;
  if (plan.many) {
    launch_attend_rows(p, plan.shape, s);
  } else {
    switch (plan.width) {
      case 1: launch_width<T, 1>(plan, s); break;
      case 2: launch_width<T, 2>(plan, s); break;
      case 3: launch_width<T, 3>(plan, s); break;
      default: launch_width<T, 4>(plan, s);
    }
  }
  if (p.splits > 1) {
    const int64_t parts = static_cast<int64_t>(p.units) * p.rows * p.by_parts.d;
    hipLaunchKernelGGL(join_kernel<T>, dim3(static_cast<uint32_t>((parts + p.join_parts - 1) / p.join_parts)), dim3(kAttendThreads), 0, s,
                       static_cast<const AttendParams&>(p));
  }
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_attend_blocks_workspace_size(const ets_attend_blocks_args* args, size_t* bytes) {
  if (!bytes) return ETS_ERR_INVALID_ARG;
  ets::BlocksPlan plan;
  if (ets_status st = ets::make_plan(args, &plan); st != ETS_OK) return st;
  *bytes = plan.bytes;
  return ETS_OK;
}

ets_status ets_attend_blocks(const ets_attend_blocks_args* args, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ets;
  BlocksPlan plan;
  if (ets_status st = make_plan(args, &plan); st != ETS_OK) return st;
  const ets_attend_args& a = plan.p.a;
  if (a.B == 0 || a.T == 0) return ETS_OK;
  if (!a.q || !a.out || !a.lse || !a.seq_lens || (a.L && !a.page_table) ||
      (a.S && (!a.k_codes || !a.k_scales || !a.v_codes || !a.v_scales)))
    return ETS_ERR_INVALID_ARG;
  if (plan.bytes) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || workspace_bytes < plan.bytes) return ETS_ERR_WORKSPACE;
    plan.p.part = static_cast<float*>(workspace);
    const int64_t rows = static_cast<int64_t>(plan.p.units) * plan.p.row_groups * plan.p.splits * plan.p.group_rows;
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
