// ets_attend.hip -- attention of one or a few tokens a sequence over an 8-bit
// cache: over selected slots or over whole paged sequences, plus a tree of
// drafted tokens (gfx950).
#include "ets_attend.h"

namespace ets {
namespace {

constexpr int kThreads = kAttendThreads;
constexpr int kWaves = kAttendWaves;
constexpr int kTile = kAttendTile;

// One wave goes over its tiles of 32 keys alone, with the running largest
// score and sum of the softmax, and the four waves of a workgroup join at the
// end.
//
// Scores are formed as K Q^T: a lane holds a head (l % 16) and 8 of the 32
// keys, so a head's statistics are per lane (two row swaps join the four lanes
// that share a head), and the probabilities are already laid out as the right
// operand of the second product, out^T = V^T P^T, whose columns are heads
// again: the running rescale is one factor a lane.  Which key stands at which
// place of the inner dimension is free, and V^T follows the places that the
// first product leaves.
//
// Keys go from global memory straight into operands (16 consecutive codes a
// lane and 64 channels).  Values are brought to bf16, which holds them
// exactly, stored row by row in the wave's part of LDS, and read back
// transposed (ds_read_b64_tr_b16).
//
// fp16 queries keep their probabilities as the sum of two bf16 numbers (16
// bits), bf16 queries as one (8 bits: each is off by at most 2^-8 of itself,
// the errors of different keys are independent, and the result is rounded to
// 8 bits anyway).
template <class T, int NP, int NV, int MT>
__global__ __launch_bounds__(kThreads) void attend_kernel(AttendParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  constexpr int W = (NP + 1) / 2, WV = (NV + 1) / 2;
  constexpr int kPitch = NV * 128 + 32;  // bytes of a row of values in LDS
  constexpr bool kTwo = M::kRowScale;    // fp16: two-part probabilities
  extern __shared__ __align__(16) char lds[];
  const ets_attend_args& a = p.a;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  char* values = lds + wave * (kTile * kPitch);
  f32x2* stats = reinterpret_cast<f32x2*>(lds + kWaves * kTile * kPitch);  // [wave][16 MT]

  const AttendSpot spot = attend_spot(p);
  const int b = spot.b, hk = spot.hk, row0 = spot.row0, main_tiles = spot.main_tiles, last = spot.last;

  // queries: lane (head col, row g) holds channels 64 i + 16 g + 0..7, 8..15
  V8 q[MT][NP][2];
  uint64_t tree_bits[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + 16 * m + col;
    int t, h;
    attend_row(p, spot, r, &t, &h);
    const char* src = static_cast<const char*>(a.q) + 2 * (b * a.q_b + t * a.q_t + h * a.q_h);
    tree_bits[m] = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      q[m][i][0] = V8{};
      q[m][i][1] = V8{};
    }
    if (r < p.rows) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (64 * i + 16 * g < a.D) {
          q[m][i][0] = load_any<V8>(src + 128 * i + 32 * g);
          q[m][i][1] = load_any<V8>(src + 128 * i + 32 * g + 16);
        }
      }
      if (a.tree_slots) tree_bits[m] = static_cast<uint64_t>(a.tree_mask[b * a.mask_b + t]);
    }
  }

  // slot of the key that this lane loads: 16 s + col of tile i
  auto slot_of = [&](int i, int s) { return attend_slot(p, spot, i, 16 * s + col, attend_ask(p, spot, i, 16 * s + col)); };

  const int nbk = a.D / kCacheBlock, nbv = a.Dv / kCacheBlock;
  const uint8_t* kc = a.k_codes + hk * a.k_h + 16 * g;
  const uint8_t* ks = a.k_scales + hk * a.ks_h;
  const uint8_t* vc = a.v_codes + hk * a.v_h + 16 * g;
  const uint8_t* vs = a.v_scales + hk * a.vs_h;
  u32v4 kraw[2][NP], vraw[2][NV];
  uint32_t ksc[2][W], vsc[2][WV];
  uint32_t seen = 0;  // keys of the fetched tile that are inside the cache
  auto fetch = [&](const int32_t (&slot)[2]) {
    const uint64_t s0 = __ballot(slot[0] >= 0), s1 = __ballot(slot[1] >= 0);
    seen = static_cast<uint32_t>(s0 & 0xffff) | static_cast<uint32_t>(s1 & 0xffff) << 16;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < NP; ++i) kraw[s][i] = u32v4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < W; ++i) ksc[s][i] = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) vraw[s][i] = u32v4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < WV; ++i) vsc[s][i] = 0;
      if (slot[s] >= 0) {
        const int64_t at = slot[s];
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (64 * i + 16 * g < a.D) kraw[s][i] = load_any<u32v4>(kc + at * a.k_s + 64 * i);
        load_scales<W>(ksc[s], ks + at * a.ks_s, nbk);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (64 * i + 16 * g < a.Dv) vraw[s][i] = load_any<u32v4>(vc + at * a.v_s + 64 * i);
        load_scales<WV>(vsc[s], vs + at * a.vs_s, nbv);
      }
    }
  };

  f32x4 out[MT][4 * NV];
  float top[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    top[m] = kNegInf, sum[m] = 0.0f;
#pragma unroll
    for (int c = 0; c < 4 * NV; ++c) out[m][c] = f32x4{};
  }

  int tile = spot.first + wave;
  int32_t slot[2] = {-1, -1};
  if (tile < last) {
    slot[0] = slot_of(tile, 0), slot[1] = slot_of(tile, 1);
    fetch(slot);
    slot[0] = slot_of(tile + kWaves, 0), slot[1] = slot_of(tile + kWaves, 1);
  }
  for (; tile < last; tile += kWaves) {
    // keys to operands, values to LDS
    f32x4 score[MT][2];
    float row_scale[2];
    const uint32_t seen_now = seen;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t r = M::kRowScale ? scales_max<W>(ksc[s]) : 0;
      row_scale[s] = __uint_as_float(r << 23);
#pragma unroll
      for (int m = 0; m < MT; ++m) score[m][s] = f32x4{};
      char* dst = values + (16 * s + col) * kPitch + 32 * g;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t byte = byte_of(ksc[s][i / 2], 16 * (i & 1) + 8 * (g >> 1));
        const float f = M::scale(byte, r);
        const u32v4 c = kraw[s][i];
        const V8 k0 = M::keys(c[0], c[1], f), k1 = M::keys(c[2], c[3], f);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          score[m][s] = M::mma(k0, q[m][i][0], score[m][s]);
          score[m][s] = M::mma(k1, q[m][i][1], score[m][s]);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float f = __uint_as_float(byte_of(vsc[s][i / 2], 16 * (i & 1) + 8 * (g >> 1)) << 23);
        const u32v4 c = vraw[s][i];
        store_any(__builtin_assume_aligned(dst + 128 * i, 16), codes_bf16(c[0], c[1], f));
        store_any(__builtin_assume_aligned(dst + 128 * i + 16, 16), codes_bf16(c[2], c[3], f));
      }
    }
    // the next tile's rows are on their way while this one is worked on
    if (tile + kWaves < last) {
      fetch(slot);
      slot[0] = slot_of(tile + 2 * kWaves, 0), slot[1] = slot_of(tile + 2 * kWaves, 1);
    }
    if constexpr (M::kRowScale) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = __uint_as_float(__builtin_amdgcn_ds_bpermute(4 * (4 * g + e), __float_as_uint(row_scale[s])));
#pragma unroll
          for (int m = 0; m < MT; ++m) score[m][s][e] *= f;
        }
    }

    bf16x8 prob[MT], rest[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t vis = seen_now;
      if (tile >= main_tiles) vis &= static_cast<uint32_t>(tree_bits[m] >> (kTile * (tile - main_tiles)));
      vis >>= 4 * g;  // bits 0..3: keys 4 g + e; bits 16..19: keys 16 + 4 g + e
      float x[8], high = kNegInf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = score[m][j >> 2][j & 3] * p.scale_log2;
        x[j] = (vis >> (16 * (j >> 2) + (j & 3))) & 1 ? x[j] : kNegInf;
        high = fmaxf(high, x[j]);
      }
      high = fmaxf(rows_max(high), top[m]);
      const float base = high == kNegInf ? 0.0f : high;
      if (__any(high > top[m])) {
        const float fade = __builtin_amdgcn_exp2f(top[m] - base);
        sum[m] *= fade;
#pragma unroll
        for (int c = 0; c < 4 * NV; ++c) out[m][c] *= fade;
        top[m] = high;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = __builtin_amdgcn_exp2f(x[j] - base);
        sum[m] += x[j];
        prob[m][j] = static_cast<__bf16>(x[j]);
        if constexpr (kTwo) rest[m][j] = static_cast<__bf16>(x[j] - static_cast<float>(prob[m][j]));
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const char* src = values + (4 * g + (col >> 2)) * kPitch + 8 * (col & 3);
#pragma unroll
    for (int c = 0; c < 4 * NV; ++c) {
      typedef __attribute__((address_space(3))) s16x4* Lds4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(src + 32 * c));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(src + 16 * kPitch + 32 * c));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const bf16x8 v = __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        out[m][c] = Mat<__bf16>::mma(v, prob[m], out[m][c]);
        if constexpr (kTwo) out[m][c] = Mat<__bf16>::mma(v, rest[m], out[m][c]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }

  // join the waves
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    sum[m] = rows_sum(sum[m]);
    if (g == 0) stats[(wave * MT + m) * 16 + col] = f32x2{top[m], sum[m]};
  }
  __syncthreads();
  const int64_t block = blockIdx.x;
  const int dv = a.Dv;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float high = kNegInf, total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) high = fmaxf(high, stats[(w * MT + m) * 16 + col][0]);
    const float base = high == kNegInf ? 0.0f : high;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const f32x2 s = stats[(w * MT + m) * 16 + col];
      total += s[1] * __builtin_amdgcn_exp2f(s[0] - base);
    }
    const float fade = __builtin_amdgcn_exp2f(top[m] - base);
    // the wave's sums, [head][64 NV] floats, over its own values
    f32x4* mine = reinterpret_cast<f32x4*>(values) + col * (16 * NV) + g;
#pragma unroll
    for (int c = 0; c < 4 * NV; ++c) mine[4 * c] = out[m][c] * fade;
    if (wave == 0 && g == 0) stats[(kWaves * MT + m) * 16 + col] = f32x2{high, total};
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 16 * NV; i += kThreads) {
      const int head = i / (16 * NV), c = (i - head * (16 * NV)) * 4;
      const int r = row0 + 16 * m + head;
      if (r >= p.rows || c >= dv) continue;
      f32x4 v = {};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        v += reinterpret_cast<const f32x4*>(lds + w * (kTile * kPitch))[i];
      const f32x2 s = stats[(kWaves * MT + m) * 16 + head];
      if (p.splits > 1) {
        const int64_t at = block * (16 * MT) + 16 * m + head;
        store_any(p.part + at * dv + c, v);
        if (c == 0) p.stat[at] = s;
      } else {
        int t, h;
        attend_row(p, spot, r, &t, &h);
        const int64_t at = (static_cast<int64_t>(b) * a.T + t) * a.Hq + h;
        const float inv = attend_inverse(s[1]);
        typedef T V4 __attribute__((ext_vector_type(4)));
        V4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(v[e] * inv);
        store_any(static_cast<T*>(a.out) + at * dv + c, y);
        if (c == 0) a.lse[at] = attend_lse(s[0], s[1]);
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a list.  A lane stands at four channels of one row; Dv / 4
// lanes by `groups` shares of the splits take the row, and a workgroup as many
// rows as it has lanes for.
template <class T>
__global__ __launch_bounds__(kThreads) void join_kernel(AttendParams p) {
  const ets_attend_args& a = p.a;
  __shared__ f32x4 sums[kThreads];
  __shared__ f32x2 joined[kThreads];
  const int lanes = a.Dv / 4;
  const int slot = static_cast<int>(div_by(threadIdx.x, p.by_lanes));  // row and share
  const int ch = 4 * (static_cast<int>(threadIdx.x) - slot * lanes);
  const int my_row = slot / p.join_groups, mine = slot - my_row * p.join_groups;
  const int64_t index = static_cast<int64_t>(blockIdx.x) * p.join_rows + my_row;
  const bool live = my_row < p.join_rows && index < static_cast<int64_t>(p.units) * p.rows;
  const uint32_t unit = live ? div_by(static_cast<uint32_t>(index), p.by_unit_rows) : 0;
  const int r = live ? static_cast<int>(index - static_cast<int64_t>(unit) * p.rows) : 0;
  const int group = static_cast<int>(div_by(r, p.by_rows)), in_group = r - group * p.group_rows;
  const int64_t at0 = (static_cast<int64_t>(unit) * p.row_groups + group) * p.splits * p.group_rows + in_group;
  float high = kNegInf, total = 0.0f;
  f32x4 v = {};
  if (live) {
#pragma unroll 4
    for (int s = mine; s < p.splits; s += p.join_groups) high = fmaxf(high, p.stat[at0 + static_cast<int64_t>(s) * p.group_rows][0]);
    const float base = high == kNegInf ? 0.0f : high;
#pragma unroll 4
    for (int s = mine; s < p.splits; s += p.join_groups) {
      const int64_t at = at0 + static_cast<int64_t>(s) * p.group_rows;
      const f32x2 st = p.stat[at];
      const float f = __builtin_amdgcn_exp2f(st[0] - base);
      total += st[1] * f;
      v += load_any<f32x4>(p.part + at * a.Dv + ch) * f;
    }
  }
  if (p.join_groups > 1) {
    sums[threadIdx.x] = v;
    joined[threadIdx.x] = f32x2{high, total};
    __syncthreads();
    if (mine != 0) return;
    for (int i = 1; i < p.join_groups; ++i) high = fmaxf(high, joined[threadIdx.x + i * lanes][0]);
    const float base = high == kNegInf ? 0.0f : high;
    v = f32x4{};
    total = 0.0f;
    for (int i = 0; i < p.join_groups; ++i) {
      const f32x2 st = joined[threadIdx.x + i * lanes];
      const float f = __builtin_amdgcn_exp2f(st[0] - base);
      total += st[1] * f;
      v += sums[threadIdx.x + i * lanes] * f;
    }
  }
  if (!live) return;
  const bool paged = a.slots == nullptr;
  const uint32_t bt = div_by(unit, p.by_heads);
  const int hk = static_cast<int>(unit - bt * a.Hkv);
  const int t = paged ? static_cast<int>(div_by(r, p.by_G)) : 0;
  const int64_t row = (static_cast<int64_t>(bt) * (paged ? a.T : 1) + t) * a.Hq + hk * p.G + (r - t * p.G);
  const float inv = attend_inverse(total);
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(v[e] * inv);
  store_any(static_cast<T*>(a.out) + row * a.Dv + ch, y);
  if (ch == 0) a.lse[row] = attend_lse(high, total);
}

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
  if (paged ? (a->L < 0 || a->page_size < 1) : a->K < 0) return ETS_ERR_INVALID_ARG;
  if (a->tree_slots && a->T > ETS_MAX_TREE) return ETS_ERR_INVALID_ARG;
  // row strides are 32-bit numbers in the wide kernel; 4 GiB from slot to slot is no cache
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
  const int most = plan->width <= 2 ? 4 : 2;
  plan->mt = 1;
  while (plan->mt < most && 16 * plan->mt < p.rows) plan->mt *= 2;
  if (plan->width == 9) plan->mt = attend_wide_rows(p.rows, plan->shared, a->dtype == ETS_BF16);
  p.group_rows = 16 * plan->mt;
  p.row_groups = (p.rows + p.group_rows - 1) / p.group_rows;
  p.tree_tiles = a->tree_slots ? (a->T + kTile - 1) / kTile : 0;
  const int tiles = ((paged ? a->L : a->K) + kTile - 1) / kTile + p.tree_tiles;
  const int64_t lists = static_cast<int64_t>(p.units) * p.row_groups;
  // enough workgroups for two a compute unit (one of the wide kernel's), each wave with a tile at least
  int64_t splits = ((plan->width == 9 ? 1 : 2) * static_cast<int64_t>(cu) + lists - 1) / lists;
  const int64_t cap = plan->width == 9 ? (tiles + 3) / 4 : (tiles + kWaves - 1) / kWaves;
  splits = splits > cap ? cap : splits;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits);
  if (lists * p.splits > INT32_MAX / 16) return ETS_ERR_INVALID_ARG;
  p.scale_log2 = static_cast<float>(1.4426950408889634074 / __builtin_sqrt(static_cast<double>(a->D)));
  p.by_page = fast_div(paged ? a->page_size : 1);
  p.by_heads = fast_div(a->Hkv);
  p.by_tokens = fast_div(a->T);
  p.by_groups = fast_div(p.row_groups);
  p.by_splits = fast_div(p.splits);
  p.by_G = fast_div(p.G);
  p.by_rows = fast_div(p.group_rows);
  const int lanes = a->Dv / 4;
  p.join_groups = kThreads / lanes < p.splits / 4 ? kThreads / lanes : p.splits / 4 > 1 ? p.splits / 4 : 1;
  p.join_rows = kThreads / (lanes * p.join_groups);
  p.by_lanes = fast_div(lanes);
  p.by_unit_rows = fast_div(p.rows);
  if (p.splits > 1) plan->bytes = static_cast<size_t>(lists) * p.splits * 16 * plan->mt * (a->Dv * 4 + 8);
  return ETS_OK;
}

template <class T, int N, int MT>
void launch_attend(const AttendParams& p, hipStream_t s) {
  const size_t lds = kWaves * kTile * (N * 128 + 32) + (kWaves + 1) * MT * 16 * sizeof(f32x2);
  const uint32_t grid = static_cast<uint32_t>(static_cast<int64_t>(p.units) * p.row_groups * p.splits);
  hipLaunchKernelGGL((attend_kernel<T, N, N, MT>), dim3(grid), dim3(kThreads), lds, s, p);
}

template <class T, int N>
void launch_width(const Plan& plan, hipStream_t s) {
  if (plan.mt == 1) {
    launch_attend<T, N, 1>(plan.p, s);
  } else if (plan.mt == 2) {
    launch_attend<T, N, 2>(plan.p, s);
  } else if constexpr (N <= 2) {
    launch_attend<T, N, 4>(plan.p, s);
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
    const int64_t rows = static_cast<int64_t>(p.units) * p.rows;
    hipLaunchKernelGGL(join_kernel<T>, dim3(static_cast<uint32_t>((rows + p.join_rows - 1) / p.join_rows)), dim3(kThreads), 0, s, p);
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
