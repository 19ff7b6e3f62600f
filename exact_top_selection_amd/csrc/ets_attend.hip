// ets_attend.hip -- attention of one or a few tokens a sequence over an 8-bit
// cache: over selected slots or over whole paged sequences, plus a tree of
// drafted tokens (gfx950).
#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 32;  // keys of a wave's step
constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.69314718055994530942f;

struct AttendParams {
  ets_attend_args a;
  int G;             // query heads of a cache head
  int rows;          // query rows that share a list of keys: G, or T * G where all tokens share it
  int units;         // lists: (b, t, hk) or (b, hk)
  int row_groups;    // of a unit
  int splits;        // workgroups that share a list
  int tree_tiles;
  float scale_log2;  // log2(e) / sqrt(D)
  FastDiv by_page, by_heads, by_tokens, by_groups, by_splits, by_G;
  float* part;       // [unit][row group][split][16 * MT][Dv] sums
  f32x2* stat;       // [unit][row group][split][16 * MT] (largest, sum)
};

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
// transposed (ds_read_b64_tr_b16).  With SHARED the values are the keys' first
// Dv channels and are loaded once for both.
//
// fp16 queries keep their probabilities as the sum of two bf16 numbers (16
// bits), bf16 queries as one (8 bits: each is off by at most 2^-8 of itself,
// the errors of different keys are independent, and the result is rounded to
// 8 bits anyway).
template <class T, int NP, int NV, bool SHARED, int MT>
__global__ __launch_bounds__(kThreads) void attend_kernel(AttendParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  constexpr int W = (NP + 1) / 2, WV = (NV + 1) / 2;
  constexpr int NVR = SHARED ? 1 : NV, WVR = SHARED ? 1 : WV;
  constexpr int kPitch = NV * 128 + 32;  // bytes of a row of values in LDS
  constexpr bool kTwo = M::kRowScale;    // fp16: two-part probabilities
  extern __shared__ __align__(16) char lds[];
  const ets_attend_args& a = p.a;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  char* values = lds + wave * (kTile * kPitch);
  f32x2* stats = reinterpret_cast<f32x2*>(lds + kWaves * kTile * kPitch);  // [wave][16 MT]

  // blocks: split fastest, then row group, then unit
  const uint32_t ug = div_by(blockIdx.x, p.by_splits);
  const int split = static_cast<int>(blockIdx.x - ug * p.splits);
  const uint32_t unit = div_by(ug, p.by_groups);
  const int row0 = static_cast<int>(ug - unit * p.row_groups) * (16 * MT);
  const bool paged = a.slots == nullptr;
  const uint32_t bt = div_by(unit, p.by_heads);
  const int hk = static_cast<int>(unit - bt * a.Hkv);
  const int b = paged ? static_cast<int>(bt) : static_cast<int>(div_by(bt, p.by_tokens));
  const int t_unit = paged ? 0 : static_cast<int>(bt) - b * a.T;

  const int n = paged ? min(max(a.seq_lens[b], 0), a.L) : a.K;
  const int main_tiles = (n + kTile - 1) / kTile, tiles = main_tiles + p.tree_tiles;
  const int per = (tiles + p.splits - 1) / p.splits;
  const int first = split * per, last = min(first + per, tiles);

  // queries: lane (head col, row g) holds channels 64 i + 16 g + 0..7, 8..15
  V8 q[MT][NP][2];
  uint64_t tree_bits[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + 16 * m + col;
    const int t = paged ? static_cast<int>(div_by(r, p.by_G)) : t_unit;
    const int h = hk * p.G + (paged ? r - t * p.G : r);
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

  // slot of the key that this lane loads: 16 s + col of tile i; -1 outside
  auto slot_of = [&](int i, int s) -> int32_t {
    int64_t slot = -1;
    if (i < main_tiles) {
      const int j = i * kTile + 16 * s + col;
      if (j < n) {
        if (paged) {
          const uint32_t page = div_by(j, p.by_page);
          slot = static_cast<int64_t>(a.page_table[b * a.pt_b + page]) * a.page_size + (j - page * p.by_page.d);
        } else {
          slot = a.slots[b * a.slots_b + t_unit * a.slots_t + j];
        }
      }
    } else {
      const int j = (i - main_tiles) * kTile + 16 * s + col;
      // one token's list leaves out what the token does not see, so nothing of it is read
      if (i < tiles && j < a.T && (paged || (a.tree_mask[b * a.mask_b + t_unit] >> j & 1)))
        slot = a.tree_slots[b * a.tree_b + j];
    }
    return slot >= 0 && slot < a.S ? static_cast<int32_t>(slot) : -1;
  };

  const int nbk = a.D / kCacheBlock, nbv = a.Dv / kCacheBlock;
  const uint8_t* kc = a.k_codes + hk * a.k_h + 16 * g;
  const uint8_t* ks = a.k_scales + hk * a.ks_h;
  const uint8_t* vc = a.v_codes + hk * a.v_h + 16 * g;
  const uint8_t* vs = a.v_scales + hk * a.vs_h;
  u32v4 kraw[2][NP], vraw[2][NVR];
  uint32_t ksc[2][W], vsc[2][WVR];
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
      for (int i = 0; i < NVR; ++i) vraw[s][i] = u32v4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < WVR; ++i) vsc[s][i] = 0;
      if (slot[s] >= 0) {
        const int64_t at = slot[s];
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (64 * i + 16 * g < a.D) kraw[s][i] = load_any<u32v4>(kc + at * a.k_s + 64 * i);
        load_scales<W>(ksc[s], ks + at * a.ks_s, nbk);
        if constexpr (!SHARED) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (64 * i + 16 * g < a.Dv) vraw[s][i] = load_any<u32v4>(vc + at * a.v_s + 64 * i);
          load_scales<WV>(vsc[s], vs + at * a.vs_s, nbv);
        }
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

  int tile = first + wave;
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
        if constexpr (SHARED) {
          if (i < NV) {
            if constexpr (kTwo) {
              const float fv = __uint_as_float(byte << 23);
              store_any(__builtin_assume_aligned(dst + 128 * i, 16), codes_bf16(c[0], c[1], fv));
              store_any(__builtin_assume_aligned(dst + 128 * i + 16, 16), codes_bf16(c[2], c[3], fv));
            } else {
              store_any(__builtin_assume_aligned(dst + 128 * i, 16), k0);
              store_any(__builtin_assume_aligned(dst + 128 * i + 16, 16), k1);
            }
          }
        }
      }
      if constexpr (!SHARED) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float f = __uint_as_float(byte_of(vsc[s][i / 2], 16 * (i & 1) + 8 * (g >> 1)) << 23);
          const u32v4 c = vraw[s][i];
          store_any(__builtin_assume_aligned(dst + 128 * i, 16), codes_bf16(c[0], c[1], f));
          store_any(__builtin_assume_aligned(dst + 128 * i + 16, 16), codes_bf16(c[2], c[3], f));
        }
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
        const int t = paged ? static_cast<int>(div_by(r, p.by_G)) : t_unit;
        const int64_t at = (static_cast<int64_t>(b) * a.T + t) * a.Hq + hk * p.G + (paged ? r - t * p.G : r);
        const float inv = s[1] > 0.0f || s[1] != s[1] ? 1.0f / s[1] : 0.0f;
        typedef T V4 __attribute__((ext_vector_type(4)));
        V4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(v[e] * inv);
        store_any(static_cast<T*>(a.out) + at * dv + c, y);
        if (c == 0) a.lse[at] = s[1] == 0.0f ? kNegInf : (s[0] + __builtin_amdgcn_logf(s[1])) * kLn2;
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a list: one wave a row.
template <class T, int MT>
__global__ __launch_bounds__(kThreads) void join_kernel(AttendParams p) {
  const ets_attend_args& a = p.a;
  const int lane = threadIdx.x & 63;
  const uint32_t i = blockIdx.x * kWaves + (threadIdx.x >> 6);  // unit * row_groups * 16 MT rows
  const uint32_t ug = i / (16 * MT);
  const int in_group = static_cast<int>(i - ug * (16 * MT));
  if (ug >= static_cast<uint32_t>(p.units) * p.row_groups) return;
  const uint32_t unit = div_by(ug, p.by_groups);
  const int r = static_cast<int>(ug - unit * p.row_groups) * (16 * MT) + in_group;
  if (r >= p.rows) return;
  const bool paged = a.slots == nullptr;
  const uint32_t bt = div_by(unit, p.by_heads);
  const int hk = static_cast<int>(unit - bt * a.Hkv);
  const int64_t at0 = static_cast<int64_t>(ug) * p.splits * (16 * MT) + in_group;
  float high = kNegInf;
  for (int s = lane; s < p.splits; s += 64) high = fmaxf(high, p.stat[at0 + s * (16 * MT)][0]);
#pragma unroll
  for (int o = 32; o; o >>= 1) high = fmaxf(high, __shfl_xor(high, o));
  const float base = high == kNegInf ? 0.0f : high;
  float total = 0.0f;
  f32x4 v[3] = {};
  for (int s = 0; s < p.splits; ++s) {
    const int64_t at = at0 + s * (16 * MT);
    const f32x2 st = p.stat[at];
    const float f = __builtin_amdgcn_exp2f(st[0] - base);
    total += st[1] * f;
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (256 * j + 4 * lane < a.Dv) v[j] += load_any<f32x4>(p.part + at * a.Dv + 256 * j + 4 * lane) * f;
  }
  const int64_t row = paged ? (static_cast<int64_t>(bt) * a.T + div_by(r, p.by_G)) * a.Hq + hk * p.G + (r - div_by(r, p.by_G) * p.G)
                            : static_cast<int64_t>(bt) * a.Hq + hk * p.G + r;
  const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    if (256 * j + 4 * lane < a.Dv) {
      typedef T V4 __attribute__((ext_vector_type(4)));
      V4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(v[j][e] * inv);
      store_any(static_cast<T*>(a.out) + row * a.Dv + 256 * j + 4 * lane, y);
    }
  }
  if (lane == 0) a.lse[row] = total == 0.0f ? kNegInf : (high + __builtin_amdgcn_logf(total)) * kLn2;
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
  const int most = plan->width <= 2 ? 4 : plan->width <= 4 ? 2 : 1;
  plan->mt = 1;
  while (plan->mt < most && 16 * plan->mt < p.rows) plan->mt *= 2;
  p.row_groups = (p.rows + 16 * plan->mt - 1) / (16 * plan->mt);
  p.tree_tiles = a->tree_slots ? (a->T + kTile - 1) / kTile : 0;
  const int tiles = ((paged ? a->L : a->K) + kTile - 1) / kTile + p.tree_tiles;
  const int64_t lists = static_cast<int64_t>(p.units) * p.row_groups;
  // enough workgroups for two a compute unit, each wave with a tile at least
  int64_t splits = (2 * static_cast<int64_t>(cu) + lists - 1) / lists;
  const int64_t cap = (tiles + kWaves - 1) / kWaves;
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
  if (p.splits > 1) plan->bytes = static_cast<size_t>(lists) * p.splits * 16 * plan->mt * (a->Dv * 4 + 8);
  return ETS_OK;
}

template <class T, int NP, int NV, bool SHARED, int MT>
void launch_attend(const Plan& plan, hipStream_t s) {
  const AttendParams& p = plan.p;
  const size_t lds = kWaves * kTile * (NV * 128 + 32) + (kWaves + 1) * MT * 16 * sizeof(f32x2);
  const int64_t lists = static_cast<int64_t>(p.units) * p.row_groups;
  hipLaunchKernelGGL((attend_kernel<T, NP, NV, SHARED, MT>), dim3(static_cast<uint32_t>(lists * p.splits)),
                     dim3(kThreads), lds, s, p);
  if (p.splits > 1)
    hipLaunchKernelGGL((join_kernel<T, MT>), dim3(static_cast<uint32_t>((lists * 16 * MT + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, s, p);
}

template <class T, int N>
void launch_width(const Plan& plan, hipStream_t s) {
  if (plan.mt == 1) {
    launch_attend<T, N, N, false, 1>(plan, s);
  } else if (plan.mt == 2) {
    launch_attend<T, N, N, false, 2>(plan, s);
  } else if constexpr (N <= 2) {
    launch_attend<T, N, N, false, 4>(plan, s);
  }
}

template <class T>
void launch_type(const Plan& plan, hipStream_t s) {
  switch (plan.width) {
    case 1: launch_width<T, 1>(plan, s); break;
    case 2: launch_width<T, 2>(plan, s); break;
    case 3: launch_width<T, 3>(plan, s); break;
    case 4: launch_width<T, 4>(plan, s); break;
    default:
      if (plan.shared) {
        launch_attend<T, 9, 8, true, 1>(plan, s);
      } else {
        launch_attend<T, 9, 9, false, 1>(plan, s);
      }
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
