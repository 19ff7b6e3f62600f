// ets_attend_wide.hip -- attention over an 8-bit cache for heads of 257 to 576
// channels, one latent head shared by many query heads above all (gfx950).
#include "ets_attend.h"

namespace ets {
namespace {

constexpr int kPairs = 9;              // 64-channel steps of a key
constexpr int kPitch = kPairs * 64;    // bytes of a row of codes in LDS
constexpr int kBlocks = 2 * kPairs;    // scale bytes of a row
constexpr int kTile = kAttendTile;
constexpr int kChunks = 5;             // 16-byte pieces of a tile that a lane brings: ceil(32 * 36 / 256)
constexpr float kSlack = 8.0f;         // how far (log2) a score may pass the reference before sums are rescaled

// Position of 16-byte piece c of row k in LDS: rows lie 576 bytes (16 banks)
// apart, and the exchange of pieces inside each 64 bytes spreads the 16 rows
// that one operand load touches over all 64 banks.
__device__ __forceinline__ int place(int k, int c) {
  return k * kPitch + 16 * (c ^ ((k >> 2) & 3));
}

template <int RT, int NC, bool SHARED, bool TWO>
struct WideLds {
  uint8_t k[3][kTile * kPitch];
  uint8_t v[SHARED ? 1 : 3][SHARED ? 16 : kTile * kPitch];
  float ks[3][kBlocks][kTile];                                             // scale of a block of a key, by key
  float vs[SHARED && !TWO ? 1 : 3][SHARED && !TWO ? 1 : kBlocks][kTile];
  float rs[TWO ? 3 : 1][kTile];                                            // fp16: scale of a key's whole row
  u32v4 prob[2][TWO ? 2 : 1][RT][64];
  float fade[2][RT][16];
  int fading[2][RT];
  int32_t slot[8][kTile];
  f32x2 stat[RT * 16];
};

// A workgroup takes 16 RT query rows (all 128 heads of a latent cache with RT
// = 8) through its share of the keys, 32 a step, so that a row of the cache is
// brought once.  Codes go to LDS as they are, through registers, two steps
// ahead.  Scores are formed as K Q^T by the wave that owns the query rows (16
// or 32 of them, in registers); the probabilities go through LDS, and each
// wave then takes a quarter of the channels of out^T = V^T P^T for all rows:
// a value is decoded once, by the wave that uses it, out of the transposed
// byte load (ds_read_b64_tr_b8), whose lanes hold one channel of 8 keys and
// multiply each by its own scale.  One barrier a step; the products of step i
// stand next to the scores of step i + 1.
//
// The softmax is taken relative to a reference that follows the largest score
// only when that passes it by more than 2^8: sums in 32 bits lose nothing by
// it, and the 64 to 256 registers of sums are rescaled once or twice a list.
template <class T, int RT, int NC, bool SHARED>
__global__ __launch_bounds__(kAttendThreads) void attend_wide_kernel(AttendParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  constexpr bool kTwo = M::kRowScale;
  constexpr int MQ = RT / kAttendWaves;  // 16-row tiles whose scores a wave forms
  typedef WideLds<RT, NC, SHARED, kTwo> Lds;
  extern __shared__ __align__(16) char lds_raw[];
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  const ets_attend_args& a = p.a;
  const AttendSpot spot = attend_spot(p);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
  const int steps = max(spot.last - spot.first, 0);

  // rows shorter than 576 leave pieces and scales that are never brought
  for (int i = tid; i < static_cast<int>(sizeof(Lds) / 16); i += kAttendThreads)
    reinterpret_cast<u32v4*>(lds_raw)[i] = u32v4{0, 0, 0, 0};

  V8 q[MQ][kPairs][2];
  uint64_t tree_bits[MQ];
#pragma unroll
  for (int m = 0; m < MQ; ++m) {
    const int r = spot.row0 + 16 * (wave * MQ + m) + col;
    int t, h;
    attend_row(p, spot, r, &t, &h);
    const char* src = static_cast<const char*>(a.q) + 2 * (spot.b * a.q_b + t * a.q_t + h * a.q_h);
    tree_bits[m] = 0;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      q[m][i][0] = V8{};
      q[m][i][1] = V8{};
      if (r < p.rows && 64 * i + 16 * g < a.D) {
        q[m][i][0] = load_any<V8>(src + 128 * i + 32 * g);
        q[m][i][1] = load_any<V8>(src + 128 * i + 32 * g + 16);
      }
    }
    if (r < p.rows && a.tree_slots) tree_bits[m] = static_cast<uint64_t>(a.tree_mask[spot.b * a.mask_b + t]);
  }
  __syncthreads();

  // the pieces of a tile that this lane brings: key (high half) and piece of its row
  const int nbk = a.D / kCacheBlock, nbv = a.Dv / kCacheBlock;
  int piece[kChunks], piece_v[SHARED ? 1 : kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = tid + kAttendThreads * j;
    piece[j] = c < kTile * 2 * nbk ? ((c / (2 * nbk)) << 16) | (c % (2 * nbk)) : -1;
    if constexpr (!SHARED) piece_v[j] = c < kTile * 2 * nbv ? ((c / (2 * nbv)) << 16) | (c % (2 * nbv)) : -1;
  }
  const uint8_t* kc = a.k_codes + spot.hk * a.k_h;
  const uint8_t* ks = a.k_scales + spot.hk * a.ks_h;
  const uint8_t* vc = a.v_codes + spot.hk * a.v_h;
  const uint8_t* vs = a.v_scales + spot.hk * a.vs_h;
  u32v4 kreg[kChunks], vreg[SHARED ? 1 : kChunks];
  uint32_t kword = 0, vword = 0;
  // word w of the scale bytes of a row: lanes 8 k .. 8 k + 7 hold key k's
  auto scale_word = [&](const uint8_t* row, int nb) -> uint32_t {
    const int w = 4 * (tid & 7);
    if (w + 4 <= nb) return load_any<uint32_t>(row + w);
    uint32_t x = 0;
    if (w < nb) x = row[w];
    if (w + 1 < nb) x |= static_cast<uint32_t>(row[w + 1]) << 8;
    if (w + 2 < nb) x |= static_cast<uint32_t>(row[w + 2]) << 16;
    return x;
  };
  auto bring = [&](int i) {  // tile i of the workgroup's share into registers
    const int32_t* slots = lds.slot[i & 7];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      kreg[j] = u32v4{0, 0, 0, 0};
      if (piece[j] >= 0) {
        const int64_t slot = slots[piece[j] >> 16];
        if (slot >= 0) kreg[j] = load_any<u32v4>(kc + slot * a.k_s + 16 * (piece[j] & 0xffff));
      }
      if constexpr (!SHARED) {
        vreg[j] = u32v4{0, 0, 0, 0};
        if (piece_v[j] >= 0) {
          const int64_t slot = slots[piece_v[j] >> 16];
          if (slot >= 0) vreg[j] = load_any<u32v4>(vc + slot * a.v_s + 16 * (piece_v[j] & 0xffff));
        }
      }
    }
    const int64_t slot = slots[tid >> 3];
    kword = 0, vword = 0;
    if (slot >= 0) {
      kword = scale_word(ks + slot * a.ks_s, nbk);
      if constexpr (!SHARED) vword = scale_word(vs + slot * a.vs_s, nbv);
    }
  };
  auto lay = [&](int i) {  // registers into LDS, as tile i
    const int at = i % 3;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      if (piece[j] >= 0) *reinterpret_cast<u32v4*>(lds.k[at] + place(piece[j] >> 16, piece[j] & 0xffff)) = kreg[j];
      if constexpr (!SHARED)
        if (piece_v[j] >= 0) *reinterpret_cast<u32v4*>(lds.v[at] + place(piece_v[j] >> 16, piece_v[j] & 0xffff)) = vreg[j];
    }
    uint32_t top = 0;
    if constexpr (kTwo) {
      const uint32_t one[1] = {kword};
      top = scales_max<1>(one);
      for (int o = 1; o < 8; o <<= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
      if ((tid & 7) == 0) lds.rs[at][tid >> 3] = __uint_as_float(top << 23);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = 4 * (tid & 7) + e;
      if (b < kBlocks) {
        const uint32_t byte = byte_of(kword, 8 * e);
        lds.ks[at][b][tid >> 3] = M::scale(byte, top);
        if constexpr (SHARED && kTwo) lds.vs[at][b][tid >> 3] = __uint_as_float(byte << 23);
        if constexpr (!SHARED) lds.vs[at][b][tid >> 3] = __uint_as_float(byte_of(vword, 8 * e) << 23);
      }
    }
  };
  auto find = [&](int i) {  // slots of tile i, by the first 32 lanes
    return i < steps ? attend_slot(p, spot, spot.first + i, tid & 31) : -1;
  };

  float ref[MQ], sum[MQ];
#pragma unroll
  for (int m = 0; m < MQ; ++m) ref[m] = kNegInf, sum[m] = 0.0f;
  // scores and probabilities of tile i
  auto scores = [&](int i) {
    const int at = i % 3, half = i & 1, tile = spot.first + i;
    f32x4 x[MQ][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int m = 0; m < MQ; ++m) x[m][s] = f32x4{};
#pragma unroll
      for (int c = 0; c < kPairs; ++c) {
        const u32v4 w = *reinterpret_cast<const u32v4*>(lds.k[at] + place(16 * s + col, 4 * c + g));
        const float f = lds.ks[at][2 * c + (g >> 1)][16 * s + col];
        const V8 k0 = M::keys(w[0], w[1], f), k1 = M::keys(w[2], w[3], f);
#pragma unroll
        for (int m = 0; m < MQ; ++m) {
          x[m][s] = M::mma(k0, q[m][c][0], x[m][s]);
          x[m][s] = M::mma(k1, q[m][c][1], x[m][s]);
        }
      }
    }
    if constexpr (kTwo) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(&lds.rs[at][16 * s + 4 * g]);
#pragma unroll
        for (int m = 0; m < MQ; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[m][s][e] *= f[e];
      }
    }
    const uint32_t seen = static_cast<uint32_t>(__ballot(lds.slot[i & 7][lane & 31] >= 0));
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
      uint32_t vis = seen;
      if (tile >= spot.main_tiles) vis &= static_cast<uint32_t>(tree_bits[m] >> (kTile * (tile - spot.main_tiles)));
      vis >>= 4 * g;
      float y[8], high = kNegInf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = (vis >> (16 * (j >> 2) + (j & 3))) & 1 ? x[m][j >> 2][j & 3] * p.scale_log2 : kNegInf;
        high = fmaxf(high, y[j]);
      }
      high = rows_max(high);
      const int row = wave * MQ + m;
      const bool pass = high > (ref[m] == kNegInf ? kNegInf : ref[m] + kSlack);
      const bool any = __any(pass);
      if (any) {
        const float next = pass ? high : ref[m];
        const float fade = ref[m] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ref[m] - next);
        ref[m] = next;
        sum[m] *= fade;
        if (g == 0) lds.fade[half][row][col] = fade;
      }
      if (lane == 0) lds.fading[half][row] = any;
      const float base = ref[m] == kNegInf ? 0.0f : ref[m];
      bf16x8 prob, rest;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = __builtin_amdgcn_exp2f(y[j] - base);
        sum[m] += y[j];
        prob[j] = static_cast<__bf16>(y[j]);
        if constexpr (kTwo) rest[j] = static_cast<__bf16>(y[j] - static_cast<float>(prob[j]));
      }
      lds.prob[half][0][row][lane] = __builtin_bit_cast(u32v4, prob);
      if constexpr (kTwo) lds.prob[half][1][row][lane] = __builtin_bit_cast(u32v4, rest);
    }
  };

  f32x4 out[RT][NC];
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int c = 0; c < NC; ++c) out[m][c] = f32x4{};
  const uint8_t* codes_at = SHARED ? &lds.k[0][0] : &lds.v[0][0];
  // products of tile i with the wave's channels
  auto products = [&](int i) {
    const int at = i % 3, half = i & 1;
    bf16x8 prob[RT], rest[kTwo ? RT : 1];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      if (__builtin_amdgcn_readfirstlane(lds.fading[half][m])) {
        const float fade = lds.fade[half][m][col];
#pragma unroll
        for (int c = 0; c < NC; ++c) out[m][c] *= fade;
      }
      prob[m] = __builtin_bit_cast(bf16x8, lds.prob[half][0][m][lane]);
      if constexpr (kTwo) rest[m] = __builtin_bit_cast(bf16x8, lds.prob[half][1][m][lane]);
    }
    // lanes 2 j, 2 j + 1 of 16 stand at the row of the group's key j: 4 g + j, then 16 + 4 g + j - 4
    const int row = 4 * g + ((col >> 1) & 3) + 16 * (col >> 3);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      typedef int i32x2 __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2* Lds2;
      const int ch = wave * NC + c;
      const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (Lds2)(codes_at + at * (kTile * kPitch) + place(row, ch) + 8 * (col & 1)));
      const float* f = SHARED && !kTwo ? &lds.ks[at][ch >> 1][0] : &lds.vs[at][ch >> 1][0];
      const f32x4 f0 = *reinterpret_cast<const f32x4*>(f + 4 * g), f1 = *reinterpret_cast<const f32x4*>(f + 16 + 4 * g);
      bf16x8 v;
      v[0] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[0], f0[0], 0));
      v[1] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[0], f0[1], 1));
      v[2] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[0], f0[2], 2));
      v[3] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[0], f0[3], 3));
      v[4] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[1], f1[0], 0));
      v[5] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[1], f1[1], 1));
      v[6] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[1], f1[2], 2));
      v[7] = static_cast<__bf16>(__builtin_amdgcn_cvt_scalef32_f32_fp8(w[1], f1[3], 3));
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        out[m][c] = Mat<__bf16>::mma(v, prob[m], out[m][c]);
        if constexpr (kTwo) out[m][c] = Mat<__bf16>::mma(v, rest[m], out[m][c]);
      }
    }
  };

  // Tile i is brought from memory in step i - 3, laid out in step i - 2, scored
  // in step i - 1 and multiplied in step i; its slots are found in step i - 5
  // and written in step i - 4.  A step ends at its barrier.
  if (steps > 0) {
    if (tid < 128) lds.slot[tid >> 5][tid & 31] = find(tid >> 5);
    __syncthreads();
    bring(0);
    lay(0);
    bring(1);
    __syncthreads();
    scores(0);
    lay(1);
    bring(2);
    int32_t found = find(4);
    __syncthreads();
    for (int i = 0; i < steps; ++i) {
      lay(i + 2);
      if (tid < 32) lds.slot[(i + 4) & 7][tid] = found;
      bring(i + 3);
      found = find(i + 5);
      products(i);
      if (i + 1 < steps) scores(i + 1);
      __syncthreads();
    }
  }

#pragma unroll
  for (int m = 0; m < MQ; ++m) {
    sum[m] = rows_sum(sum[m]);
    if (g == 0) lds.stat[(wave * MQ + m) * 16 + col] = f32x2{ref[m], sum[m]};
  }
  __syncthreads();
  const int64_t block = blockIdx.x;
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    const int r = spot.row0 + 16 * m + col;
    if (r >= p.rows) continue;
    const f32x2 s = lds.stat[16 * m + col];
    if (p.splits > 1) {
      const int64_t at = block * (16 * RT) + 16 * m + col;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 16 * (wave * NC + c) + 4 * g;
        if (ch < a.Dv) store_any(p.part + at * a.Dv + ch, out[m][c]);
      }
      if (wave == 0 && g == 0) p.stat[at] = s;
    } else {
      int t, h;
      attend_row(p, spot, r, &t, &h);
      const int64_t at = (static_cast<int64_t>(spot.b) * a.T + t) * a.Hq + h;
      const float inv = attend_inverse(s[1]);
      typedef T V4 __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 16 * (wave * NC + c) + 4 * g;
        V4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(out[m][c][e] * inv);
        if (ch < a.Dv) store_any(static_cast<T*>(a.out) + at * a.Dv + ch, y);
      }
      if (wave == 0 && g == 0) a.lse[at] = attend_lse(s[0], s[1]);
    }
  }
}

template <class T, int RT, int NC, bool SHARED>
void launch(const AttendParams& p, hipStream_t s) {
  const uint32_t grid = static_cast<uint32_t>(static_cast<int64_t>(p.units) * p.row_groups * p.splits);
  hipLaunchKernelGGL((attend_wide_kernel<T, RT, NC, SHARED>), dim3(grid), dim3(kAttendThreads),
                     sizeof(WideLds<RT, NC, SHARED, Mat<T>::kRowScale>), s, p);
}

}  // namespace

void launch_attend_wide(const AttendParams& p, int row_tiles, bool shared, hipStream_t s) {
  const bool bf16 = p.a.dtype == ETS_BF16;
  if (row_tiles == 8) {
    shared ? launch<__bf16, 8, 8, true>(p, s) : launch<__bf16, 8, 8, false>(p, s);
  } else if (shared) {
    bf16 ? launch<__bf16, 4, 8, true>(p, s) : launch<_Float16, 4, 8, true>(p, s);
  } else {
    bf16 ? launch<__bf16, 4, 9, false>(p, s) : launch<_Float16, 4, 9, false>(p, s);
  }
}

}  // namespace ets
