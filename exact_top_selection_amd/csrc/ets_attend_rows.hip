// ets_attend_rows.hip -- attention of many query rows that share a list of
// keys over a block cache: pieces of prompts, wide trees, many heads on one
// head of the cache (gfx950).
#include "ets_attend_rows.h"

namespace ets {
namespace {

constexpr int kKeys = 64;  // of a step
// How far (log2) a score may pass its softmax's reference here, and what values are multiplied by for it.  As part of a
// block's scale 2^-18 takes the bits of values under 448 * 2^(18 - 127) < 2^-100 only, which 2^-24 would not.
constexpr float kRowsSlack = 18.0f;
constexpr uint32_t kRowsDown = 18;
constexpr float kToDown = 0x1p-6f;  // to what the other kernels' sums are multiplied by

// Bytes of a key's decoded channels in LDS (16 rows start in different banks),
// of half a value's, and of a value's (as in the narrow kernel).
constexpr int key_pitch(int n) { return 128 * n + 16; }
constexpr int rows_plane(int n) { return 64 * n + (n % 4 ? 0 : 64); }
constexpr int value_pitch(int n) { return 2 * rows_plane(n) + 16; }
constexpr int step_bytes(int n) { return kKeys * (key_pitch(n) + value_pitch(n)); }
constexpr int lds_bytes(int n, int waves) { return 2 * step_bytes(n) + 2 * 64 * waves * 8; }

// WAVES waves share a step of 64 keys and values, decoded once into LDS, and
// take 16 NT query rows each.  A step is brought three steps ahead into
// registers and decoded one step ahead into the other half of LDS, so one
// barrier a step is enough.
//
// Scores are K Q^T and results V^T P^T, as in the narrow kernel: a lane holds
// one query row's column, probabilities stay in registers between the
// products, and the softmax's reference follows the largest score only when
// one passes it by 2^18.  The 2^-18 that keeps sums of values finite is part of
// the values' scale.
//
// Slots and scales come through LDS too, found by a lane each: every thread
// finding those of its own piece cost 60 vector instructions a step.
//
// Measured, a call in a row of them: 342 us for pieces of 1000 tokens of two
// prompts of 8192 and 7329, 280 of 8192 and 4430, 32 heads on 8 of 128 channels,
// bf16 (690 TFLOP/s of the formula's, half as many again with the probabilities'
// second part; 750 on four full prompts).  65 us and 7 of join for 12 trees of 13
// tokens behind up to 10007 (92945 positions in all), 32 heads on 4 of 96, fp16.
// The bound is the issue of a SIMD: vector instructions take half of its cycles
// and matrix instructions two fifths, and little of one runs under the other.
// Two waves a SIMD leave no registers for a third.  The vector instructions count
// lane moves: no vector register spills, but 62 to 128 scalar ones do, into lanes
// (110 in the bf16 instance of 128 channels).  There the block that finds the
// slots of 4 steps holds 47 reads and 18 writes of lanes beside 248 other vector
// instructions, the one that brings and decodes a step 49 and 1 beside 93, and
// those of the products 2 between them.
//
// KB: 32-key parts of a step that a wave has in its registers at once.
template <class T, int N, int NT, int KB, int WAVES>
__global__ __launch_bounds__(64 * WAVES, rows_per_unit(N, WAVES)) void attend_rows_kernel(AttendBlocksParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  constexpr int kKeyPitch = key_pitch(N), kPlane = rows_plane(N), kPitch = value_pitch(N);
  constexpr int kThreads = 64 * WAVES;
  constexpr int kTurn = kThreads;           // keys whose slots and scales are found at a time, one a lane
  constexpr int kPieces = 4 * N;            // 16 channels each, of a key or a value
  constexpr int kItems = 2 * kPieces / WAVES;  // pieces of a step that a thread brings
  static_assert(kItems % 2 == 0, "as many of keys as of values");
  extern __shared__ __align__(16) char lds[];
  const ets_attend_args& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;
  const AttendSpot spot = attend_spot<true>(p);
  if (!spot.live) return;
  const int b = spot.b, hk = spot.hk;
  const int k0 = spot.first * kAttendTile, k1 = min(spot.last * kAttendTile, spot.n);
  const int steps = k1 > k0 ? (k1 - k0 + kKeys - 1) / kKeys : 0;

  // queries: lane (row col, g) holds channels 32 i + 8 g .. + 7
  V8 q[NT][2 * N];
  uint64_t tree_bits[NT];
  int upto[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    const int r = spot.row0 + (wave * NT + m) * 16 + col;
    int t, h;
    attend_row(p, spot, hk, r, &t, &h);
    const char* src = static_cast<const char*>(a.q) + 2 * (b * a.q_b + t * a.q_t + h * a.q_h);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
      q[m][i] = V8{};
      if (r < p.rows && 32 * i + 8 * g < a.D) q[m][i] = load_any<V8>(src + 64 * i + 16 * g);
    }
    attend_sight(p, spot, r < p.rows, t, &upto[m], &tree_bits[m]);
  }

  // Slots and scales of kTurn keys at a time, found by a lane each in three turns (page, then slot and scale bytes, then LDS)
  // and kept for the steps to read: slot, -1 for a key that is not there, and both scales' upper halves as floats.
  int32_t* slots = reinterpret_cast<int32_t*>(lds + 2 * step_bytes(N));  // [2][kTurn]
  uint32_t* scales = reinterpret_cast<uint32_t*>(slots + 2 * kTurn);     // [2][kTurn]
  const uint64_t nothing = reinterpret_cast<uint64_t>(&kNothing[0]);
  int32_t asked = 0, found = -1;
  uint32_t key_byte = 0, value_byte = 0;
  auto ask = [&](int turn) {  // past the end: the last key's page
    const int at = min(k0 + turn * kTurn + static_cast<int>(threadIdx.x), k1 - 1);
    asked = a.page_table[b * a.pt_b + div_by(static_cast<uint32_t>(at), p.by_page)];
  };
  auto find = [&](int turn) {
    const int at = k0 + turn * kTurn + static_cast<int>(threadIdx.x);
    const uint32_t page = div_by(static_cast<uint32_t>(min(at, k1 - 1)), p.by_page);
    const int64_t slot = static_cast<int64_t>(asked) * a.page_size + (at - static_cast<int>(page * p.by_page.d));
    const bool there = at < k1 && asked >= 0 && slot < a.S;
    const uint64_t block = div_by(static_cast<uint32_t>(slot) & 0x7fffffffu, p.by_block);
    const uint64_t k = reinterpret_cast<uint64_t>(a.k_scales + hk * a.ks_h) + block * static_cast<uint32_t>(a.ks_s);
    const uint64_t v = reinterpret_cast<uint64_t>(a.v_scales + hk * a.vs_h) + block * static_cast<uint32_t>(a.vs_s);
    found = there ? static_cast<int32_t>(slot) : -1;
    key_byte = load_global<uint8_t>(there ? k : nothing);
    value_byte = load_global<uint8_t>(there ? v : nothing);
  };
  auto keep = [&](int turn) {
    const int to = (turn & 1) * kTurn + static_cast<int>(threadIdx.x);
    slots[to] = found;
    scales[to] = key_byte << 23 | (value_byte > kRowsDown ? (value_byte - kRowsDown) << 7 : 0);
  };

  // A thread's part of a step: pieces of 16 codes, keys' before values'; a wave's pieces are of one kind.
  uint64_t row[kItems];
  uint32_t stride[kItems];
  bool is_value[kItems];
  int key[kItems], piece[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    is_value[j] = j >= kItems / 2;
    const int i = static_cast<int>(threadIdx.x) + j * kThreads - (is_value[j] ? kKeys * kPieces : 0);
    key[j] = i / kPieces, piece[j] = i % kPieces;
    row[j] = reinterpret_cast<uint64_t>(is_value[j] ? a.v_codes + hk * a.v_h : a.k_codes + hk * a.k_h) + 16 * piece[j];
    stride[j] = static_cast<uint32_t>(is_value[j] ? a.v_s : a.k_s);
    if (16 * piece[j] >= (is_value[j] ? a.Dv : a.D)) row[j] = nothing, stride[j] = 0;  // channels that are not there
  }
  struct Codes {
    u32v4 code[kItems];
    uint32_t scale[kItems];
  };
  auto fetch = [&](Codes& c, int step) {
    const int from = (step * kKeys) & (2 * kTurn - 1);
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int32_t slot = slots[from + key[j]];
      c.scale[j] = scales[from + key[j]];
      const uint64_t at = row[j] + static_cast<uint64_t>(static_cast<uint32_t>(slot)) * stride[j];
      c.code[j] = load_global<u32v4>(slot >= 0 ? at : nothing);
    }
  };
  auto decode = [&](const Codes& from, int step) {
    char* to = lds + (step & 1) * step_bytes(N);
    char* values = to + kKeys * kKeyPitch;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const u32v4 c = from.code[j];
      if (is_value[j]) {
        const float f = __uint_as_float(from.scale[j] << 16);
        char* dst = values + key[j] * kPitch + 16 * piece[j];
        *reinterpret_cast<bf16x8*>(dst) = codes_bf16(c[0], c[1], f);
        *reinterpret_cast<bf16x8*>(dst + kPlane) = codes_bf16(c[2], c[3], f);
      } else {
        const float f = M::kRowScale ? 1.0f : __uint_as_float(from.scale[j] & 0xffff0000u);
        V8* dst = reinterpret_cast<V8*>(to + key[j] * kKeyPitch + 32 * piece[j]);
        dst[0] = M::keys(c[0], c[1], f);
        dst[1] = M::keys(c[2], c[3], f);
      }
    }
  };

  f32x4 out[NT][4 * N];
  float top[NT], sum[NT];
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    top[m] = kNegInf, sum[m] = 0.0f;
#pragma unroll
    for (int c = 0; c < 4 * N; ++c) out[m][c] = f32x4{};
  }

  // 32 KB keys from position `at` on: keys and values in LDS, which of them are there, their scales
  auto work = [&](const char* keys, char* values, int at, uint64_t here, const uint32_t* key_scale) {
    constexpr uint64_t kAll = KB == 2 ? ~0ull : 0xffffffffull;
    const bool ragged = at + 32 * KB > spot.edge;
    f32x4 score[NT][2 * KB];
#pragma unroll
    for (int s = 0; s < 2 * KB; ++s)
#pragma unroll
      for (int m = 0; m < NT; ++m) score[m][s] = f32x4{};
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
#pragma unroll
      for (int s = 0; s < 2 * KB; ++s) {
        const V8 k = *reinterpret_cast<const V8*>(keys + (16 * s + col) * kKeyPitch + 64 * i + 16 * g);
#pragma unroll
        for (int m = 0; m < NT; ++m) score[m][s] = M::mma(k, q[m][i], score[m][s]);
      }
    }
    if constexpr (M::kRowScale) {
#pragma unroll
      for (int s = 0; s < 2 * KB; ++s) {
        const u32v4 f = *reinterpret_cast<const u32v4*>(key_scale + 16 * s + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int m = 0; m < NT; ++m) score[m][s][e] *= __uint_as_float(f[e] & 0xffff0000u);
      }
    }
    bf16x8 prob[NT][KB], rest[NT][KB];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      // x: what goes into the exponential.  First as if all keys were seen and the reference stayed.
      float x[8 * KB], high = kNegInf;
#pragma unroll
      for (int j = 0; j < 8 * KB; ++j) {
        x[j] = __builtin_fmaf(score[m][j >> 2][j & 3], p.scale_log2, -top[m]);
        high = __builtin_elementwise_maximum(high, x[j]);  // no number passes no test
      }
      if (here != kAll || ragged || !__all(high <= kRowsSlack)) {
        high = kNegInf;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          uint32_t vis = static_cast<uint32_t>(here >> (32 * k));
          if (ragged) vis &= attend_seen_by(spot, upto[m], tree_bits[m], at + 32 * k);
          vis >>= 4 * g;  // bits 0..3: keys 4 g + e; bits 16..19: keys 16 + 4 g + e
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[8 * k + j] = (vis >> (16 * (j >> 2) + (j & 3))) & 1 ? score[m][2 * k + (j >> 2)][j & 3] * p.scale_log2 : kNegInf;
            high = fmaxf(high, x[8 * k + j]);
          }
        }
        high = rows_max(high);
        if (__any(high > top[m] + kRowsSlack || top[m] == kNegInf)) {
          const float next = high > top[m] + kRowsSlack || top[m] == kNegInf ? high : top[m];
          const float fade = __builtin_amdgcn_exp2f(top[m] - (next == kNegInf ? 0.0f : next));
          sum[m] *= fade;
#pragma unroll
          for (int c = 0; c < 4 * N; ++c) out[m][c] *= fade;
          top[m] = next;
        }
        const float base = top[m] == kNegInf ? 0.0f : top[m];
#pragma unroll
        for (int j = 0; j < 8 * KB; ++j) x[j] -= base;
      }
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        u32v4 first, second;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y = __builtin_amdgcn_exp2f(x[8 * k + 2 * j]), z = __builtin_amdgcn_exp2f(x[8 * k + 2 * j + 1]);
          sum[m] += y;
          sum[m] += z;
          first[j] = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(y), static_cast<__bf16>(z)});
          asm("" : "+v"(first[j]));  // else the compiler converts y once more for its half
          second[j] = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(y - __uint_as_float(first[j] << 16)),
                                                          static_cast<__bf16>(z - __uint_as_float(first[j] & 0xffff0000u))});
        }
        prob[m][k] = __builtin_bit_cast(bf16x8, first);
        rest[m][k] = __builtin_bit_cast(bf16x8, second);
      }
    }
    const char* src = values + (4 * g + (col >> 2)) * kPitch + kPlane * ((col >> 1) & 1) + 8 * (col & 1);
    auto value = [&](int k, int c) {
      typedef __attribute__((address_space(3))) s16x4* Lds4;
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(src + 32 * k * kPitch + 16 * c));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(src + (32 * k + 16) * kPitch + 16 * c));
      return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    };
    if (ragged) {
      // values that are no numbers: every wave sees the same ones, so all of them come to these barriers or none
      uint32_t any = 0;
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int c = 0; c < 4 * N; ++c) {
          const u16x8 bits = __builtin_bit_cast(u16x8, value(k, c));
#pragma unroll
          for (int e = 0; e < 8; ++e) any |= no_number(bits[e]);
        }
      if (__any(any != 0)) {
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            const uint32_t vis = static_cast<uint32_t>(here >> (32 * k)) & attend_seen_by(spot, upto[m], tree_bits[m], at + 32 * k);
            const bf16x8 sees = seen_places(vis >> (4 * g));
#pragma unroll
            for (int c = 0; c < 4 * N; ++c) out[m][c] = spoilt(out[m][c], odd_places(value(k, c)), sees);
          }
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * KB * 8 * N; i += kThreads) {
          const int r = i / (8 * N), eight = i % (8 * N);
          clear_odd(values + r * kPitch + (eight & 1) * kPlane + 16 * (eight >> 1));
        }
        __syncthreads();
      }
    }
    // two channels' products side by side: each waits for the one before it of its own sum
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int c = 0; c < 4 * N; c += 2) {
        const bf16x8 v = value(k, c), w = value(k, c + 1);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          out[m][c] = Mat<__bf16>::mma(v, prob[m][k], out[m][c]);
          out[m][c + 1] = Mat<__bf16>::mma(w, prob[m][k], out[m][c + 1]);
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          out[m][c] = Mat<__bf16>::mma(v, rest[m][k], out[m][c]);
          out[m][c + 1] = Mat<__bf16>::mma(w, rest[m][k], out[m][c + 1]);
        }
      }
  };

  if (steps > 0) {
    ask(0);
    find(0);
    ask(1);
    keep(0);
    find(1);
    ask(2);
    __syncthreads();
    Codes even, odd;
    fetch(even, 0);
    fetch(odd, 1);
    decode(even, 0);
    fetch(even, 2);
    // one step: `codes` hold the next one's, and then those of the step two behind it
    auto advance = [&](Codes& codes, int step) {
      __syncthreads();  // this step is decoded, and nobody reads the other half any more
      decode(codes, step + 1);  // past the end: zeros
      fetch(codes, step + 3);   // its slots were kept at least one barrier ago
      if (step % (kTurn / kKeys) == 0) {  // the last turn's half of the slots is read no more
        const int turn = step / (kTurn / kKeys);
        keep(turn + 1);
        find(turn + 2);
        ask(turn + 3);
      }
      char* from = lds + (step & 1) * step_bytes(N);
      const int in = (step * kKeys) & (2 * kTurn - 1);
      const uint64_t here = __ballot(slots[in + lane] >= 0);
#pragma unroll 1
      for (int part = 0; part < 2 / KB; ++part)
        work(from + 32 * part * kKeyPitch, from + kKeys * kKeyPitch + 32 * part * kPitch, k0 + step * kKeys + 32 * part,
             KB == 2 ? here : here >> (32 * part) & 0xffffffffull, scales + in + 32 * part);
    };
    for (int step = 0; step < steps; step += 2) {
      advance(odd, step);
      if (step + 1 < steps) advance(even, step + 1);
    }
  }

#pragma unroll
  for (int m = 0; m < NT; ++m) {
    if (attend_blind(upto[m], tree_bits[m])) {
      top[m] = kNegInf, sum[m] = 0.0f;
#pragma unroll
      for (int c = 0; c < 4 * N; ++c) out[m][c] = f32x4{};
    }
    sum[m] = rows_sum(sum[m]);
    const int in_group = (wave * NT + m) * 16 + col, r = spot.row0 + in_group;
    if (r >= p.rows) continue;
    if (p.splits > 1) {
      const int64_t place = attend_place(p, spot, hk) * p.group_rows + in_group;
#pragma unroll
      for (int c = 0; c < 4 * N; ++c) {
        if (16 * c + 4 * g < a.Dv) store_any(p.part + place * a.Dv + 16 * c + 4 * g, out[m][c] * kToDown);
      }
      if (g == 0) p.stat[place] = f32x2{top[m], sum[m]};
    } else {
      int t, h;
      attend_row(p, spot, hk, r, &t, &h);
      const int64_t place = (static_cast<int64_t>(b) * a.T + t) * a.Hq + h;
      const float inv = attend_inverse(sum[m]) * kToDown;
      typedef T V4 __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int c = 0; c < 4 * N; ++c) {
        if (16 * c + 4 * g >= a.Dv) continue;
        V4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(out[m][c][e] * inv);
        store_any(static_cast<T*>(a.out) + place * a.Dv + 16 * c + 4 * g, y);
      }
      if (g == 0) a.lse[place] = attend_lse(top[m], sum[m]);
    }
  }
}

template <class T, int N, int NT, int KB, int WAVES>
void launch(const AttendBlocksParams& p, hipStream_t s) {
  const uint32_t grid = static_cast<uint32_t>(attend_rows_groups(p));
  hipLaunchKernelGGL((attend_rows_kernel<T, N, NT, KB, WAVES>), dim3(grid), dim3(64 * WAVES), lds_bytes(N, WAVES), s, p);
}

template <class T>
void launch_type(const AttendBlocksParams& p, const RowsShape& r, hipStream_t s) {
  switch (r.width) {
    case 1: return r.tiles == 1 ? launch<T, 1, 1, 2, 4>(p, s) : launch<T, 1, 2, 1, 4>(p, s);
    case 2:
      if (r.waves == 8) return launch<T, 2, 2, 1, 8>(p, s);
      return r.tiles == 1 ? launch<T, 2, 1, 2, 4>(p, s) : launch<T, 2, 2, 1, 4>(p, s);
    case 3: return launch<T, 3, 2, 1, 4>(p, s);
    default: return launch<T, 4, 2, 1, 4>(p, s);
  }
}

}  // namespace

void launch_attend_rows(const AttendBlocksParams& p, const RowsShape& r, hipStream_t s) {
  if (p.a.dtype == ETS_BF16) {
    launch_type<__bf16>(p, r, s);
  } else {
    launch_type<_Float16>(p, r, s);
  }
}

}  // namespace ets
