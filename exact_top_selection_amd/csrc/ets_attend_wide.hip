// ets_attend_wide.hip -- attention over an 8-bit cache for heads of 257 to 576
// channels, one latent head shared by many query heads above all (gfx950).
#include <type_traits>

#include "ets_attend.h"

namespace ets {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = kAttendTile;
constexpr int kPairs = 9;            // 64-channel steps of a key
constexpr int kPieces = 36;          // 16-code pieces of a key
constexpr int kPlane = 16 * kPieces; // bytes of one half of each decoded piece of a row
// Bytes of a decoded row in LDS: first the lower halves of its pieces, then
// the upper ones, so that lanes write next to each other; rows lie 36 banks
// apart, so that the 16 rows of an operand load fill all 64.
constexpr int kPitch = 2 * kPlane + 16;
constexpr int kDepth = 2;            // tiles on their way from memory

// Pieces of a tile on their way through a lane, and their scale bytes.
template <int N>
struct Pieces {
  static constexpr int n = N;
  u32v4 w[N];
  uint32_t byte[N];
};

// What lanes address by themselves comes first: an LDS instruction's own offset
// reaches 64 KiB, and each address behind that took a register through the loop.
template <int RT, bool SHARED>
struct WideLds {
  u32v2 prob[2][2][2][RT][64];  // [parity][part][team]
  f32x2 stat[2][RT * 16];
  float ref[2][2][RT * 16];     // [parity][team]
  int32_t slot[4][kTile];       // -1: not there
  uint32_t seen[8];             // which keys of a tile are there
  uint32_t sees[2][2][RT * 16]; // [parity][team] which drafted tokens a row sees
  alignas(16) uint8_t k[SHARED ? 3 : 2][kTile * kPitch];
  uint8_t v[SHARED ? 1 : 2][SHARED ? 16 : kTile * kPitch];
};

// A workgroup takes 16 RT query rows through its share of the keys, 32 a step.
// Codes come through registers, two steps ahead (rows lie anywhere in the
// cache, so a row takes 1 to 2 us to arrive), and are decoded to bf16, which
// holds them exactly, on their way into LDS: once for all query rows, and once
// for keys and values where the values are the keys' first channels (SHARED).
//
// Waves 0 to 3 form scores as K Q^T: half of the query rows, in registers, by
// half of the step's keys (a "team").  Their probabilities go through LDS to
// waves 4 to 7, which hold the sums out^T = V^T P^T, a quarter of the channels
// each, with V^T out of transposed loads (ds_read_b64_tr_b16).  Each SIMD has
// one wave of either kind, scores run one step ahead of the sums, and a step
// has one barrier; within it one wave lays out rows while the other multiplies.
//
// The softmax is taken relative to a whole-numbered reference that each team
// raises only when a score passes it by more than 2^24, and that follows the
// other team's of the step before.  While no score does and all keys are seen,
// a step needs no largest score and no rescaling; where a reference has
// changed, or the two differ, sums and probabilities are brought together by
// powers of two, which is exact.  (With 2^8 every second step of 64 rows had
// such a change; both together took 74 us to 62.)
//
// Probabilities are the sum of two bf16 numbers (16 bits), and fp16 queries are
// so too, exactly (kTwo).  One part of 8 bits took 62 us on the case below in
// the place of 70, but its results were off by up to 3.4 times their own
// rounding to bf16 with few keys, and 1.1 times when divided by the sum of the
// rounded probabilities.
//
// Measured: 70 us for 64 sequences, 128 heads on one latent head of 576
// channels, 2048 slots each (36.5 GFLOP: 520 TFLOP/s), and 11 us for the join
// of its two shares.  Of the 70, 8 go by until the first product (queries and
// first rows come at once, 28 MB) and 4 after the last (33 MB of sums).  A step
// of 32 keys is 100 matrix instructions a SIMD (1600 cycles), and those of one
// wave leave another wave of their SIMD every second vector slot.
template <class T, int RT, int NC, bool SHARED>
__global__ __launch_bounds__(kThreads, 2) void attend_wide_kernel(AttendParams p) {
  constexpr bool kTwo = Mat<T>::kRowScale;  // fp16: queries of two parts
  constexpr int MQ = RT / 2;  // 16-row tiles of a score wave
  typedef WideLds<RT, SHARED> Lds;
  typedef T T8 __attribute__((ext_vector_type(8)));
  typedef __bf16 B4 __attribute__((ext_vector_type(4)));
  extern __shared__ __align__(16) char lds_raw[];
  Lds& lds = *reinterpret_cast<Lds*>(lds_raw);
  const ets_attend_args& a = p.a;
  const AttendSpot spot = attend_spot(p);
  if (!spot.live) return;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = max(spot.last - spot.first, 0);
  const bool forked = spot.paged && p.tree_tiles > 0;  // rows of the workgroup see different drafted tokens
  const int steps = (tiles + 1) & ~1;  // pairs: the staging registers of either parity keep their places

  // The 1152 pieces of a tile: waves 4 to 7 bring three a lane, waves 0 and 1
  // two, waves 2 and 3, which also find the rows, one.  (64 rows: 71 us; with
  // four a lane of waves 4 to 7 and one of waves 0 and 1 72, with two, three and
  // two 75.)
  const bool sums = wave >= 4;
  const int piece0 = sums ? tid - 256 : wave < 2 ? 768 + tid : 1024 + tid - 128;
  const int apart = sums ? 256 : 128;
  // addresses as numbers: a row that is not there is read from kNothing, without a branch
  const uint64_t nothing = reinterpret_cast<uint64_t>(&kNothing[0]);
  auto bring = [&](auto& set, int i, uint64_t codes, uint32_t row, uint64_t scales, uint32_t scale_row, int pieces) {
    const int32_t* slots = lds.slot[i & 3];
    constexpr int N = std::remove_reference_t<decltype(set)>::n;
    int32_t slot[N];
#pragma unroll
    for (int j = 0; j < N; ++j) slot[j] = slots[(piece0 + apart * j) / kPieces];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int at = (piece0 + apart * j) % kPieces;
      const bool there = slot[j] >= 0 && at < pieces;
      const uint64_t w = codes + static_cast<uint64_t>(static_cast<uint32_t>(slot[j])) * row + 16 * at;
      const uint64_t b = scales + static_cast<uint64_t>(static_cast<uint32_t>(slot[j])) * scale_row + (at >> 1);
      set.w[j] = load_global<u32v4>(there ? w : nothing);
      set.byte[j] = load_global<uint8_t>(there ? b : nothing);
    }
  };
  auto lay = [&](const auto& set, uint8_t* tile) {
#pragma unroll
    for (int j = 0; j < set.n; ++j) {
      const int c = piece0 + apart * j;
      const float f = __uint_as_float(set.byte[j] << 23);
      uint8_t* dst = tile + c / kPieces * kPitch + 16 * (c % kPieces);
      *reinterpret_cast<bf16x8*>(dst) = codes_bf16(set.w[j][0], set.w[j][1], f);
      *reinterpret_cast<bf16x8*>(dst + kPlane) = codes_bf16(set.w[j][2], set.w[j][3], f);
    }
  };
  const uint64_t kc = reinterpret_cast<uint64_t>(a.k_codes + spot.hk * a.k_h);
  const uint64_t ks = reinterpret_cast<uint64_t>(a.k_scales + spot.hk * a.ks_h);
  const uint64_t vc = reinterpret_cast<uint64_t>(a.v_codes + spot.hk * a.v_h);
  const uint64_t vs = reinterpret_cast<uint64_t>(a.v_scales + spot.hk * a.vs_h);
  const uint32_t k_row = static_cast<uint32_t>(a.k_s), ks_row = static_cast<uint32_t>(a.ks_s);
  const uint32_t v_row = static_cast<uint32_t>(a.v_s), vs_row = static_cast<uint32_t>(a.vs_s);
  auto bring_k = [&](auto& set, int i) { bring(set, i, kc, k_row, ks, ks_row, a.D / 16); };
  auto bring_v = [&](auto& set, int i) { bring(set, i, vc, v_row, vs, vs_row, a.Dv / 16); };
  // the slots of tile i, by 32 lanes: first what they depend on, later themselves
  auto ask = [&](int i) { return attend_ask(p, spot, spot.first + i, tid & 31); };
  auto keep = [&](int i, int32_t asked) {
    const int32_t slot = attend_slot(p, spot, spot.first + i, tid & 31, asked);
    const bool there = slot >= 0 && i < tiles;
    lds.slot[i & 3][tid & 31] = there ? slot : -1;
    const uint64_t seen = __ballot(there);
    if ((tid & 31) == 0) lds.seen[i & 7] = static_cast<uint32_t>(seen >> (tid & 32));
  };

  auto begin = [&](auto& kset, auto& vset) {  // before the first step: tiles 0 and 1 in LDS (values: 0)
    bring_k(kset[0], 0);
    bring_k(kset[1], 1);
    if constexpr (!SHARED) {
      bring_v(vset[0], 0);
      bring_v(vset[1], 1);
    }
    lay(kset[0], lds.k[0]);
    bring_k(kset[0], 2);
    lay(kset[1], lds.k[1]);
    bring_k(kset[1], 3);
    if constexpr (!SHARED) {
      lay(vset[0], lds.v[0]);
      bring_v(vset[0], 2);
    }
  };
  // step i: tile i + 2 into LDS (values: i + 1), tile i + 4 (i + 3) asked for; `odd` is i % 2, `to` the place of tile i + 2
  auto stage = [&](auto& kset, auto& vset, auto odd, int i, int to) {
    constexpr int O = decltype(odd)::value;
    lay(kset[O], lds.k[to]);
    bring_k(kset[O], i + 4);
    if constexpr (!SHARED) {
      lay(vset[O ^ 1], lds.v[O ^ 1]);
      bring_v(vset[O ^ 1], i + 3);
    }
  };
  // Runs step(odd, i, places of tiles i, i + 1, i + 2).  Nothing in it depends
  // on i by a branch: a load that is under way where branches meet is waited for.
  auto run = [&](auto step) {
    int at = 0, next = 1;
    for (int i = 0; i < steps; i += 2) {
      const int after = SHARED ? 3 - at - next : at;
      step(std::integral_constant<int, 0>{}, i, at, next, after);
      __syncthreads();
      step(std::integral_constant<int, 1>{}, i + 1, next, after, SHARED ? at : next);
      __syncthreads();
      const int a0 = after, a1 = SHARED ? at : next;
      at = a0, next = a1;
    }
  };

  if (wave < 4) {
    // ---- scores
    const int hg = wave & 1, team = wave >> 1;
    bf16x8 q[MQ][kPairs][2], q_rest[kTwo ? MQ : 1][kPairs][2];
    uint64_t tree_bits[MQ];
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
      const int r = spot.row0 + 16 * (MQ * hg + m) + col;
      int t, h;
      attend_row(p, spot, spot.hk, r, &t, &h);
      const char* src = static_cast<const char*>(a.q) + 2 * (spot.b * a.q_b + t * a.q_t + h * a.q_h);
      tree_bits[m] = 0;
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool there = r < p.rows && 64 * i + 16 * g < a.D;
          const T8 x = load_any<T8>(there ? src + 128 * i + 32 * g + 16 * j : reinterpret_cast<const char*>(&kNothing));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            q[m][i][j][e] = static_cast<__bf16>(static_cast<float>(x[e]));
            if constexpr (kTwo)
              q_rest[m][i][j][e] = static_cast<__bf16>(static_cast<float>(x[e]) - static_cast<float>(q[m][i][j][e]));
          }
        }
      if (r < p.rows && a.tree_slots) tree_bits[m] = static_cast<uint64_t>(a.tree_mask[spot.b * a.mask_b + t]);
      lds.ref[1][team][(MQ * hg + m) * 16 + col] = kNegInf;
    }
    __syncthreads();
    float ref[MQ], sum[MQ];
#pragma unroll
    for (int m = 0; m < MQ; ++m) ref[m] = kNegInf, sum[m] = 0.0f;

    auto scores = [&](int i, const uint8_t* tile) {
      float other[MQ];  // the other team's reference of the step before
#pragma unroll
      for (int m = 0; m < MQ; ++m) other[m] = lds.ref[(i & 1) ^ 1][team ^ 1][(MQ * hg + m) * 16 + col];
      f32x4 x[MQ], x1[MQ];  // two sums each: half as long a chain of products
#pragma unroll
      for (int m = 0; m < MQ; ++m) x[m] = f32x4{}, x1[m] = f32x4{};
      const uint8_t* row = tile + (16 * team + col) * kPitch + 16 * g;
      constexpr int kAhead = 6;  // operands asked for ahead of their products
      bf16x8 k[kAhead];
      auto operand = [&](int n) { return *reinterpret_cast<const bf16x8*>(row + (n & 1) * kPlane + 64 * (n >> 1)); };
#pragma unroll
      for (int n = 0; n < kAhead; ++n) k[n] = operand(n);
#pragma unroll
      for (int n = 0; n < 2 * kPairs; ++n) {
#pragma unroll
        for (int m = 0; m < MQ; ++m) {
          f32x4& sum = n & 1 ? x1[m] : x[m];
          sum = Mat<__bf16>::mma(k[n % kAhead], q[m][n >> 1][n & 1], sum);
          if constexpr (kTwo) sum = Mat<__bf16>::mma(k[n % kAhead], q_rest[m][n >> 1][n & 1], sum);
        }
        if (n + kAhead < 2 * kPairs) k[n % kAhead] = operand(n + kAhead);
      }
      // y: what goes into the exponential.  First as if all keys were seen and the reference stayed.
      const int at = spot.first + i, half = i & 1;
      const uint32_t seen = (__builtin_amdgcn_readfirstlane(lds.seen[i & 7]) >> (16 * team)) & 0xffffu;
      f32x4 y[MQ];
      bool stays = true;
#pragma unroll
      for (int m = 0; m < MQ; ++m) {
        x[m] += x1[m];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[m][e] = __builtin_fmaf(x[m][e], p.scale_log2, -ref[m]);
        const float high = fmaxf(fmaxf(y[m][0], y[m][1]), fmaxf(y[m][2], y[m][3]));
        stays = stays && high <= kSlack && other[m] <= ref[m];
      }
      if (seen != 0xffffu || at >= spot.main_tiles || !__all(stays)) {
#pragma unroll
        for (int m = 0; m < MQ; ++m) {
          uint32_t vis = seen;
          if (at >= spot.main_tiles) vis &= static_cast<uint32_t>(tree_bits[m] >> (kTile * (at - spot.main_tiles) + 16 * team & 63));
          if (!SHARED && forked && g == 0) lds.sees[half][team][(MQ * hg + m) * 16 + col] = vis;
          vis >>= 4 * g;
          float high = kNegInf;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[m][e] = (vis >> e) & 1 ? x[m][e] * p.scale_log2 : kNegInf;
            high = fmaxf(high, x[m][e]);
          }
          high = rows_max(high);
          float next = fmaxf(ref[m], other[m]);
          if (high > next + kSlack || next == kNegInf) next = ceilf(high);
          const float fade = ref[m] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ref[m] - next);
          sum[m] *= fade;
          ref[m] = next;
          y[m] = x[m] - (next == kNegInf ? 0.0f : next);
        }
      }
#pragma unroll
      for (int m = 0; m < MQ; ++m) {
        const int rt = MQ * hg + m;
        if (g == 0) lds.ref[half][team][rt * 16 + col] = ref[m];
        B4 prob, rest;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z = __builtin_amdgcn_exp2f(y[m][e]);
          sum[m] += z;
          z *= kDown;
          prob[e] = static_cast<__bf16>(z);
          rest[e] = static_cast<__bf16>(z - static_cast<float>(prob[e]));
        }
        lds.prob[half][0][team][rt][lane] = __builtin_bit_cast(u32v2, prob);
        lds.prob[half][1][team][rt][lane] = __builtin_bit_cast(u32v2, rest);
      }
    };

    if (wave < 2) {
      Pieces<2> kset[kDepth], vset[SHARED ? 1 : kDepth];
      begin(kset, vset);
      __syncthreads();
      scores(0, lds.k[0]);
      __syncthreads();
      run([&](auto odd, int i, int, int next, int after) {
        scores(i + 1, lds.k[next]);
        stage(kset, vset, odd, i, after);
      });
    } else {  // these two find the rows (both the same ones)
      Pieces<1> kset[kDepth], vset[SHARED ? 1 : kDepth];
      int32_t asked = ask(4);
      begin(kset, vset);
      __syncthreads();
      keep(4, asked);
      asked = ask(5);
      scores(0, lds.k[0]);
      __syncthreads();
      run([&](auto odd, int i, int, int next, int after) {
        keep(i + 5, asked);
        asked = ask(i + 6);
        scores(i + 1, lds.k[next]);
        stage(kset, vset, odd, i, after);
      });
    }
#pragma unroll
    for (int m = 0; m < MQ; ++m) {
      sum[m] = rows_sum(sum[m]);
      if (g == 0) lds.stat[team][(MQ * hg + m) * 16 + col] = f32x2{ref[m], sum[m]};
    }
    __syncthreads();
    return;
  }

  // ---- sums
  const int quarter = wave - 4;
  f32x4 out[RT][NC];
  float base[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    base[m] = kNegInf;
#pragma unroll
    for (int c = 0; c < NC; ++c) out[m][c] = f32x4{};
  }
  // Two row tiles at a time: the probabilities of four spill (74 us), and the loads of one pair are not kept for the
  // next by the compiler, for which rows is a new value.
  auto products = [&](int i, uint8_t* tile) {
    typedef __attribute__((address_space(3))) s16x4* Lds4;
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const int half = i & 1;
    // 16 channels by 4 keys a load: lane (key col / 4, four channels col % 4) of the upper or lower halves
    uint32_t rows = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (Lds4)(tile + (4 * g + (col >> 2)) * kPitch + kPlane * ((col >> 1) & 1) + 8 * (col & 1) + 16 * (quarter * NC))));
    auto join = [](u32v2 lo, u32v2 hi) { return __builtin_bit_cast(bf16x8, u32v4{lo[0], lo[1], hi[0], hi[1]}); };
    auto value = [&](int c) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(uintptr_t)(rows + 16 * c));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(uintptr_t)(rows + 16 * kPitch + 16 * c));
      return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    };
    // The wave's channels of a tile are its own.  Where they are the keys' too, the row's score has told (it is no number either).
    if (forked && spot.first + i >= spot.main_tiles) {
      if constexpr (!SHARED) {
        bf16x8 sees[RT];
#pragma unroll
        for (int m = 0; m < RT; ++m)
          sees[m] = seen_places((lds.sees[half][0][16 * m + col] | lds.sees[half][1][16 * m + col] << 16) >> (4 * g));
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const bf16x8 odd = odd_places(value(c));
#pragma unroll
          for (int m = 0; m < RT; ++m) out[m][c] = spoilt(out[m][c], odd, sees[m]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      for (int n = lane; n < kTile * 2 * NC; n += 64) {
        const int row = n / (2 * NC), piece = n % (2 * NC);
        clear_odd(tile + row * kPitch + (piece & 1) * kPlane + 16 * (quarter * NC + (piece >> 1)));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int m0 = 0; m0 < RT; m0 += 2) {
      bf16x8 prob[2][2];
      bool moved = false;
      float r0[2], r1[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        r0[m] = lds.ref[half][0][16 * (m0 + m) + col];
        r1[m] = lds.ref[half][1][16 * (m0 + m) + col];
        moved = moved || r0[m] != base[m0 + m] || r1[m] != base[m0 + m];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          prob[k][m] = join(lds.prob[half][k][0][m0 + m][lane], lds.prob[half][k][1][m0 + m][lane]);
      }
      if (__any(moved)) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float next = fmaxf(base[m0 + m], fmaxf(r0[m], r1[m])), zero = next == kNegInf ? 0.0f : next;
          const float fade = __builtin_amdgcn_exp2f(base[m0 + m] - zero);
          const float f0 = __builtin_amdgcn_exp2f(r0[m] - zero), f1 = __builtin_amdgcn_exp2f(r1[m] - zero);
          base[m0 + m] = next;
#pragma unroll
          for (int c = 0; c < NC; ++c) out[m0 + m][c] *= fade;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              prob[k][m][e] = static_cast<__bf16>(static_cast<float>(prob[k][m][e]) * (e < 4 ? f0 : f1));
        }
      }
      asm volatile("" : "+v"(rows));
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const bf16x8 v = value(c);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m) out[m0 + m][c] = Mat<__bf16>::mma(v, prob[k][m], out[m0 + m][c]);
      }
    }
  };

  if (tid - 256 < 4 * kTile) keep((tid - 256) >> 5, ask((tid - 256) >> 5));
  __syncthreads();
  Pieces<3> kset[kDepth], vset[SHARED ? 1 : kDepth];
  begin(kset, vset);
  __syncthreads();
  __syncthreads();
  run([&](auto odd, int i, int at, int, int after) {
    stage(kset, vset, odd, i, after);
    products(i, SHARED ? lds.k[at] : lds.v[decltype(odd)::value]);
  });
  __syncthreads();

  const int64_t block = attend_place(p, spot, spot.hk);
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    const int r = spot.row0 + 16 * m + col;
    if (r >= p.rows) continue;
    const f32x2 s0 = lds.stat[0][16 * m + col], s1 = lds.stat[1][16 * m + col];
    const float zero = base[m] == kNegInf ? 0.0f : base[m];
    const float f0 = __builtin_amdgcn_exp2f(s0[0] - zero), f1 = __builtin_amdgcn_exp2f(s1[0] - zero);
    const f32x2 s = {base[m], s0[1] * f0 + s1[1] * f1};
    const bool first = quarter == 0 && g == 0;
    if (p.splits > 1) {
      const int64_t at = block * (16 * RT) + 16 * m + col;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 16 * (quarter * NC + c) + 4 * g;
        if (ch < a.Dv) store_any(p.part + at * a.Dv + ch, out[m][c]);
      }
      if (first) p.stat[at] = s;
    } else {
      int t, h;
      attend_row(p, spot, spot.hk, r, &t, &h);
      const int64_t at = (static_cast<int64_t>(spot.b) * a.T + t) * a.Hq + h;
      const float inv = attend_inverse(s[1]);
      typedef T V4 __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int ch = 16 * (quarter * NC + c) + 4 * g;
        V4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(out[m][c][e] * inv);
        if (ch < a.Dv) store_any(static_cast<T*>(a.out) + at * a.Dv + ch, y);
      }
      if (first) a.lse[at] = attend_lse(s[0], s[1]);
    }
  }
}

template <class T, int RT, int NC, bool SHARED>
void launch(const AttendParams& p, hipStream_t s) {
  hipLaunchKernelGGL((attend_wide_kernel<T, RT, NC, SHARED>), dim3(attend_grid(p)), dim3(kThreads),
                     sizeof(WideLds<RT, SHARED>), s, p);
}

}  // namespace

void launch_attend_wide(const AttendParams& p, int row_tiles, bool shared, hipStream_t s) {
  const bool bf16 = p.a.dtype == ETS_BF16;
  if (row_tiles == 4) {
    launch<__bf16, 4, 8, true>(p, s);
  } else if (shared) {
    bf16 ? launch<__bf16, 2, 8, true>(p, s) : launch<_Float16, 2, 8, true>(p, s);
  } else {
    bf16 ? launch<__bf16, 2, 9, false>(p, s) : launch<_Float16, 2, 9, false>(p, s);
  }
}

}  // namespace ets
