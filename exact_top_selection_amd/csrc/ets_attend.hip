// ets_attend.hip -- attention of one or a few tokens a sequence over an 8-bit
// cache: over selected slots or over whole paged sequences, plus a tree of
// drafted tokens (gfx950).
#include "ets_attend.h"

namespace ets {
namespace {

constexpr int kThreads = kAttendThreads;
constexpr int kWaves = kAttendWaves;
constexpr int kTile = kAttendTile;

constexpr int kChunk = 16;  // tiles whose slots are brought at a time

// Bytes of half a decoded row of 64 nv channels.
constexpr int value_plane(int nv) { return 64 * nv + (nv % 4 ? 0 : 64); }

// Workgroups of a compute unit, by registers (256 channels: also by LDS; two spilled, and were slower).
constexpr int attend_per_unit(int np, int mt) { return mt == 1 && np <= 2 ? 3 : (mt == 1 && np == 3) || (mt == 2 && np <= 2) ? 2 : 1; }

// One wave goes over its tiles of 32 keys alone, with the softmax's reference
// and running sum, and the four waves of a workgroup join at the end.  The
// reference is the largest score so far, raised only when one passes it by
// more than 2^24: a step in which none does, and all keys are seen, needs no
// largest score over the lanes and no rescaling.
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
// FULL: keys and values have 64 NP channels, so that no lane stands past a row
// (which saves a quarter of a step's vector instructions) and a row's scale
// bytes come in one load (64.0 to 58.4 us on the first case below).
//
// Measured: 59 us and 5 us of join for 16 sequences of 7 drafted tokens, 1024
// slots each, 32 heads on 8 of 128 channels, fp16 (265 MB brought for 235 MB of
// rows, the rest being the lines of the scales: 4.5 TB/s); 24 us and 4 us for
// one sequence of 32771, 64 heads on 8, bf16 (70 MB: 2.9 TB/s).  Rows of 128
// bytes come at 5.5 to 6.2 TB/s alone.  The bound is memory, less 5 to 8 us
// until the first rows are there (slots, then rows), which weighs most on the
// short case.  A wave has one tile under way while it works on another, twelve
// waves a compute unit; two tiles under way in registers spilled and were
// slower.
//
// Probabilities are the sum of two bf16 numbers (16 bits): with one, results of
// few keys were off by up to three times their own rounding to bf16, and the
// second costs nothing where the memory is what is waited for.
template <class T, int NP, int NV, int MT, bool FULL>
__global__ __launch_bounds__(kThreads, attend_per_unit(NP, MT)) void attend_kernel(AttendParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  // decoded values in LDS: rows of two planes, the lower and the upper halves of
  // their 16-channel pieces; rows lie 4 banks apart, planes not a multiple of 64
  constexpr int kPlane = value_plane(NV), kPitch = 2 * kPlane + 16;
  extern __shared__ __align__(16) char lds[];
  const ets_attend_args& a = p.a;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  char* values = lds + wave * (kTile * kPitch);
  f32x2* stats = reinterpret_cast<f32x2*>(lds + kWaves * kTile * kPitch);  // [wave][16 MT], then [head][16]
  int32_t* slots = reinterpret_cast<int32_t*>(stats + kWaves * 16 * (MT + 1));  // [3][kChunk * kTile]

  const AttendSpot spot = attend_spot(p);
  if (!spot.live) return;
  const int b = spot.b, row0 = spot.row0, main_tiles = spot.main_tiles, last = spot.last;
  const bool forked = spot.paged && p.tree_tiles > 0;  // rows of the workgroup see different drafted tokens
  // a wave's head, and the team of waves that share the head's keys
  const int hk = spot.hk + wave % p.heads, team = wave / p.heads, teams = kWaves / p.heads;

  // queries: lane (head col, row g) holds channels 64 i + 16 g + 0..7, 8..15
  V8 q[MT][NP][2];
  uint64_t tree_bits[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + 16 * m + col;
    int t, h;
    attend_row(p, spot, hk, r, &t, &h);
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

  // A tile's rows on their way: lane (key col of either half, row g) brings codes 64 i + 16 g .. + 15 and their
  // scale byte.  Rows and channels that are not there come from kNothing, without a branch.
  typedef RowScales<NP, FULL> KS;
  typedef RowScales<NV, FULL> VS;
  const uint64_t nothing = reinterpret_cast<uint64_t>(&kNothing[0]);
  const uint64_t kc = reinterpret_cast<uint64_t>(a.k_codes + hk * a.k_h + 16 * g);
  const uint64_t ks = KS::start(reinterpret_cast<uint64_t>(a.k_scales + hk * a.ks_h), g);
  const uint64_t vc = reinterpret_cast<uint64_t>(a.v_codes + hk * a.v_h + 16 * g);
  const uint64_t vs = VS::start(reinterpret_cast<uint64_t>(a.v_scales + hk * a.vs_h), g);
  const uint32_t k_row = static_cast<uint32_t>(a.k_s), ks_row = static_cast<uint32_t>(a.ks_s);
  const uint32_t v_row = static_cast<uint32_t>(a.v_s), vs_row = static_cast<uint32_t>(a.vs_s);
  struct Rows {
    u32v4 k[2][NP], v[2][NV];
    uint32_t kbyte[2][KS::n], vbyte[2][VS::n];
    uint32_t seen;  // keys that are there
  };

  // Slots come through LDS, kChunk tiles at a time, asked for two chunks ahead
  // by all lanes, so that the steps' own loads stay in one straight line.
  constexpr int kEach = kChunk * kTile / kThreads;
  int32_t asked[kEach];
  auto ask = [&](int c) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int key = threadIdx.x + j * kThreads;
      asked[j] = attend_ask(p, spot, spot.first + c * kChunk + key / kTile, key % kTile);
    }
  };
  auto keep = [&](int c) {
    int32_t* to = slots + c % 3 * (kChunk * kTile);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int key = threadIdx.x + j * kThreads, tile = spot.first + c * kChunk + key / kTile;
      to[key] = tile < last ? attend_slot(p, spot, tile, key % kTile, asked[j]) : -1;
    }
  };
  auto fetch = [&](Rows& rows, int i) {  // tile i of the workgroup's share
    const int32_t* from = slots + i / kChunk % 3 * (kChunk * kTile) + i % kChunk * kTile + col;
    const int32_t slot[2] = {from[0], from[16]};
    const uint64_t s0 = __ballot(slot[0] >= 0), s1 = __ballot(slot[1] >= 0);
    rows.seen = static_cast<uint32_t>(s0 & 0xffff) | static_cast<uint32_t>(s1 & 0xffff) << 16;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool there = slot[s] >= 0;
      const uint64_t at = static_cast<uint32_t>(slot[s]);
      // formed first and chosen then: an expression inside the choice would become a branch
      const uint64_t k0 = kc + at * k_row, k1 = ks + at * ks_row, v0 = vc + at * v_row, v1 = vs + at * vs_row;
      const uint64_t k = there ? k0 : nothing, kb = there ? k1 : nothing;
      const uint64_t v = there ? v0 : nothing, vb = there ? v1 : nothing;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const bool in = FULL || 64 * i + 16 * g < a.D;
        const uint64_t c = k + 64 * i;
        rows.k[s][i] = load_global<u32v4>(in ? c : nothing);
      }
      KS::load(rows.kbyte[s], kb, nothing, [&](int i) { return 64 * i + 16 * g < a.D; });
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = FULL || 64 * i + 16 * g < a.Dv;
        const uint64_t c = v + 64 * i;
        rows.v[s][i] = load_global<u32v4>(in ? c : nothing);
      }
      VS::load(rows.vbyte[s], vb, nothing, [&](int i) { return 64 * i + 16 * g < a.Dv; });
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

  auto work = [&](Rows& now, int step) {  // one tile; its rows' registers are asked to be filled again
    const int tile = spot.first + step;
    // keys to operands, values to LDS
    f32x4 score[MT][2];
    float row_scale[2];
    const uint32_t seen_now = now.seen;
    hold(now.k), hold(now.kbyte);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t r = 0;
      if constexpr (M::kRowScale) r = row_top<NP, FULL>(now.kbyte[s], now.k[s], g);
      row_scale[s] = __uint_as_float(r << 23);
#pragma unroll
      for (int m = 0; m < MT; ++m) score[m][s] = f32x4{};
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float f = M::scale(KS::byte(now.kbyte[s], i, g), r);
        const u32v4 c = now.k[s][i];
        const V8 k0 = M::keys(c[0], c[1], f), k1 = M::keys(c[2], c[3], f);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          score[m][s] = M::mma(k0, q[m][i][0], score[m][s]);
          score[m][s] = M::mma(k1, q[m][i][1], score[m][s]);
        }
      }
    }
    hold(now.v), hold(now.vbyte);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      char* dst = values + (16 * s + col) * kPitch + 16 * g;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float f = __uint_as_float(VS::byte(now.vbyte[s], i, g) << 23);
        const u32v4 c = now.v[s][i];
        *reinterpret_cast<bf16x8*>(dst + 64 * i) = codes_bf16(c[0], c[1], f);
        *reinterpret_cast<bf16x8*>(dst + kPlane + 64 * i) = codes_bf16(c[2], c[3], f);
      }
    }
    // the next tile's rows are on their way while this one is worked on; past the end they are zeros
    fetch(now, step + teams);
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
      // x: what goes into the exponential.  First as if all keys were seen and the reference stayed.
      float x[8], high = kNegInf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = __builtin_fmaf(score[m][j >> 2][j & 3], p.scale_log2, -top[m]);
        high = __builtin_elementwise_maximum(high, x[j]);  // no number (a score of -inf less a reference of -inf) passes no test
      }
      if (seen_now != ~0u || tile >= main_tiles || !__all(high <= kSlack)) {
        uint32_t vis = seen_now;
        if (tile >= main_tiles) vis &= static_cast<uint32_t>(tree_bits[m] >> (kTile * (tile - main_tiles) & 63));
        vis >>= 4 * g;  // bits 0..3: keys 4 g + e; bits 16..19: keys 16 + 4 g + e
        high = kNegInf;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (vis >> (16 * (j >> 2) + (j & 3))) & 1 ? score[m][j >> 2][j & 3] * p.scale_log2 : kNegInf;
          high = fmaxf(high, x[j]);
        }
        high = rows_max(high);
        if (__any(high > top[m] + kSlack || top[m] == kNegInf)) {
          const float next = high > top[m] + kSlack || top[m] == kNegInf ? high : top[m];
          const float fade = __builtin_amdgcn_exp2f(top[m] - (next == kNegInf ? 0.0f : next));
          sum[m] *= fade;
#pragma unroll
          for (int c = 0; c < 4 * NV; ++c) out[m][c] *= fade;
          top[m] = next;
        }
        const float base = top[m] == kNegInf ? 0.0f : top[m];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] -= base;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = __builtin_amdgcn_exp2f(x[j]);
        sum[m] += x[j];
        x[j] *= kDown;
        prob[m][j] = static_cast<__bf16>(x[j]);
        rest[m][j] = static_cast<__bf16>(x[j] - static_cast<float>(prob[m][j]));
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const char* src = values + (4 * g + (col >> 2)) * kPitch + kPlane * ((col >> 1) & 1) + 8 * (col & 1);
    auto value = [&](int c) {
      typedef __attribute__((address_space(3))) s16x4* Lds4;
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(src + 16 * c));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(src + 16 * kPitch + 16 * c));
      return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    };
    if (forked && tile >= main_tiles) {
      bf16x8 sees[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        sees[m] = seen_places((seen_now & static_cast<uint32_t>(tree_bits[m] >> (kTile * (tile - main_tiles) & 63))) >> (4 * g));
#pragma unroll
      for (int c = 0; c < 4 * NV; ++c) {
        const bf16x8 odd = odd_places(value(c));
#pragma unroll
        for (int m = 0; m < MT; ++m) out[m][c] = spoilt(out[m][c], odd, sees[m]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      for (int i = lane; i < kTile * 8 * NV; i += 64) {
        const int row = i / (8 * NV), piece = i % (8 * NV);
        clear_odd(values + row * kPitch + (piece & 1) * kPlane + 16 * (piece >> 1));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
#pragma unroll
    for (int c = 0; c < 4 * NV; ++c) {
      const bf16x8 v = value(c);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        out[m][c] = Mat<__bf16>::mma(v, prob[m], out[m][c]);
        out[m][c] = Mat<__bf16>::mma(v, rest[m], out[m][c]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  // Every wave takes as many steps (the barriers are shared); those past the end see nothing.
  const int steps = last - spot.first;
  if (steps > 0) {
    ask(0);
    keep(0);
    ask(1);
    __syncthreads();
    Rows rows;
    fetch(rows, team);
    hold(rows.kbyte), hold(rows.vbyte);  // else the loop carries 8-bit values and widens them as soon as they are loaded
    for (int step = team; step < steps + team; step += teams) {
      if (step % kChunk == team) {
        keep(step / kChunk + 1);
        ask(step / kChunk + 2);
        __syncthreads();
      }
      work(rows, step);
    }
  }

  // join the waves
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    sum[m] = rows_sum(sum[m]);
    if (g == 0) stats[(wave * MT + m) * 16 + col] = f32x2{top[m], sum[m]};
  }
  __syncthreads();
  const int dv = a.Dv;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    // over the waves of the same head: wave % heads, that plus heads, ...
    auto joined = [&](int of) {
      float high = kNegInf, total = 0.0f;
      for (int w = of; w < kWaves; w += p.heads) high = fmaxf(high, stats[(w * MT + m) * 16 + col][0]);
      const float base = high == kNegInf ? 0.0f : high;
      for (int w = of; w < kWaves; w += p.heads) {
        const f32x2 s = stats[(w * MT + m) * 16 + col];
        total += s[1] * __builtin_amdgcn_exp2f(s[0] - base);
      }
      return f32x2{high, total};
    };
    const f32x2 of_head = joined(wave % p.heads);
    const float fade = __builtin_amdgcn_exp2f(top[m] - (of_head[0] == kNegInf ? 0.0f : of_head[0]));
    // the wave's sums, [head][64 NV] floats, over its own values
    f32x4* mine = reinterpret_cast<f32x4*>(values) + col * (16 * NV) + g;
#pragma unroll
    for (int c = 0; c < 4 * NV; ++c) mine[4 * c] = out[m][c] * fade;
    f32x2* final = stats + kWaves * MT * 16;  // [head][16]
    if (team == 0 && g == 0) final[(wave % p.heads) * 16 + col] = of_head;
    __syncthreads();
    for (int i = threadIdx.x; i < p.heads * 256 * NV; i += kThreads) {
      const int of = i / (256 * NV), at = i - of * (256 * NV), row = at / (16 * NV), c = (at - row * (16 * NV)) * 4;
      const int r = row0 + 16 * m + row;
      if (r >= p.rows || c >= dv) continue;
      f32x4 v = {};
      for (int w = of; w < kWaves; w += p.heads)
        v += reinterpret_cast<const f32x4*>(lds + w * (kTile * kPitch))[at];
      const f32x2 s = final[of * 16 + row];
      if (p.splits > 1) {
        const int64_t place = attend_place(p, spot, spot.hk + of) * (16 * MT) + 16 * m + row;
        store_any(p.part + place * dv + c, v);
        if (c == 0) p.stat[place] = s;
      } else {
        int t, h;
        attend_row(p, spot, spot.hk + of, r, &t, &h);
        const int64_t place = (static_cast<int64_t>(b) * a.T + t) * a.Hq + h;
        const float inv = attend_inverse(s[1]);
        typedef T V4 __attribute__((ext_vector_type(4)));
        V4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<T>(v[e] * inv);
        store_any(static_cast<T*>(a.out) + place * dv + c, y);
        if (c == 0) a.lse[place] = attend_lse(s[0], s[1]);
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a list.  A lane stands at four channels of one row;
// join_lanes of them by join_groups shares of the splits take a part of the
// row, and a workgroup as many parts as it has lanes for: with few rows the
// splits are many, and their loads go out side by side.  4 us for 64 rows of
// 128 channels in 64 splits (the launch and three loads in turn), 11 us for
// 8192 rows of 512 in 2 (42 MB).
template <class T>
__global__ __launch_bounds__(kThreads) void join_kernel(AttendParams p) {
  const ets_attend_args& a = p.a;
  __shared__ f32x4 sums[kThreads];
  __shared__ f32x2 joined[kThreads];
  const int lanes = p.join_lanes;
  const int slot = static_cast<int>(div_by(threadIdx.x, p.by_lanes));  // part and share
  const int my_part = slot / p.join_groups, mine = slot - my_part * p.join_groups;
  const int64_t index = static_cast<int64_t>(blockIdx.x) * p.join_parts + my_part;
  const int64_t row_index = static_cast<int64_t>(div_by(static_cast<uint32_t>(index), p.by_parts));
  const int ch = 4 * (static_cast<int>(index - row_index * p.by_parts.d) * lanes + static_cast<int>(threadIdx.x) - slot * lanes);
  const bool live = my_part < p.join_parts && row_index < static_cast<int64_t>(p.units) * p.rows;
  const uint32_t unit = live ? div_by(static_cast<uint32_t>(row_index), p.by_unit_rows) : 0;
  const int r = live ? static_cast<int>(row_index - static_cast<int64_t>(unit) * p.rows) : 0;
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
    // lanes of no part stand past the last share: theirs would be read behind the arrays
    if (mine != 0 || !live) return;
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
