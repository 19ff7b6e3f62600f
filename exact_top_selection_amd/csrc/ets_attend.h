// What the attention kernels share: the launch's parameters and the finding of
// a list's keys (gfx950).
#ifndef ETS_ATTEND_H
#define ETS_ATTEND_H

#include <type_traits>

#include "ets_cache_format.h"

namespace ets {

constexpr int kAttendThreads = 256;
constexpr int kAttendWaves = 4;
constexpr int kAttendTile = 32;  // keys of a step
constexpr float kNegInf = -__builtin_inff();
// How far (log2) a score may pass the reference that its softmax is taken relative to, before the reference
// follows: probabilities up to 2^24 are as exact as those up to 1, and a list raises its reference once or twice.
// They enter the product with the values times 2^-24, so that the sums stay as far from overflow as the values' own.
// (A reference put 2^24 above the score instead left arguments of the exponential near -24: log-sum-exps of few keys were
// off by twice as much.)
constexpr float kSlack = 24.0f;
constexpr float kDown = 0x1p-24f, kUp = 0x1p24f;
constexpr float kLn2 = 0.69314718055994530942f;

struct AttendParams {
  ets_attend_args a;
  int G;             // query heads of a cache head
  int rows;          // query rows that share a list of keys: G, or T * G where all tokens share it
  int units;         // lists: (b, t, hk) or (b, hk)
  int row_groups;    // of a unit
  int splits;        // workgroups that share a list
  int heads;         // heads of a workgroup: 1, 2 or 4
  int tree_tiles;
  float scale_log2;  // log2(e) / sqrt(D)
  FastDiv by_page, by_heads, by_tokens, by_groups, by_splits, by_G, by_rows, by_inner, by_lanes, by_parts, by_unit_rows;
  int join_lanes, join_groups, join_parts;  // the join: lanes of a part of a row, shares of its splits, parts of a workgroup
  int group_rows;    // query rows of a workgroup, a multiple of 16
  float* part;       // [unit][row group][split][group_rows][Dv] sums
  f32x2* stat;       // [unit][row group][split][group_rows] (reference, sum)
};
// ... over a cache whose scales belong to blocks of slots
struct AttendBlocksParams : AttendParams {
  const int32_t* first;  // where a sequence's tokens stand, or null
  FastDiv by_block;
  int dealt;  // many rows; to the XCDs: 0, shares with all their heads; 1, lists; 2, workgroups
};

// Where a workgroup stands: its list, its query rows, its share of the keys.
// Workgroups are dealt out to the 8 XCDs in turn.  Those that read the same
// slots (the row groups and the heads of one share: 128 bytes of scales hold
// all heads of a slot, and often several slots) follow each other on one XCD,
// so that its L2 brings a line once: block = ((share / 8 * heads + head) *
// groups + group) * 8 + share % 8, where a "head" is what one workgroup takes.
struct AttendSpot {
  bool live;
  int split, group, row0, b, t;  // t: the token of a selected list, 0 for paged ones
  int hk;                        // the first of its heads
  uint32_t bt;
  bool paged;
  int n, main_tiles, tiles, first, last;
  uint64_t tree;  // drafted tokens that stand in the list
  int64_t begin;  // block caches: position of the first token
  int edge;       // block caches: positions from here on are not seen by all rows (but those of padding, which see none)
};
__device__ __forceinline__ uint32_t attend_deal(const AttendParams& p, AttendSpot* s) {
  const uint32_t y = blockIdx.x >> 3, eight = div_by(y, p.by_inner), in = y - eight * p.by_inner.d;
  const uint32_t share = eight * 8 + (blockIdx.x & 7), bt = div_by(share, p.by_splits);
  s->bt = bt;
  s->split = static_cast<int>(share - bt * p.splits);
  const int heads = static_cast<int>(div_by(in, p.by_groups));
  s->hk = heads * p.heads;
  s->group = static_cast<int>(in) - heads * p.row_groups;
  return bt;
}
// MANY: of the kernel for many rows.  All row groups of a list read the same rows, so they follow each other on one XCD
// where there are lists for all, and go to the XCDs in turn where not.
template <bool MANY = false, class P>
__device__ __forceinline__ AttendSpot attend_spot(const P& p) {
  const ets_attend_args& a = p.a;
  AttendSpot s;
  s.paged = a.slots == nullptr;
  uint32_t bt;
  if constexpr (MANY) {
    if (p.dealt == 1 || p.dealt == 2) {
      const uint32_t i = p.dealt == 1 ? blockIdx.x >> 3 : blockIdx.x, turn = div_by(i, p.by_groups);
      const uint32_t list = p.dealt == 1 ? turn * 8 + (blockIdx.x & 7) : turn, share = div_by(list, p.by_heads);
      bt = div_by(share, p.by_splits);
      s.bt = bt;
      s.split = static_cast<int>(share - bt * p.splits);
      s.hk = static_cast<int>(list - share * a.Hkv);
      s.group = static_cast<int>(i - turn * p.row_groups);
    } else {
      bt = attend_deal(p, &s);
    }
  } else {
    bt = attend_deal(p, &s);
  }
  s.row0 = s.group * p.group_rows;
  s.live = bt * a.Hkv < static_cast<uint32_t>(p.units);
  s.b = s.paged ? static_cast<int>(bt) : static_cast<int>(div_by(bt, p.by_tokens));
  s.t = s.paged ? 0 : static_cast<int>(bt) - s.b * a.T;
  if (!s.live) return s;
  s.n = s.paged ? min(max(a.seq_lens[s.b], 0), a.L) : a.K;
  if constexpr (std::is_same_v<P, AttendBlocksParams>) {
    s.begin = 0, s.edge = INT32_MAX;
    if (p.first) {
      // the workgroup's tokens, and how far they see
      s.begin = p.first[s.b];
      const int t0 = static_cast<int>(div_by(s.row0, p.by_G)), t1 = static_cast<int>(div_by(min(s.row0 + p.group_rows, p.rows) - 1, p.by_G));
      const int64_t clear = s.begin + (a.tree_mask ? 0 : t0 + 1), reach = s.begin + (a.tree_mask ? a.T : t1 + 1);
      const int n = s.begin + t0 < s.n ? static_cast<int>(min(static_cast<int64_t>(s.n), max(reach, static_cast<int64_t>(0)))) : 0;
      s.edge = static_cast<int>(min(max(clear, static_cast<int64_t>(0)), static_cast<int64_t>(INT32_MAX)));
      s.n = n;
    }
  }
  s.main_tiles = (s.n + kAttendTile - 1) / kAttendTile;
  s.tiles = s.main_tiles + p.tree_tiles;
  const int per = (s.tiles + p.splits - 1) / p.splits;
  s.first = s.split * per;
  s.last = min(s.first + per, s.tiles);
  // one token's list leaves out the drafted tokens that it does not see, so nothing of them is read
  s.tree = ~0ull;
  if (!s.paged && a.tree_slots) s.tree = static_cast<uint64_t>(a.tree_mask[s.b * a.mask_b + s.t]);
  if (a.T < 64) s.tree &= (1ull << a.T) - 1;
  return s;
}

// The slot of key `at` (0 to 31) of tile i, in two parts: the first asks memory
// for what it depends on, the second makes the slot of it (-1 where there is
// none), so that the wait can stand far from the request.  Neither branches (a
// load under way is waited for where branches meet): a key that is not there
// reads the kernel's first query.  The tree's tiles stand behind the main ones.
__device__ __forceinline__ bool attend_there(const AttendSpot& s, int i, int at) {
  const int j = i * kAttendTile + at, k = (i - s.main_tiles) * kAttendTile + at;
  return i < s.main_tiles ? j < s.n : i < s.tiles && (s.tree >> (k & 63) & 1);
}
__device__ __forceinline__ int32_t attend_ask(const AttendParams& p, const AttendSpot& s, int i, int at) {
  const ets_attend_args& a = p.a;
  const int j = i * kAttendTile + at, k = (i - s.main_tiles) * kAttendTile + at;
  const uint64_t list = s.paged ? reinterpret_cast<uint64_t>(a.page_table + s.b * a.pt_b)
                                : reinterpret_cast<uint64_t>(a.slots + s.b * a.slots_b + s.t * a.slots_t);
  const uint64_t tree = reinterpret_cast<uint64_t>(a.tree_slots + s.b * a.tree_b);
  const uint32_t page = div_by(static_cast<uint32_t>(j) & 0x7fffffffu, p.by_page);
  uint64_t from = i < s.main_tiles ? list + 4ull * (s.paged ? page : static_cast<uint32_t>(j)) : tree + 4ull * (k & 63);
  from = attend_there(s, i, at) ? from : reinterpret_cast<uint64_t>(a.q) & ~3ull;
  return load_global<int32_t>(from);
}
__device__ __forceinline__ int32_t attend_slot(const AttendParams& p, const AttendSpot& s, int i, int at, int32_t asked) {
  const int j = i * kAttendTile + at;
  const uint32_t page = div_by(static_cast<uint32_t>(j) & 0x7fffffffu, p.by_page);
  const int64_t paged = static_cast<int64_t>(asked) * p.a.page_size + (j - static_cast<int64_t>(page) * p.by_page.d);
  const int64_t slot = s.paged && i < s.main_tiles ? paged : asked;
  return attend_there(s, i, at) && asked >= 0 && slot < p.a.S ? static_cast<int32_t>(slot) : -1;
}

// (token, query head) of row r of head hk.
__device__ __forceinline__ void attend_row(const AttendParams& p, const AttendSpot& s, int hk, int r, int* t, int* h) {
  *t = s.paged ? static_cast<int>(div_by(r, p.by_G)) : s.t;
  *h = hk * p.G + (s.paged ? r - *t * p.G : r);
}

// Place of head hk's partial sums: [unit][row group][split].
__device__ __forceinline__ int64_t attend_place(const AttendParams& p, const AttendSpot& s, int hk) {
  return ((static_cast<int64_t>(s.bt) * p.a.Hkv + hk) * p.row_groups + s.group) * p.splits + s.split;
}

// Drafted tokens that some rows of a workgroup see and others do not: their
// probability is zero there, and zero times a value that is no number is not
// zero.  Such values are taken out of a tile before the second product, and
// two products of their places with what each row sees bring them back where
// they belong: large times large is infinity, and that less infinity no number.
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
constexpr uint16_t kLarge = 0x7f7f;  // the largest bf16
__device__ __forceinline__ bool no_number(uint16_t bf16) { return (bf16 & 0x7f80) == 0x7f80; }
__device__ __forceinline__ bf16x8 odd_places(bf16x8 v) {
  const u16x8 bits = __builtin_bit_cast(u16x8, v);
  u16x8 x;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = no_number(bits[e]) ? kLarge : 0;
  return __builtin_bit_cast(bf16x8, x);
}
// Bits 0..3 and 16..19 of vis: a lane's keys in the second product.
__device__ __forceinline__ bf16x8 seen_places(uint32_t vis) {
  u16x8 x;
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = vis >> (16 * (j >> 2) + (j & 3)) & 1 ? kLarge : 0;
  return __builtin_bit_cast(bf16x8, x);
}
__device__ __forceinline__ f32x4 spoilt(f32x4 x, bf16x8 odd, bf16x8 seen) {
  x = Mat<__bf16>::mma(odd, seen, x);
  return Mat<__bf16>::mma(odd, -seen, x);
}
__device__ __forceinline__ void clear_odd(void* eight) {  // in LDS
  u16x8 bits = *static_cast<u16x8*>(eight);
#pragma unroll
  for (int e = 0; e < 8; ++e) bits[e] = no_number(bits[e]) ? 0 : bits[e];
  *static_cast<u16x8*>(eight) = bits;
}

__device__ __forceinline__ float attend_lse(float reference, float sum) {
  // the sum's exponent first: it may cancel most of the reference
  const float whole = reference + static_cast<float>(__builtin_amdgcn_frexp_expf(sum) - 1);
  return sum == 0.0f ? kNegInf : (whole + __builtin_amdgcn_logf(2.0f * __builtin_amdgcn_frexp_mantf(sum))) * kLn2;
}
// What sums of values times kDown are multiplied by.
__device__ __forceinline__ float attend_inverse(float sum) {
  return sum > 0.0f || sum != sum ? kUp / sum : 0.0f;
}

inline int64_t attend_groups(const AttendParams& p) {
  const int64_t shares = static_cast<int64_t>(p.units / p.a.Hkv) * p.splits;
  return (shares + 7) / 8 * 8 * (p.a.Hkv / p.heads) * p.row_groups;
}
// ... of which a launch holds fewer than 2^32 lanes, as the plans see to
inline uint32_t attend_grid(const AttendParams& p) { return static_cast<uint32_t>(attend_groups(p)); }

// The launch of the kernel for heads over 256 channels (ets_attend_wide.hip);
// row_tiles: tiles of 16 query rows of a workgroup, as attend_wide_rows gives.
inline int attend_wide_rows(int rows, bool shared, bool bf16) {
  return shared && bf16 && rows > 32 ? 4 : 2;
}
void launch_attend_wide(const AttendParams& p, int row_tiles, bool shared, hipStream_t s);

}  // namespace ets

#endif  // ETS_ATTEND_H
