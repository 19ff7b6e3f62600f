// Device helpers shared by the kernels around the selection: vector types,
// the 8-bit cache format and cross-lane sums (gfx950, wave64).
#ifndef ETS_CACHE_FORMAT_H
#define ETS_CACHE_FORMAT_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ets_decode.h"

namespace ets {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kCacheBlock = 32;    // values that share a scale byte
constexpr int kScaleBias = 127;    // value = code * 2^(byte - 127)
constexpr int kScaleLow = -126, kScaleHigh = 119;

// Loads and stores of V at any address (one instruction whatever the alignment).
template <class V>
__device__ __forceinline__ V load_any(const void* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}
template <class V>
__device__ __forceinline__ void store_any(void* p, const V& v) {
  __builtin_memcpy(p, &v, sizeof(V));
}

// A load from a global address held as a number (so that an address can be
// chosen without a branch and the load stays a global one), at any alignment.
template <class V>
__device__ __forceinline__ V load_global(uint64_t address) {
  struct __attribute__((packed)) Any { V v; };
  return reinterpret_cast<const __attribute__((address_space(1))) Any*>(address)->v;
}

// Read in the place of a row that is not there (576 zeros).
static __device__ const u32v4 kNothing[ETS_MAX_HEAD_DIM / 16] = {};

// Keeps what is made of loaded values behind this point: made earlier, it would wait for the load there.
template <class V, int A, int B>
__device__ __forceinline__ void hold(V (&x)[A][B]) {
#pragma unroll
  for (int i = 0; i < A; ++i)
#pragma unroll
    for (int j = 0; j < B; ++j) asm volatile("" : "+v"(x[i][j]));
}

// The scale bytes of a row on their way through the lanes that hold it (lane row g: codes 64 i + 16 g .. + 15).  A
// row of 2 NP bytes (FULL; NP 1, 2 or 4) comes in one load that its four lanes share, other rows byte by byte.
template <int NP, bool FULL>
struct RowScales {
  static constexpr bool kWhole = FULL && NP != 3;
  static constexpr int n = kWhole ? (NP + 1) / 2 : NP;  // registers
  // where a lane starts to read
  static __device__ __forceinline__ uint64_t start(uint64_t row, int g) { return kWhole ? row : row + (g >> 1); }
  // w <- the bytes at `from`; a byte of a step i that `in` does not have is read from `nothing`
  template <class In>
  static __device__ __forceinline__ void load(uint32_t (&w)[n], uint64_t from, uint64_t nothing, In in) {
    if constexpr (kWhole && NP == 1) {
      w[0] = load_global<uint16_t>(from);
    } else if constexpr (kWhole && NP == 2) {
      w[0] = load_global<uint32_t>(from);
    } else if constexpr (kWhole) {
      const u32v2 two = load_global<u32v2>(from);
      w[0] = two[0], w[1] = two[1];
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint64_t b = from + 2 * i;
        w[i] = load_global<uint8_t>(in(i) ? b : nothing);
      }
    }
  }
  static __device__ __forceinline__ uint32_t byte(const uint32_t (&w)[n], int i, int g) {
    return kWhole ? __builtin_amdgcn_ubfe(w[kWhole ? i / 2 : i], 16 * (i & 1) + 8 * (g >> 1), 8) : w[i];
  }
};

// n / d for 0 <= n < 2^31 and a divisor d >= 1 fixed at launch: with l =
// ceil(log2 d) and m = ceil(2^(31 + l) / d), n * m / 2^(31 + l) exceeds n / d
// by less than n / 2^(31 + l) <= 1 / d, so the floor is exact.  d lies in
// (2^(l - 1), 2^l], so m lies in [2^31, 2^32).
struct FastDiv {
  uint32_t m, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  const uint32_t shift = 31 + l;
  const uint64_t q = (static_cast<uint64_t>(1) << shift) / d, r = (static_cast<uint64_t>(1) << shift) % d;
  return {static_cast<uint32_t>(q + (r ? 1 : 0)), shift, d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * f.m) >> f.shift);
}

// Sum, largest over the lanes l, l ^ 16, l ^ 32, l ^ 48: the swaps exchange
// whole 16-lane rows, without LDS.
__device__ __forceinline__ float rows_sum(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const float y = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  const uint32_t c = __float_as_uint(y);
  const auto t = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}
__device__ __forceinline__ float rows_max(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const float y = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  const uint32_t c = __float_as_uint(y);
  const auto t = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return fmaxf(__uint_as_float(t[0]), __uint_as_float(t[1]));
}

// The exponent that a row is taken over, in all of its lanes, as a scale byte:
// the row's largest one where every 16 codes have one of at least 2, as those
// of cache_write nearly always do (so that the largest block's values reach
// high).  A block of zeros, or of codes that are small for their scale, says
// nothing of the row's size: with one in sight the byte follows the largest
// value, so that it comes to lie in [2^8, 2^9).  (Byte 0: a row or channels that are
// not there.)
template <int NP, bool FULL>
__device__ __forceinline__ uint32_t row_top(const uint32_t (&w)[RowScales<NP, FULL>::n], const u32v4 (&codes)[NP], int g) {
  typedef RowScales<NP, FULL> R;
  uint32_t least = ~0u;  // 0: some 16 codes without one of 2
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const u32v4 c = codes[i];
    const uint32_t any = (c[0] | c[1] | c[2] | c[3]) & 0x40404040u;
    least = min(least, FULL || R::byte(w, i, g) ? any : ~0u);
  }
  const bool small = least == 0 && (!FULL || w[0] != 0);
  uint32_t top = 0;
  if (__any(small)) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      u16x2 high = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        high = __builtin_elementwise_max(high, __builtin_bit_cast(u16x2, codes[i][j] & 0x007f007fu));
        high = __builtin_elementwise_max(high, __builtin_bit_cast(u16x2, codes[i][j] >> 8 & 0x007f007fu));
      }
      const uint32_t code = max(high[0], high[1]);
      const int byte = static_cast<int>(R::byte(w, i, g)) - 15 + static_cast<int>(code >> 3);
      top = code ? max(top, static_cast<uint32_t>(max(byte, 1))) : top;
    }
    return __float_as_uint(rows_max(__uint_as_float(top << 23))) >> 23;
  }
  if constexpr (R::kWhole) {
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) top = max(top, __builtin_amdgcn_ubfe(w[i / 4], 8 * (i & 3), 8));
    return top;
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) top = max(top, w[i]);
    return __float_as_uint(rows_max(__uint_as_float(top << 23))) >> 23;
  }
}

// Eight codes (two words) to eight values times `scale`, a power of two.
// bf16 holds every value of the format exactly (4 significant bits; results
// below 2^-133 round).
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ f16x8 codes_f16(uint32_t lo, uint32_t hi, float scale) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The matrix operand types of a query type.  A key is brought to the query's
// own type, so that products are exact in 32 bits:
//   bf16  the key's values;
//   fp16  the key's values over 2^(r - 127), r from row_top: less than 2^9, and
//         a block far below the row's largest loses bits only beneath 2^-25,
//         which is 2^-33 of the row's largest value (2^-26 where no code of the
//         largest block is over 2).  The product is multiplied by 2^(r - 127)
//         afterwards.
template <class T>
struct Mat;
template <>
struct Mat<__bf16> {
  typedef bf16x8 V8;
  static constexpr bool kRowScale = false;
  static __device__ __forceinline__ float scale(uint32_t byte, uint32_t) { return __uint_as_float(byte << 23); }
  static __device__ __forceinline__ V8 keys(uint32_t lo, uint32_t hi, float s) { return codes_bf16(lo, hi, s); }
  static __device__ __forceinline__ f32x4 mma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mat<_Float16> {
  typedef f16x8 V8;
  static constexpr bool kRowScale = true;
  static __device__ __forceinline__ float scale(uint32_t byte, uint32_t top) {
    const int e = static_cast<int>(byte) - static_cast<int>(top) + kScaleBias;
    return __uint_as_float(static_cast<uint32_t>(min(max(e, 0), 254)) << 23);  // over 142 for blocks of zeros only
  }
  static __device__ __forceinline__ V8 keys(uint32_t lo, uint32_t hi, float s) { return codes_f16(lo, hi, s); }
  static __device__ __forceinline__ f32x4 mma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// HIP launches fewer than 2^32 lanes at a time.  More workgroups than that go out in several launches, each told the
// number of its first one: launch(first, how many).
constexpr int64_t kMostLanes = static_cast<int64_t>(1) << 31;
template <class F>
void launch_in_turn(int64_t groups, int threads, F launch) {
  const int64_t most = kMostLanes / threads;
  for (int64_t first = 0; first < groups; first += most)
    launch(static_cast<uint32_t>(first), static_cast<uint32_t>(groups - first < most ? groups - first : most));
}

inline bool dtype_known(int32_t dtype) { return dtype == ETS_BF16 || dtype == ETS_FP16 || dtype == ETS_FP32; }

// ETS_OK where the current device is a gfx950; the device's compute units.
inline ets_status device_ready(int32_t* cu_count) {
  int32_t xcd = 0, occ = 0;
  return ets_device_limits(-1, cu_count, &xcd, &occ);
}

}  // namespace ets

#endif  // ETS_CACHE_FORMAT_H
