// ets_rope_cache.hip -- rotary positions and the 8-bit cache's write and read
// (gfx950).  All three move each byte once and are bound by memory; the
// sources below keep 16-byte accesses and several loads in flight a lane.
#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kRopeTable = 2048;  // (cos, sin) pairs of a workgroup's tokens, in LDS (16 KiB)
constexpr int kBatch = 4;         // vectors a lane has in flight
constexpr int kRopeStage = 16 * kBatch * kThreads;  // bytes of rows that the staged form holds in LDS: all of a workgroup's
// vectors of a lane of the read: one more load under way hides the slot's; 4 and more took longer (131072 x 576: 46 us with
// 2, 47 with 1, 50 with 4, 56 with 8, whose few workgroups end unevenly)
constexpr int kReadBatch = 2;
// Outputs over this size pass the L2s by (they hold 32 MiB in all): the rows being read keep their place there.
constexpr int64_t kStream = 32 << 20;

enum RopeMode { kInterleaved = 0, kHalf = 1, kStaged = 2 };

struct RopeParams {
  const char* x;
  char* out;
  int64_t x_n, x_h, out_n, out_h;  // bytes
  int64_t N;
  int H, D, R, offset, layout, inverse;
  const int32_t* positions;
  const double* inv_freq;
  double scale;
  int tokens, heads;  // of a workgroup
  bool stream;
  int head_groups;
  FastDiv by_items, by_heads, by_pairs, by_groups;
};

template <class T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
};

template <class V>
__device__ __forceinline__ void put(char* to, const V& v, bool stream) {
  typedef u32v4 Any __attribute__((aligned(2)));
  if (stream) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32v4, v), reinterpret_cast<Any*>(to));
  } else {
    store_any(to, v);
  }
}

// Cosine and sine of an angle in radians, in 64 bits.  The angle goes to turns
// with 1 / (2 pi) in two parts (one alone is off by 2e-7 radians at 2^31), less
// the nearest whole quarter; the rest lies within pi / 4, where Taylor's series
// to the 12th and 13th power are off by less than 4e-13.
struct Turn {
  double c, s;
};
__device__ __forceinline__ Turn turn_of(double angle) {
  const double high = 0.15915494309189535, low = -9.839338337591243e-18;
  const double turns = angle * high, rest = fma(angle, high, -turns) + angle * low;
  const double quarters = rint(4.0 * turns);
  const double a = ((turns - 0.25 * quarters) + rest) * 6.283185307179586, b = a * a;
  double c = 1.0 / 479001600, s = 1.0 / 6227020800;
  c = fma(c, b, -1.0 / 3628800), s = fma(s, b, -1.0 / 39916800);
  c = fma(c, b, 1.0 / 40320), s = fma(s, b, 1.0 / 362880);
  c = fma(c, b, -1.0 / 720), s = fma(s, b, -1.0 / 5040);
  c = fma(c, b, 1.0 / 24), s = fma(s, b, 1.0 / 120);
  c = fma(c, b, -1.0 / 2), s = fma(s, b, -1.0 / 6);
  c = fma(c, b, 1.0), s = fma(s * b, a, a);
  const int quarter = static_cast<int>(quarters - 4.0 * rint(0.25 * quarters)) & 3;
  const double x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? Turn{-x, -y} : Turn{x, y};
}

// Rotary positions.  A workgroup takes `tokens` tokens and `heads` of their
// heads.  The cosines and sines of a token serve all its heads: they are
// formed once, in LDS, times the scale, in 64 bits and rounded once.
//
// kInterleaved / kHalf: a lane turns one or two 16-byte vectors whose pairs it
// holds whole.  kStaged: pairs that cross vectors (odd offsets, odd R / 2, D
// not a multiple of a vector).  A lane holds its vectors as in the other forms,
// all rows of the workgroup go to LDS as well (out may be x), and the partners
// of a vector's channels come from there as one or two vectors at any address.
//
// Measured: 42 us for 16384 x 32 heads of 128 channels in bf16 (268 MB, 6.4
// TB/s; a copy of 1 GiB reaches 5.2), 7.2 us for the transposed map of 4099 x 9
// x 96 in fp32 (28 MB), 3 us for a single token (the launch); staged: 46 us for
// 8344 x 10 x 480 in bf16, 200 channels from 259 on (160 MB: 3.5 TB/s), bound by
// vector instructions, which take 87000 of a SIMD's 98000 cycles (choosing each
// channel's partner, coefficient and sign).
template <class T, int MODE>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p) {
  constexpr int V = Vec<T>::n;
  typedef typename Vec<T>::type VT;
  __shared__ f32x2 table[kRopeTable];
  __shared__ __align__(16) char stage[MODE == kStaged ? kRopeStage + 32 : 16];

  const uint32_t tile = div_by(blockIdx.x, p.by_groups);
  const int64_t n0 = static_cast<int64_t>(tile) * p.tokens;
  const int h0 = static_cast<int>(blockIdx.x - tile * p.head_groups) * p.heads;
  const int tokens = static_cast<int>(p.N - n0 < p.tokens ? p.N - n0 : p.tokens);
  const int heads = min(p.heads, p.H - h0);
  const int pairs = p.R >> 1;
  // vectors of a row: whole ones, and for the staged form a short last one
  const int items = MODE == kHalf ? pairs / V + (p.D - p.R) / V : (p.D + V - 1) / V;
  // rows are numbered token by token over p.heads heads; those past the last head are skipped
  const int total = tokens * p.heads * items;

  struct Item {
    int64_t in, out;
    int token, v;
    bool live;
  };
  auto item_of = [&](int i) {
    Item it;
    it.live = i < total;
    const uint32_t row = div_by(it.live ? i : 0, p.by_items);
    it.v = (it.live ? i : 0) - static_cast<int>(row) * items;
    it.token = static_cast<int>(div_by(row, p.by_heads));
    const int h = static_cast<int>(row) - it.token * p.heads;
    it.live = it.live && h < heads;
    it.in = (n0 + it.token) * p.x_n + static_cast<int64_t>(h0 + h) * p.x_h;
    it.out = (n0 + it.token) * p.out_n + static_cast<int64_t>(h0 + h) * p.out_h;
    return it;
  };
  // first channel of vector v; kHalf: v below pairs / V are the first members of pairs
  const int half_vecs = pairs / V;
  auto channel = [&](int v) {
    if (MODE != kHalf) return v * V;
    if (v < half_vecs) return p.offset + v * V;
    const int c = (v - half_vecs) * V;
    return c < p.offset ? c : c + p.R;
  };

  VT a[kBatch], b[kBatch];
  Item it[kBatch];
  auto fetch = [&](int base) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      it[u] = item_of(base + u * kThreads + static_cast<int>(threadIdx.x));
      if (it[u].live) {
        const char* src = p.x + it[u].in + static_cast<int64_t>(channel(it[u].v)) * sizeof(T);
        const int left = p.D - it[u].v * V;
        if (MODE == kStaged && left < V) {  // a short last vector
          a[u] = VT{};
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j < left) a[u][j] = reinterpret_cast<const T*>(src)[j];
          continue;
        }
        a[u] = load_any<VT>(src);
        if (MODE == kHalf && it[u].v < half_vecs) b[u] = load_any<VT>(src + static_cast<int64_t>(pairs) * sizeof(T));
      }
    }
  };
  fetch(0);  // all of them in the staged form

  const double sine = p.inverse ? -p.scale : p.scale;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = static_cast<int>(div_by(i, p.by_pairs)), f = i - t * pairs;
    const Turn turn = turn_of(static_cast<double>(p.positions[n0 + t]) * p.inv_freq[f]);
    table[i] = f32x2{static_cast<float>(turn.c * p.scale), static_cast<float>(turn.s * sine)};
  }

  // staged rows lie 16 * items bytes apart, with a vector of room before and behind them
  T* const rows = reinterpret_cast<T*>(stage) + V;
  if (MODE == kStaged) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = u * kThreads + static_cast<int>(threadIdx.x);
      if (it[u].live) *reinterpret_cast<VT*>(rows + i * V) = a[u];
    }
  }
  __syncthreads();

  if (MODE == kStaged) {
    const bool half = p.layout == ETS_ROPE_HALF;
    const int apart = half ? pairs : 1;  // channels between the members of a pair
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!it[u].live) continue;
      const int at = it[u].v * V, r0 = at - p.offset, count = min(V, p.D - at);
      const f32x2* cs = table + it[u].token * pairs;
      const T* own = rows + (u * kThreads + static_cast<int>(threadIdx.x)) * V;
      VT y = a[u];
      if (r0 + V > 0 && r0 < p.R) {
        // the partners of first and of second members; a vector that has none reads its own place
        const VT next = load_any<VT>(half && r0 >= pairs ? own : own + apart);
        const VT before = load_any<VT>(half && r0 + V <= pairs ? own : own - apart);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int r = r0 + j;
          const bool turns = static_cast<uint32_t>(r) < static_cast<uint32_t>(p.R), second = half ? r >= pairs : r & 1;
          const f32x2 c = cs[turns ? half ? (second ? r - pairs : r) : r >> 1 : 0];
          const float v = static_cast<float>(a[u][j]), w = static_cast<float>(second ? before[j] : next[j]);
          const T to = static_cast<T>(second ? v * c[0] + w * c[1] : v * c[0] - w * c[1]);
          y[j] = turns ? to : y[j];
        }
      }
      char* dst = p.out + it[u].out + static_cast<int64_t>(at) * sizeof(T);
      if (count == V) {
        put(dst, y, p.stream);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j < count) reinterpret_cast<T*>(dst)[j] = y[j];
      }
    }
    return;
  }

  for (int base = 0; base < total; base += kBatch * kThreads) {
    if (base) fetch(base);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!it[u].live) continue;
      const int at = channel(it[u].v);
      char* dst = p.out + it[u].out + static_cast<int64_t>(at) * sizeof(T);
      const f32x2* cs = table + it[u].token * pairs;
      if (MODE == kHalf) {
        if (it[u].v < half_vecs) {
          VT y, z;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const f32x2 c = cs[it[u].v * V + j];
            const float v = static_cast<float>(a[u][j]), w = static_cast<float>(b[u][j]);
            y[j] = static_cast<T>(v * c[0] - w * c[1]);
            z[j] = static_cast<T>(w * c[0] + v * c[1]);
          }
          put(dst, y, p.stream);
          put(dst + static_cast<int64_t>(pairs) * sizeof(T), z, p.stream);
        } else {
          put(dst, a[u], p.stream);
        }
      } else {
        VT y = a[u];
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const int r = at + j - p.offset;
          if (static_cast<uint32_t>(r) < static_cast<uint32_t>(p.R)) {
            const f32x2 c = cs[r >> 1];
            const float v = static_cast<float>(a[u][j]), w = static_cast<float>(a[u][j + 1]);
            y[j] = static_cast<T>(v * c[0] - w * c[1]);
            y[j + 1] = static_cast<T>(w * c[0] + v * c[1]);
          }
        }
        put(dst, y, p.stream);
      }
    }
  }
}

struct CacheParams {
  const char* x;     // write: rows in
  char* out;         // read: rows out, contiguous
  int64_t x_n, x_h;  // bytes
  const int32_t* slots;
  uint8_t* codes;
  uint8_t* scales;
  int64_t codes_s, codes_h, scales_s, scales_h, S;
  uint32_t items;  // of this launch
  bool stream;
  FastDiv by_row, by_heads;
};

template <int CTRL>
__device__ __forceinline__ float quad(float x) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// Cache write: a lane holds 8 values, four neighbouring lanes a block of 32;
// the block's largest magnitude goes round the four lanes.  Non-finite values
// take no part in it.
//
// Measured: 19 us for 32768 rows of 8 x 128 in fp16 to random slots (102 MB,
// 5.3 TB/s), as long as a copy takes; 4 us for 64 rows of 576 (the launch).
template <class T>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheParams p) {
  typedef T V8 __attribute__((ext_vector_type(8)));
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.items) return;  // items is a multiple of 4: quads leave whole
  const uint32_t row = div_by(i, p.by_row), v = i - row * p.by_row.d;
  const uint32_t n = div_by(row, p.by_heads), h = row - n * p.by_heads.d;
  const int64_t slot = p.slots[n];
  const V8 in = load_any<V8>(p.x + n * p.x_n + h * p.x_h + static_cast<int64_t>(v) * 8 * sizeof(T));
  if (slot < 0 || slot >= p.S) return;
  float x[8], top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = static_cast<float>(in[j]);
    const float size = fabsf(x[j]);
    top = size < __builtin_inff() ? fmaxf(top, size) : top;
  }
  top = fmaxf(top, quad<0xB1>(top));
  top = fmaxf(top, quad<0x4E>(top));
  // top = m * 2^q with m in [1/2, 1): 448 = 7/8 * 2^9, so e = q - 9 where m <= 7/8, else q - 8
  int q;
  const float m = frexpf(top, &q);
  int e = m <= 0.875f ? q - 9 : q - 8;
  e = min(max(e, kScaleLow), kScaleHigh);
  const float inv = __uint_as_float(static_cast<uint32_t>(kScaleBias - e) << 23);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = x[j] * inv;
    x[j] = y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  store_any(p.codes + slot * p.codes_s + h * p.codes_h + v * 8,
            u32v2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)});
  if ((v & 3) == 0) p.scales[slot * p.scales_s + h * p.scales_h + (v >> 2)] = static_cast<uint8_t>(e + kScaleBias);
}

// Cache read: a lane makes kReadBatch 16-byte vectors of values.  They are
// formed in 32 bits and rounded once.
//
// Measured: 46 us for 131072 random rows of 576 in bf16 (229 MB, 5.0 TB/s; 255
// MB with the whole lines of codes and scales that the rows touch).
template <class T>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheParams p) {
  constexpr int V = Vec<T>::n;
  typedef typename Vec<T>::type VT;
  const uint32_t base = blockIdx.x * (kReadBatch * kThreads) + threadIdx.x;
  u32v2 code[kReadBatch];
  uint32_t byte[kReadBatch];
#pragma unroll
  for (int u = 0; u < kReadBatch; ++u) {
    const uint32_t i = base + u * kThreads;
    code[u] = u32v2{0, 0};
    byte[u] = 0;
    if (i >= p.items) continue;
    const uint32_t row = div_by(i, p.by_row), v = i - row * p.by_row.d;
    const uint32_t n = div_by(row, p.by_heads), h = row - n * p.by_heads.d;
    const int64_t slot = p.slots[n];
    if (slot < 0 || slot >= p.S) continue;
    const uint8_t* src = p.codes + slot * p.codes_s + h * p.codes_h + v * V;
    if (V == 8) {
      code[u] = load_any<u32v2>(src);
    } else {
      code[u][0] = load_any<uint32_t>(src);
    }
    byte[u] = p.scales[slot * p.scales_s + h * p.scales_h + v * V / kCacheBlock];
  }
#pragma unroll
  for (int u = 0; u < kReadBatch; ++u) {
    const uint32_t i = base + u * kThreads;
    if (i >= p.items) continue;
    VT y;
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const uint32_t w = code[u][j / 4];
      const f32x2 f = (j & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
      const int e = static_cast<int>(byte[u]) - kScaleBias;
      y[j] = static_cast<T>(ldexpf(f[0], e));
      y[j + 1] = static_cast<T>(ldexpf(f[1], e));
    }
    put(p.out + static_cast<int64_t>(i) * 16, y, p.stream);
  }
}

int64_t size_of(int32_t dtype) { return dtype == ETS_FP32 ? 4 : 2; }

template <class T>
void launch_rope(const RopeParams& p, int mode, uint32_t grid, hipStream_t s) {
  if (mode == kInterleaved) {
    hipLaunchKernelGGL((rope_kernel<T, kInterleaved>), dim3(grid), dim3(kThreads), 0, s, p);
  } else if (mode == kHalf) {
    hipLaunchKernelGGL((rope_kernel<T, kHalf>), dim3(grid), dim3(kThreads), 0, s, p);
  } else {
    hipLaunchKernelGGL((rope_kernel<T, kStaged>), dim3(grid), dim3(kThreads), 0, s, p);
  }
}

ets_status check_cache(int64_t N, int32_t H, int32_t D, int64_t S, const void* slots, const void* rows,
                       const void* codes, const void* scales, int32_t dtype) {
  if (N < 0 || H < 1 || D < kCacheBlock || D % kCacheBlock || S < 0 || !dtype_known(dtype)) return ETS_ERR_INVALID_ARG;
  if (static_cast<int64_t>(H) * D > (1 << 28)) return ETS_ERR_INVALID_ARG;
  if (N && (!slots || !rows || !codes || !scales)) return ETS_ERR_INVALID_ARG;
  return ETS_OK;
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_rope(const void* x, int64_t x_n, int64_t x_h, void* out, int64_t out_n, int64_t out_h,
                    int64_t N, int32_t H, int32_t D, const int32_t* positions, const double* inv_freq,
                    int32_t R, int32_t offset, int32_t layout, double scale, int32_t inverse,
                    int32_t dtype, void* stream) {
  using namespace ets;
  if (N < 0 || H < 0 || D < 1 || D > ETS_MAX_ROPE_DIM || R < 0 || (R & 1) || offset < 0 || offset > D - R || !dtype_known(dtype) ||
      (layout != ETS_ROPE_INTERLEAVED && layout != ETS_ROPE_HALF))
    return ETS_ERR_INVALID_ARG;
  if (N == 0 || H == 0) return ETS_OK;
  if (!x || !out || !positions || (R && !inv_freq)) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int size = static_cast<int>(size_of(dtype)), V = 16 / size, pairs = R / 2;
  int mode = kStaged;
  if (D % V == 0) {
    if (layout == ETS_ROPE_INTERLEAVED && offset % 2 == 0) mode = kInterleaved;
    if (layout == ETS_ROPE_HALF && offset % V == 0 && pairs % V == 0) mode = kHalf;
  }
  const int items = mode == kHalf ? pairs / V + (D - R) / V : (D + V - 1) / V;
  RopeParams p{};
  p.x = static_cast<const char*>(x);
  p.out = static_cast<char*>(out);
  p.x_n = x_n * size, p.x_h = x_h * size, p.out_n = out_n * size, p.out_h = out_h * size;
  p.N = N, p.H = H, p.D = D, p.R = R, p.offset = offset, p.layout = layout, p.inverse = inverse;
  p.stream = N * H * D * size > kStream;
  p.positions = positions, p.inv_freq = inv_freq, p.scale = scale;
  // vectors of a workgroup: one a lane where the whole call has few, up to kBatch
  // a lane where it fills the device
  const int64_t all = N * H * items;
  int64_t want = all / (static_cast<int64_t>(cu) * 8);
  want = want < kThreads ? kThreads : want > kBatch * kThreads ? kBatch * kThreads : want;
  int64_t rows = want / items;
  if (rows < 1) rows = 1;
  p.heads = static_cast<int>(rows < H ? rows : H);
  int64_t tokens = rows / p.heads;
  if (pairs && tokens * pairs > kRopeTable) tokens = kRopeTable / pairs;
  p.tokens = static_cast<int>(tokens < N ? tokens : N);
  p.head_groups = (H + p.heads - 1) / p.heads;
  const int64_t grid = (N + p.tokens - 1) / p.tokens * p.head_groups;
  if (grid > INT32_MAX) return ETS_ERR_INVALID_ARG;
  p.by_items = fast_div(items);
  p.by_heads = fast_div(p.heads);
  p.by_pairs = fast_div(pairs ? pairs : 1);
  p.by_groups = fast_div(p.head_groups);
  auto s = static_cast<hipStream_t>(stream);
  const uint32_t g = static_cast<uint32_t>(grid);
  if (dtype == ETS_BF16) {
    launch_rope<__bf16>(p, mode, g, s);
  } else if (dtype == ETS_FP16) {
    launch_rope<_Float16>(p, mode, g, s);
  } else {
    launch_rope<float>(p, mode, g, s);
  }
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

ets_status ets_cache_write(const void* x, int64_t x_n, int64_t x_h, int64_t N, int32_t H, int32_t D,
                           const int32_t* slots, uint8_t* codes, int64_t codes_s, int64_t codes_h,
                           uint8_t* scales, int64_t scales_s, int64_t scales_h, int64_t S,
                           int32_t dtype, void* stream) {
  using namespace ets;
  if (ets_status st = check_cache(N, H, D, S, slots, x, codes, scales, dtype); st != ETS_OK) return st;
  if (N == 0 || S == 0) return ETS_OK;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int64_t size = size_of(dtype);
  const uint32_t row = D / 8;
  const int64_t step = (static_cast<int64_t>(1) << 30) / (static_cast<int64_t>(row) * H);  // rows of a launch
  auto s = static_cast<hipStream_t>(stream);
  for (int64_t n = 0; n < N; n += step) {
    const int64_t count = N - n < step ? N - n : step;
    CacheParams p{};
    p.x = static_cast<const char*>(x) + n * x_n * size;
    p.x_n = x_n * size, p.x_h = x_h * size;
    p.slots = slots + n;
    p.codes = codes, p.codes_s = codes_s, p.codes_h = codes_h;
    p.scales = scales, p.scales_s = scales_s, p.scales_h = scales_h, p.S = S;
    p.items = static_cast<uint32_t>(count * H * row);
    p.by_row = fast_div(row);
    p.by_heads = fast_div(H);
    const uint32_t grid = (p.items + kThreads - 1) / kThreads;
    if (dtype == ETS_BF16) {
      hipLaunchKernelGGL(cache_write_kernel<__bf16>, dim3(grid), dim3(kThreads), 0, s, p);
    } else if (dtype == ETS_FP16) {
      hipLaunchKernelGGL(cache_write_kernel<_Float16>, dim3(grid), dim3(kThreads), 0, s, p);
    } else {
      hipLaunchKernelGGL(cache_write_kernel<float>, dim3(grid), dim3(kThreads), 0, s, p);
    }
    if (hipGetLastError() != hipSuccess) return ETS_ERR_HIP;
  }
  return ETS_OK;
}

ets_status ets_cache_read(const uint8_t* codes, int64_t codes_s, int64_t codes_h, const uint8_t* scales,
                          int64_t scales_s, int64_t scales_h, int64_t S, const int32_t* slots, int64_t N,
                          int32_t H, int32_t D, void* out, int32_t dtype, void* stream) {
  using namespace ets;
  if (ets_status st = check_cache(N, H, D, S, slots, out, S ? codes : static_cast<const void*>(out),
                                  S ? scales : static_cast<const void*>(out), dtype);
      st != ETS_OK)
    return st;
  if (N == 0) return ETS_OK;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int64_t size = size_of(dtype);
  const uint32_t row = static_cast<uint32_t>(D * size / 16);
  const int64_t step = (static_cast<int64_t>(1) << 30) / (static_cast<int64_t>(row) * H);
  auto s = static_cast<hipStream_t>(stream);
  for (int64_t n = 0; n < N; n += step) {
    const int64_t count = N - n < step ? N - n : step;
    CacheParams p{};
    p.out = static_cast<char*>(out) + n * H * D * size;
    p.slots = slots + n;
    p.stream = N * H * D * size > kStream;
    p.codes = const_cast<uint8_t*>(codes), p.codes_s = codes_s, p.codes_h = codes_h;
    p.scales = const_cast<uint8_t*>(scales), p.scales_s = scales_s, p.scales_h = scales_h, p.S = S;
    p.items = static_cast<uint32_t>(count * H * row);
    p.by_row = fast_div(row);
    p.by_heads = fast_div(H);
    const uint32_t grid = (p.items + kReadBatch * kThreads - 1) / (kReadBatch * kThreads);
    if (dtype == ETS_BF16) {
      hipLaunchKernelGGL(cache_read_kernel<__bf16>, dim3(grid), dim3(kThreads), 0, s, p);
    } else if (dtype == ETS_FP16) {
      hipLaunchKernelGGL(cache_read_kernel<_Float16>, dim3(grid), dim3(kThreads), 0, s, p);
    } else {
      hipLaunchKernelGGL(cache_read_kernel<float>, dim3(grid), dim3(kThreads), 0, s, p);
    }
    if (hipGetLastError() != hipSuccess) return ETS_ERR_HIP;
  }
  return ETS_OK;
}

}  // extern "C"
