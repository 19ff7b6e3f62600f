// ets_block_cache.hip -- the writes of an 8-bit cache with one power-of-two
// scale for a block of tokens and a head (gfx950).
#include "ets_speculate.h"

#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kKept = 8;  // vectors of 8 values that a lane keeps between the two looks at them

struct BlockParams {
  const char* x;  // rows in (write)
  int64_t x_b, x_t, x_h;  // bytes
  int32_t B, T, H, D;
  uint8_t* codes;
  uint8_t* scales;
  int64_t codes_s, codes_h, scales_s, scales_h, pages;  // whole pages of the cache
  int32_t block, page_size;
  const int32_t* page_table;
  int64_t pt_b, capacity;  // positions of a table row
  const int32_t* first;
  const int32_t* counts;
  const int32_t* path;  // keep
  int64_t path_b;
  int32_t blocks;  // that a sequence's new rows may touch
  uint32_t group;  // the launch's first workgroup
  FastDiv by_blocks, by_heads, by_row;
};

// The smallest e in [kScaleLow, kScaleHigh] with top <= 448 * 2^e: top = m * 2^q
// with m in [1/2, 1) and 448 = 7/8 * 2^9, so e = q - 9 where m <= 7/8, else q - 8.
__device__ __forceinline__ int block_exponent(float top) {
  int q;
  const float m = frexpf(top, &q);
  const int e = top == 0.0f ? kScaleLow : m <= 0.875f ? q - 9 : q - 8;
  return min(max(e, kScaleLow), kScaleHigh);
}
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 <= e <= 127

// Eight values times a power of two as codes, limited to the format's range; no number stays none.
__device__ __forceinline__ u32v2 to_codes(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = x[j] * inv;
    y[j] = v != v ? v : fminf(fmaxf(v, -448.0f), 448.0f);
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  return u32v2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}
__device__ __forceinline__ void from_codes(u32v2 c, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c[j], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c[j], true);
    x[4 * j] = a[0], x[4 * j + 1] = a[1], x[4 * j + 2] = b[0], x[4 * j + 3] = b[1];
  }
}
__device__ __forceinline__ float largest(const float (&x)[8], float top) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float size = fabsf(x[j]);
    top = size < __builtin_inff() ? fmaxf(top, size) : top;
  }
  return top;
}

// The largest of a value over the workgroup, in all of its lanes.
template <int THREADS>
__device__ __forceinline__ float widest(float top, float* waves) {
#pragma unroll
  for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
  if (THREADS == 64) return top;
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = top;
  __syncthreads();
  top = waves[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) top = fmaxf(top, waves[w]);
  __syncthreads();  // the next use of `waves` comes behind every lane's look
  return top;
}

// First slot of the block that holds position `at`, or -1 where the position or its page is not there.
__device__ __forceinline__ int64_t block_slot(const BlockParams& p, int b, int64_t at) {
  if (at < 0 || at >= p.capacity) return -1;
  const uint32_t page = static_cast<uint32_t>(at) / static_cast<uint32_t>(p.page_size);  // capacity is under 2^31
  const int64_t number = p.page_table[b * p.pt_b + page];
  if (number < 0 || number >= p.pages) return -1;
  const int in = static_cast<int>(static_cast<uint32_t>(at) - page * static_cast<uint32_t>(p.page_size));
  return number * p.page_size + in / p.block * p.block;
}

// Brings a block's `stay` first rows to a larger exponent.
template <int THREADS>
__device__ __forceinline__ void raise_rows(const BlockParams& p, uint8_t* codes, int stay, int from, int to) {
  const float inv = power(max(from - to, -127));  // under 2^-19 every code rounds to zero
  const int row = p.D / 8, items = stay * row;
  for (int i = threadIdx.x; i < items; i += THREADS) {
    const uint32_t r = div_by(i, p.by_row), v = i - r * row;
    uint8_t* at = codes + r * p.codes_s + v * 8;
    float x[8];
    from_codes(load_any<u32v2>(at), x);
    store_any(at, to_codes(x, inv));
  }
}

// One workgroup takes the new rows of one block and head: they are looked at
// twice, for their largest magnitude and for their codes, and up to kKept
// vectors a lane (16384 values of 256 lanes) stay in registers between.  Up to
// 4096 values are one wave's, which waits at no barrier, and x is asked for
// before the page is known.
//
// Measured: 20 us for pieces of 8192 tokens of four prompts, 8 x 128, fp16,
// blocks of 32 (75 MB, 3.7 TB/s; 29 us with 256 lanes and the page first), in one
// turn of waves, each with three loads in turn; 4.6 us for 64 rows (the loads).
template <class T, int THREADS>
__global__ __launch_bounds__(THREADS) void block_write_kernel(BlockParams p) {
  typedef T V8 __attribute__((ext_vector_type(8)));
  __shared__ float waves[THREADS / 64];
  const uint32_t group = p.group + blockIdx.x, bj = div_by(group, p.by_heads), h = group - bj * p.H;
  const uint32_t b = div_by(bj, p.by_blocks), j = bj - b * p.blocks;
  const int rows = min(p.counts[b], p.T);
  const int64_t first = p.first[b], end = first + rows;
  const int64_t start = (first / p.block + j) * p.block;
  // a sequence without rows does not own the block that its next position stands in
  if (first < 0 || rows <= 0 || start >= end) return;
  const int64_t slot = block_slot(p, b, start);  // on its way while the rows are read
  const int64_t low = first > start ? first : start, high = end < start + p.block ? end : start + p.block;
  const int stay = static_cast<int>(low - start), count = static_cast<int>(high - low);
  const char* src = p.x + b * p.x_b + (low - first) * p.x_t + h * p.x_h;
  const int row = p.D / 8, items = count * row;
  auto value = [&](int i) {
    const uint32_t r = div_by(i, p.by_row), v = i - r * row;
    return load_any<V8>(src + r * p.x_t + v * (8 * sizeof(T)));
  };
  auto widen = [](const V8& in, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = static_cast<float>(in[k]);
  };

  V8 kept[kKept];
  float top = 0.0f;
#pragma unroll
  for (int u = 0; u < kKept; ++u) {
    const int i = threadIdx.x + u * THREADS;
    kept[u] = V8{};
    if (i < items) kept[u] = value(i);
  }
  if (slot < 0) return;
  uint8_t* codes = p.codes + slot * p.codes_s + h * p.codes_h;
  uint8_t* scale = p.scales + slot / p.block * p.scales_s + h * p.scales_h;
#pragma unroll
  for (int u = 0; u < kKept; ++u) {
    float x[8];
    widen(kept[u], x);
    top = largest(x, top);
  }
  for (int i = threadIdx.x + kKept * THREADS; i < items; i += THREADS) {
    float x[8];
    widen(value(i), x);
    top = largest(x, top);
  }
  const int before = stay ? static_cast<int>(*scale) - kScaleBias : kScaleLow;
  const int e = max(block_exponent(widest<THREADS>(top, waves)), before);  // the scale is read before the barriers, written behind them
  const float inv = power(max(-e, -127));
  if (stay && e > before) raise_rows<THREADS>(p, codes, stay, before, e);
  if (threadIdx.x == 0) *scale = static_cast<uint8_t>(e + kScaleBias);
  codes += stay * p.codes_s;
  auto put = [&](int i, const V8& in) {
    const uint32_t r = div_by(i, p.by_row), v = i - r * row;
    float x[8];
    widen(in, x);
    store_any(codes + r * p.codes_s + v * 8, to_codes(x, inv));
  };
#pragma unroll
  for (int u = 0; u < kKept; ++u) {
    const int i = threadIdx.x + u * THREADS;
    if (i < items) put(i, kept[u]);
  }
  for (int i = threadIdx.x + kKept * THREADS; i < items; i += THREADS) put(i, value(i));
}

// One workgroup takes one sequence and head: the rows that move come into LDS
// with their scales (64 rows of 256 codes at most), and go out block by block.
// 7 us for 64 trees of 40, 8 x 128: five loads in turn and the barriers.
__global__ __launch_bounds__(kThreads) void block_keep_kernel(BlockParams p) {
  __shared__ float waves[kThreads / 64];
  __shared__ __align__(16) u32v2 rows[ETS_MAX_TREE * ETS_MAX_BLOCK_DIM / 8];
  __shared__ int exponent[ETS_MAX_TREE];
  __shared__ int64_t source[ETS_MAX_TREE];
  const uint32_t group = p.group + blockIdx.x, b = div_by(group, p.by_heads), h = group - b * p.H;
  const int64_t first = p.first[b];
  const int count = min(p.counts[b], p.T), lane = threadIdx.x & 63;
  if (first < 0 || count <= 0) return;
  // every wave looks at the line for itself; the first one writes down what all need
  const int step = lane < count ? p.path[b * p.path_b + lane] : -1;
  const uint64_t moves = __ballot(lane < count && step != lane);
  if (!moves) return;
  const int same = __builtin_ctzll(moves);  // rows that stay where they are
  if (threadIdx.x < static_cast<uint32_t>(count)) {
    int64_t slot = -1;
    if (step >= 0 && step < p.T) {
      const int64_t at = first + step;
      slot = block_slot(p, b, at);
      if (slot >= 0) slot += at % p.block;  // blocks divide pages
    }
    source[lane] = slot;
    exponent[lane] = slot < 0 ? 0 : static_cast<int>(p.scales[slot / p.block * p.scales_s + h * p.scales_h]) - kScaleBias;
  }
  __syncthreads();
  const int row = p.D / 8;
  for (int i = threadIdx.x; i < (count - same) * row; i += kThreads) {
    const uint32_t r = div_by(i, p.by_row), v = i - r * row;
    const int64_t slot = source[same + r];
    rows[i] = slot < 0 ? u32v2{0, 0} : load_any<u32v2>(p.codes + slot * p.codes_s + h * p.codes_h + v * 8);
  }
  __syncthreads();
  const int64_t begin = first + same, end = first + count;
  for (int64_t start = begin / p.block * p.block; start < end; start += p.block) {
    const int64_t low = begin > start ? begin : start, high = end < start + p.block ? end : start + p.block;
    const int64_t slot = block_slot(p, b, start);
    if (slot < 0) continue;
    const int stay = static_cast<int>(low - start), items = static_cast<int>(high - low) * row;
    const int at = static_cast<int>(low - begin);  // of the rows that move
    uint8_t* codes = p.codes + slot * p.codes_s + h * p.codes_h;
    uint8_t* scale = p.scales + slot / p.block * p.scales_s + h * p.scales_h;
    float top = 0.0f;
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const uint32_t r = div_by(i, p.by_row);
      float x[8];
      from_codes(rows[at * row + i], x);
      // scales of 2^119 and codes of 448 end just under infinity
      top = fmaxf(top, ldexpf(largest(x, 0.0f), exponent[same + at + r]));
    }
    const int before = stay ? static_cast<int>(*scale) - kScaleBias : kScaleLow;
    const int e = max(block_exponent(widest<kThreads>(top, waves)), before);
    if (stay && e > before) raise_rows<kThreads>(p, codes, stay, before, e);
    if (threadIdx.x == 0) *scale = static_cast<uint8_t>(e + kScaleBias);
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const uint32_t r = div_by(i, p.by_row), v = i - r * row;
      float x[8];
      from_codes(rows[at * row + i], x);
      // the new exponent may lie far under or above the old one: a row of zeros or of small codes under a large scale
      const int up = min(max(exponent[same + at + r] - e, -127), 127);
      store_any(codes + (stay + r) * p.codes_s + v * 8, to_codes(x, power(up)));
    }
  }
}

ets_status block_params(BlockParams* p, int32_t B, int32_t T, int32_t H, int32_t D, uint8_t* codes, int64_t codes_s, int64_t codes_h,
                        uint8_t* scales, int64_t scales_s, int64_t scales_h, int64_t S, int32_t block, const int32_t* page_table,
                        int64_t pt_b, int32_t table_pages, int32_t page_size, const int32_t* first, const int32_t* counts) {
  if (B < 0 || T < 0 || H < 1 || D < kCacheBlock || D % kCacheBlock || D > ETS_MAX_BLOCK_DIM || S < 0 || S > INT32_MAX)
    return ETS_ERR_INVALID_ARG;
  if (block < 1 || page_size < 1 || page_size % block || S % block || table_pages < 0) return ETS_ERR_INVALID_ARG;
  if (static_cast<int64_t>(H) * D > (1 << 28) || static_cast<int64_t>(B) * H > INT32_MAX) return ETS_ERR_INVALID_ARG;
  if (static_cast<int64_t>(table_pages) * page_size > ETS_MAX_LENGTH) return ETS_ERR_INVALID_ARG;
  if (B && T && ((S && (!codes || !scales)) || !first || !counts || (table_pages && !page_table))) return ETS_ERR_INVALID_ARG;
  *p = BlockParams{};
  p->B = B, p->T = T, p->H = H, p->D = D;
  p->codes = codes, p->codes_s = codes_s, p->codes_h = codes_h;
  p->scales = scales, p->scales_s = scales_s, p->scales_h = scales_h;
  p->pages = S / page_size, p->block = block, p->page_size = page_size;
  p->page_table = page_table, p->pt_b = pt_b, p->capacity = static_cast<int64_t>(table_pages) * page_size;
  p->first = first, p->counts = counts;
  p->by_heads = fast_div(H);
  p->by_row = fast_div(D / 8);
  return ETS_OK;
}

template <class T>
void launch_write(BlockParams p, int64_t groups, bool narrow, hipStream_t s) {
  launch_in_turn(groups, narrow ? 64 : kThreads, [&](uint32_t first, uint32_t grid) {
    p.group = first;
    if (narrow) {
      hipLaunchKernelGGL((block_write_kernel<T, 64>), dim3(grid), dim3(64), 0, s, p);
    } else {
      hipLaunchKernelGGL((block_write_kernel<T, kThreads>), dim3(grid), dim3(kThreads), 0, s, p);
    }
  });
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_block_write(const void* x, int64_t x_b, int64_t x_t, int64_t x_h, int32_t B, int32_t T, int32_t H, int32_t D,
                           uint8_t* codes, int64_t codes_s, int64_t codes_h, uint8_t* scales, int64_t scales_s, int64_t scales_h,
                           int64_t S, int32_t block, const int32_t* page_table, int64_t pt_b, int32_t table_pages, int32_t page_size,
                           const int32_t* first, const int32_t* counts, int32_t dtype, void* stream) {
  using namespace ets;
  if (!dtype_known(dtype)) return ETS_ERR_INVALID_ARG;
  BlockParams p;
  if (ets_status st = block_params(&p, B, T, H, D, codes, codes_s, codes_h, scales, scales_s, scales_h, S, block, page_table, pt_b,
                                   table_pages, page_size, first, counts);
      st != ETS_OK)
    return st;
  if (B == 0 || T == 0 || p.pages == 0) return ETS_OK;
  if (!x) return ETS_ERR_INVALID_ARG;
  // rows of one block and head are numbered in 32 bits, vector by vector
  const int64_t most = block < T ? block : T;
  if (most * (D / 8) > INT32_MAX / 2) return ETS_ERR_INVALID_ARG;
  const int64_t touched = (static_cast<int64_t>(T) + block - 2) / block + 1, within = (p.capacity + block - 1) / block;
  const int64_t blocks = touched < within ? touched : within;  // no more than a table row has
  if (blocks == 0) return ETS_OK;
  const int64_t grid = blocks * B * H;
  if (grid > INT32_MAX) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int64_t size = dtype == ETS_FP32 ? 4 : 2;
  p.x = static_cast<const char*>(x), p.x_b = x_b * size, p.x_t = x_t * size, p.x_h = x_h * size;
  p.blocks = static_cast<int32_t>(blocks);
  p.by_blocks = fast_div(p.blocks);
  // a wave alone has no barrier to wait at, and holds what a step brings
  const bool narrow = most * D <= 64 * 8 * kKept;
  auto s = static_cast<hipStream_t>(stream);
  if (dtype == ETS_BF16) {
    launch_write<__bf16>(p, grid, narrow, s);
  } else if (dtype == ETS_FP16) {
    launch_write<_Float16>(p, grid, narrow, s);
  } else {
    launch_write<float>(p, grid, narrow, s);
  }
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

ets_status ets_block_keep(int32_t B, int32_t T, int32_t H, int32_t D, uint8_t* codes, int64_t codes_s, int64_t codes_h, uint8_t* scales,
                          int64_t scales_s, int64_t scales_h, int64_t S, int32_t block, const int32_t* page_table, int64_t pt_b,
                          int32_t table_pages, int32_t page_size, const int32_t* first, const int32_t* path, int64_t path_b,
                          const int32_t* counts, void* stream) {
  using namespace ets;
  if (T > ETS_MAX_TREE) return ETS_ERR_INVALID_ARG;
  BlockParams p;
  if (ets_status st = block_params(&p, B, T, H, D, codes, codes_s, codes_h, scales, scales_s, scales_h, S, block, page_table, pt_b,
                                   table_pages, page_size, first, counts);
      st != ETS_OK)
    return st;
  if (B == 0 || T == 0 || p.pages == 0) return ETS_OK;
  if (!path) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  p.path = path, p.path_b = path_b;
  launch_in_turn(static_cast<int64_t>(B) * H, kThreads, [&](uint32_t first_group, uint32_t grid) {
    p.group = first_group;
    hipLaunchKernelGGL(block_keep_kernel, dim3(grid), dim3(kThreads), 0, static_cast<hipStream_t>(stream), p);
  });
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"
