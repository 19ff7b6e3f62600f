// ets_scores.hip -- the indexer scores that the selection ranks (gfx950):
//   I[t][p] = sum_h w[t][h] max(0, q[t][h] . k[p])
// over a paged 8-bit cache, for one or several tokens a sequence.
#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 64;           // keys of a wave's step, held in registers
constexpr int kChunkMax = 1024;     // keys of a workgroup
constexpr int kQueryBytes = 65536;  // queries that a workgroup keeps in LDS
constexpr float kNegInf = -__builtin_inff();

struct ScoreParams {
  const char* q;
  int64_t q_b, q_t, q_h;  // bytes
  const float* w;
  int64_t w_b, w_t;
  int T, H, D, L;
  int tokens, head_tiles;  // tokens of a workgroup; 16-row tiles of a token
  int chunk;               // keys of a workgroup
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t codes_s, scales_s, S;
  const int32_t* table;
  int64_t pt_b;
  const int32_t* lens;
  FastDiv by_page;
  float* out;
  int64_t out_stride;
};

// The keys stay, the queries stream: a wave brings 64 keys from global memory
// straight into matrix operands (lane l holds 16 consecutive codes of key l %
// 16 for every 64 channels; the order of the channels inside a product is
// free, and the queries are laid out in LDS in the same one), then takes the
// 16-row query tiles from LDS one by one, each feeding 4 * D / 32 matrix
// instructions.  Rows of the result are heads, columns keys, so the weighted
// sum over heads runs down a lane's registers and over four lanes at the end.
template <class T, int NP>
__global__ __launch_bounds__(kThreads, 2) void scores_kernel(ScoreParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  constexpr int W = (NP + 1) / 2;
  extern __shared__ __align__(16) char lds[];
  const int tiles_max = p.tokens * p.head_tiles;
  V8* qs = reinterpret_cast<V8*>(lds);                                      // [tile][pair][half][lane]
  float* ws = reinterpret_cast<float*>(lds + tiles_max * NP * 2048);        // [tile][16]
  int32_t* slots = reinterpret_cast<int32_t*>(ws + tiles_max * 16);         // [chunk]

  const int b = blockIdx.y, t0 = blockIdx.z * p.tokens;
  const int tokens = min(p.tokens, p.T - t0), tiles = tokens * p.head_tiles;
  const int k0 = static_cast<int>(blockIdx.x) * p.chunk, keys = min(p.chunk, p.L - k0);
  const int n = min(max(p.lens[b], 0), p.L);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;

  if (k0 >= n) {  // nothing but the padding
    for (int t = 0; t < tokens; ++t)
      for (int i = threadIdx.x; i < keys; i += kThreads)
        p.out[(static_cast<int64_t>(b) * p.T + t0 + t) * p.out_stride + k0 + i] = kNegInf;
    return;
  }

  for (int i = threadIdx.x; i < p.chunk; i += kThreads) {
    int32_t slot = -1;
    if (k0 + i < n) {
      const uint32_t page = div_by(k0 + i, p.by_page);
      const int64_t s = static_cast<int64_t>(p.table[b * p.pt_b + page]) * p.by_page.d + (k0 + i - page * p.by_page.d);
      slot = s >= 0 && s < p.S ? static_cast<int32_t>(s) : -1;
    }
    slots[i] = slot;
  }
  for (int i = threadIdx.x; i < tiles * NP * 128; i += kThreads) {
    const int l = i & 63, half = (i >> 6) & 1, tp = i >> 7;
    const int tile = tp / NP, pair = tp - tile * NP, t = tile / p.head_tiles;
    const int h = (tile - t * p.head_tiles) * 16 + (l & 15), d = 64 * pair + 16 * (l >> 4) + 8 * half;
    V8 v = {};
    if (h < p.H && d < p.D)
      v = load_any<V8>(p.q + b * p.q_b + (t0 + t) * p.q_t + h * p.q_h + static_cast<int64_t>(d) * 2);
    qs[i] = v;
  }
  for (int i = threadIdx.x; i < tiles * 16; i += kThreads) {
    const int t = (i >> 4) / p.head_tiles, h = i - t * p.head_tiles * 16;
    ws[i] = h < p.H ? p.w[b * p.w_b + (t0 + t) * p.w_t + h] : 0.0f;
  }
  __syncthreads();

  const int nb = p.D / kCacheBlock;
  u32v4 raw[4][NP];
  uint32_t sc[4][W];
  auto fetch = [&](int k) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int32_t slot = slots[k + 16 * s + col];
#pragma unroll
      for (int i = 0; i < NP; ++i) raw[s][i] = u32v4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < W; ++i) sc[s][i] = 0;
      if (slot >= 0) {
        const uint8_t* row = p.codes + slot * p.codes_s + 16 * g;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (64 * i + 16 * g < p.D) raw[s][i] = load_any<u32v4>(row + 64 * i);
        load_scales<W>(sc[s], p.scales + slot * p.scales_s, nb);
      }
    }
  };

  const int last = min(keys, n - k0);  // keys of the chunk that have a score
  int k = wave * kTile;
  if (k < last) fetch(k);
  for (; k < keys; k += kWaves * kTile) {
    float* out = p.out + (static_cast<int64_t>(b) * p.T + t0) * p.out_stride + k0 + k + lane;
    if (k >= last) {
      for (int t = 0; t < tokens; ++t)
        if (k + lane < keys) out[t * p.out_stride] = kNegInf;
      continue;
    }
    V8 key[4][NP][2];
    uint32_t top[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      top[s] = M::kRowScale ? scales_max<W>(sc[s]) : 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float f = M::scale(byte_of(sc[s][i / 2], 16 * (i & 1) + 8 * (g >> 1)), top[s]);
        key[s][i][0] = M::keys(raw[s][i][0], raw[s][i][1], f);
        key[s][i][1] = M::keys(raw[s][i][2], raw[s][i][3], f);
      }
    }
    if (k + kWaves * kTile < last) fetch(k + kWaves * kTile);
    const bool seen = slots[k + lane] >= 0;
    float size = 1.0f;
    if (M::kRowScale) {
      const uint32_t r = g == 0 ? top[0] : g == 1 ? top[1] : g == 2 ? top[2] : top[3];
      size = __uint_as_float(r << 23);
    }
    int tile = 0;
    for (int t = 0; t < tokens; ++t) {
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int i = 0; i < p.head_tiles; ++i, ++tile) {
        f32x4 acc[4] = {};
#pragma unroll
        for (int j = 0; j < NP; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const V8 q = qs[((tile * NP + j) * 2 + h) * 64 + lane];
#pragma unroll
            for (int s = 0; s < 4; ++s) acc[s] = M::mma(q, key[s][j][h], acc[s]);
          }
        }
        const f32x4 w = *reinterpret_cast<const f32x4*>(ws + tile * 16 + 4 * g);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            part[s] = fmaf(w[e], __builtin_elementwise_maximum(acc[s][e], 0.0f), part[s]);
      }
      // over the four lanes of a key, leaving key 16 s + col in the lanes of row s
      const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(part[0]), __float_as_uint(part[2]), false, false);
      const auto c = __builtin_amdgcn_permlane32_swap(__float_as_uint(part[1]), __float_as_uint(part[3]), false, false);
      const float x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
      const float y = __uint_as_float(c[0]) + __uint_as_float(c[1]);
      const auto e = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
      const float sum = (__uint_as_float(e[0]) + __uint_as_float(e[1])) * size;
      if (k + lane < keys) out[t * p.out_stride] = seen ? sum : kNegInf;
    }
  }
}

template <class T>
void launch_scores(const ScoreParams& p, int np, dim3 grid, size_t lds, hipStream_t s) {
  if (np == 1) {
    hipLaunchKernelGGL((scores_kernel<T, 1>), grid, dim3(kThreads), lds, s, p);
  } else if (np == 2) {
    hipLaunchKernelGGL((scores_kernel<T, 2>), grid, dim3(kThreads), lds, s, p);
  } else if (np == 3) {
    hipLaunchKernelGGL((scores_kernel<T, 3>), grid, dim3(kThreads), lds, s, p);
  } else {
    hipLaunchKernelGGL((scores_kernel<T, 4>), grid, dim3(kThreads), lds, s, p);
  }
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_index_scores(const void* q, int64_t q_b, int64_t q_t, int64_t q_h, const float* weights,
                            int64_t w_b, int64_t w_t, int32_t B, int32_t T, int32_t H, int32_t D,
                            const uint8_t* codes, int64_t codes_s, const uint8_t* scales,
                            int64_t scales_s, int64_t S, const int32_t* page_table, int64_t pt_b,
                            const int32_t* seq_lens, int32_t page_size, int32_t L, float* out,
                            int64_t out_stride, int32_t dtype, void* stream) {
  using namespace ets;
  if (B < 0 || T < 0 || H < 1 || H > ETS_MAX_INDEX_HEADS || D < kCacheBlock || D % kCacheBlock ||
      D > ETS_MAX_INDEX_DIM || S < 0 || S > INT32_MAX || page_size < 1 || L < 0 || out_stride < L ||
      (dtype != ETS_BF16 && dtype != ETS_FP16) || B > 65535)
    return ETS_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || L == 0) return ETS_OK;
  if (!q || !weights || !page_table || !seq_lens || !out || (S && (!codes || !scales))) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int np = (D + 63) / 64;
  ScoreParams p{};
  p.q = static_cast<const char*>(q), p.q_b = 2 * q_b, p.q_t = 2 * q_t, p.q_h = 2 * q_h;
  p.w = weights, p.w_b = w_b, p.w_t = w_t;
  p.T = T, p.H = H, p.D = D, p.L = L;
  p.head_tiles = (H + 15) / 16;
  const int room = kQueryBytes / (np * 2048) / p.head_tiles;
  p.tokens = T < room ? T : room;
  const int groups = (T + p.tokens - 1) / p.tokens;
  if (groups > 65535) return ETS_ERR_INVALID_ARG;
  p.codes = codes, p.codes_s = codes_s, p.scales = scales, p.scales_s = scales_s, p.S = S;
  p.table = page_table, p.pt_b = pt_b, p.lens = seq_lens;
  p.by_page = fast_div(page_size);
  p.out = out, p.out_stride = out_stride;
  p.chunk = kChunkMax;
  while (p.chunk > kWaves * kTile && (static_cast<int64_t>(L) + p.chunk - 1) / p.chunk * B * groups < 8 * cu) p.chunk /= 2;
  const int tiles = p.tokens * p.head_tiles;
  const size_t lds = static_cast<size_t>(tiles) * np * 2048 + tiles * 64 + p.chunk * 4;
  const dim3 grid((static_cast<int64_t>(L) + p.chunk - 1) / p.chunk, B, groups);
  auto s = static_cast<hipStream_t>(stream);
  if (dtype == ETS_BF16) {
    launch_scores<__bf16>(p, np, grid, lds, s);
  } else {
    launch_scores<_Float16>(p, np, grid, lds, s);
  }
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"
