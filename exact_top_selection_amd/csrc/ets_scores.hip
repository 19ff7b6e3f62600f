// ets_scores.hip -- the indexer scores that the selection ranks (gfx950):
//   I[t][p] = sum_h w[t][h] max(0, q[t][h] . k[p])
// over a paged 8-bit cache, for one or several tokens a sequence.
#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kSub = 2;             // 16-key tiles of a wave's step
constexpr int kTile = 16 * kSub;    // keys of a wave's step, held in registers
constexpr int kUnit = 128;          // keys by which the work is dealt out: a step of all waves
constexpr int kPiece = 2048;        // keys of a workgroup between barriers
constexpr int kFill = 1024;         // positions past a length that are filled at a time
static_assert(ETS_MAX_LENGTH <= INT32_MAX - kPiece, "positions are 32-bit numbers, and stand up to a piece behind a length");
constexpr int kQueryBytes = 65536;  // queries that a workgroup keeps in LDS
constexpr float kNegInf = -__builtin_inff();

struct ScoreParams {
  const char* q;
  int64_t q_b, q_t, q_h;  // bytes
  const float* w;
  int64_t w_b, w_t;
  int B, T, H, D, L;
  int tokens, head_tiles;  // tokens of a workgroup; 16-row tiles of a token
  const uint8_t* codes;
  const uint8_t* scales;
  uint32_t codes_s, scales_s;
  int64_t S;
  const int32_t* table;
  int64_t pt_b;
  const int32_t* lens;
  FastDiv by_page, by_fills, by_head_tiles;
  float* out;
  int64_t out_stride;
};

// The keys stay, the queries stream: a wave brings 32 keys from global memory
// straight into matrix operands (lane l holds 16 consecutive codes of key l %
// 16 for every 64 channels; the order of the channels inside a product is
// free, and the queries are laid out in LDS in the same one), then takes the
// 16-row query tiles from LDS one by one, each feeding 2 * D / 32 matrix
// instructions (64 keys a step halve the LDS reads, but leave three waves a
// SIMD in the place of four: 60 us against 58).  Rows of the result are heads,
// columns keys, so the weighted sum over heads runs down a lane's registers
// and over four lanes at the end.
//
// The lengths are known on the device only.  All keys, in units of 128, are
// numbered through the batch and dealt out to the workgroups in equal runs: a
// grid by sequence and chunk left a quarter of it idle with lengths between L
// / 2 and L (67 us against 58).  FULL: D is 64 NP.
//
// Measured: 56 us for 64 sequences of up to 32768 positions, 64 heads of 128
// channels (218 MB, 3.9 TB/s, 460 TFLOP/s), 47 us for 4 tokens of each of 4
// sequences of up to 262144, 32 heads in fp16 (129 MB, 590 TFLOP/s; 1.5 of them
// for finding blocks that say nothing of a row's size).  Beyond the
// last-level cache a further 2^21 keys take 72 us with 1 head as with 64: it
// is bound by how fast half lines of rows come in (4 TB/s), and with few keys
// by three loads in turn (length, page, row), about 8 us before the first
// product.  Several tokens add matrix and vector instructions, which share
// the issue of a SIMD: a weighted sum is two vector instructions a product.
template <class T, int NP, bool FULL>
__global__ __launch_bounds__(kThreads, NP <= 2 ? 4 : NP == 3 ? 3 : 2) void scores_kernel(ScoreParams p) {
  typedef Mat<T> M;
  typedef typename M::V8 V8;
  extern __shared__ __align__(16) char lds[];
  const int tiles_max = p.tokens * p.head_tiles;
  V8* qs = reinterpret_cast<V8*>(lds);                                // [tile][pair][half][lane]
  float* ws = reinterpret_cast<float*>(lds + tiles_max * NP * 2048);  // [tile][16]
  int32_t* slots = reinterpret_cast<int32_t*>(ws + tiles_max * 16);   // [kPiece]
  float* held = reinterpret_cast<float*>(slots + kPiece);             // [wave][token][lane]
  __shared__ int64_t found[2 + kWaves];

  const int t0 = blockIdx.y * p.tokens;
  const int tokens = min(p.tokens, p.T - t0), tiles = tokens * p.head_tiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  auto length = [&](int b) { return min(max(p.lens[b], 0), p.L); };
  auto units = [&](int b) { return (length(b) + kUnit - 1) / kUnit; };

  // positions past the lengths
  for (int64_t i = blockIdx.x; i < static_cast<int64_t>(p.B) * p.by_fills.d; i += gridDim.x) {
    const int b = static_cast<int>(div_by(static_cast<uint32_t>(i), p.by_fills));
    const int from = static_cast<int>(i - static_cast<int64_t>(b) * p.by_fills.d) * kFill, n = length(b);
    const int to = min(from + kFill, p.L);
    if (n < to)
      for (int t = 0; t < tokens; ++t)
        for (int k = max(from, n) + threadIdx.x; k < to; k += kThreads)
          p.out[(static_cast<int64_t>(b) * p.T + t0 + t) * p.out_stride + k] = kNegInf;
  }

  // this workgroup's run of units: lane i counts sequences i * each ..; the one in whose count the run starts says where
  const int each = (p.B + kThreads - 1) / kThreads, b0 = static_cast<int>(threadIdx.x) * each;
  int64_t mine = 0;
  for (int b = b0; b < min(b0 + each, p.B); ++b) mine += units(b);
  int64_t upto = mine;  // through this lane
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t x = __shfl_up(upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 63) found[2 + wave] = upto;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) upto += found[2 + w];
    all += found[2 + w];
  }
  const int64_t run = (all + gridDim.x - 1) / gridDim.x, start = run * blockIdx.x;
  if (start >= all) return;
  if (start >= upto - mine && start < upto) {
    int64_t left = start - (upto - mine);
    int b = b0;
    for (int u = units(b); left >= u; u = units(b)) left -= u, ++b;
    found[0] = b, found[1] = left;
  }
  __syncthreads();
  int b = __builtin_amdgcn_readfirstlane(static_cast<int>(found[0])), k0 = __builtin_amdgcn_readfirstlane(static_cast<int>(found[1])) * kUnit;
  int64_t todo = all - start < run ? all - start : run;

  // a step's rows on their way: lane (key col of each 16, row g) brings codes 64 i + 16 g .. + 15 and their scale
  // byte; rows and channels that are not there come from kNothing, without a branch
  typedef RowScales<NP, FULL> KS;
  const uint64_t nothing = reinterpret_cast<uint64_t>(&kNothing[0]);
  const uint64_t kc = reinterpret_cast<uint64_t>(p.codes) + 16 * g, ks = KS::start(reinterpret_cast<uint64_t>(p.scales), g);
  u32v4 raw[kSub][NP];
  uint32_t byte[kSub][KS::n];
  auto fetch = [&](int k) {
    int32_t slot[kSub];
#pragma unroll
    for (int s = 0; s < kSub; ++s) slot[s] = slots[min(k, kPiece - kTile) + 16 * s + col];
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      const bool there = slot[s] >= 0 && k < kPiece;
      const uint64_t at = static_cast<uint32_t>(slot[s]), c0 = kc + at * p.codes_s, b0 = ks + at * p.scales_s;
      const uint64_t c1 = there ? c0 : nothing, b1 = there ? b0 : nothing;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const bool in = FULL || 64 * i + 16 * g < p.D;
        const uint64_t c = c1 + 64 * i;
        raw[s][i] = load_global<u32v4>(in ? c : nothing);
      }
      KS::load(byte[s], b1, nothing, [&](int i) { return 64 * i + 16 * g < p.D; });
    }
  };

  for (bool new_b = true; todo > 0;) {
    const int n = length(b);
    if (k0 >= n) {
      ++b, k0 = 0, new_b = true;
      continue;
    }
    const int keys = min(static_cast<int>(min(todo * kUnit, static_cast<int64_t>(kPiece))), n - k0);
    __syncthreads();  // the piece before has been read
    // all of a lane's loads first: one wait in the place of eight (four for the queries)
    constexpr int kEach = kPiece / kThreads;
    int32_t page_id[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = min(k0 + static_cast<int>(threadIdx.x) + i * kThreads, n - 1);  // past the piece's keys: any page of its, not used
      page_id[i] = p.table[b * p.pt_b + div_by(j, p.by_page)];
    }
    if (new_b) {
      constexpr int kQueries = 4;
      for (int base = threadIdx.x; base < tiles * NP * 128; base += kQueries * kThreads) {
        V8 v[kQueries];
#pragma unroll
        for (int u = 0; u < kQueries; ++u) {
          const int i = base + u * kThreads, l = i & 63, half = (i >> 6) & 1, tp = i >> 7;
          const int tile = tp / NP, pair = tp - tile * NP, t = static_cast<int>(div_by(tile, p.by_head_tiles));
          const int h = (tile - t * p.head_tiles) * 16 + (l & 15), d = 64 * pair + 16 * (l >> 4) + 8 * half;
          v[u] = V8{};
          if (tile < tiles && h < p.H && d < p.D)
            v[u] = load_any<V8>(p.q + b * p.q_b + (t0 + t) * p.q_t + h * p.q_h + static_cast<int64_t>(d) * 2);
        }
#pragma unroll
        for (int u = 0; u < kQueries; ++u)
          if (base + u * kThreads < tiles * NP * 128) qs[base + u * kThreads] = v[u];
      }
      for (int i = threadIdx.x; i < tiles * 16; i += kThreads) {
        const int t = static_cast<int>(div_by(i >> 4, p.by_head_tiles)), h = i - t * p.head_tiles * 16;
        ws[i] = h < p.H ? p.w[b * p.w_b + (t0 + t) * p.w_t + h] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = static_cast<int>(threadIdx.x) + i * kThreads, j = min(k0 + at, n - 1);
      const int64_t s = static_cast<int64_t>(page_id[i]) * p.by_page.d + (j - div_by(j, p.by_page) * p.by_page.d);
      slots[at] = at < keys && s >= 0 && s < p.S ? static_cast<int32_t>(s) : -1;
    }
    new_b = false;
    __syncthreads();

  int k = wave * kTile;
  fetch(k);
  hold(byte);  // else the loop carries 8-bit values and widens them as soon as they are loaded
  // Sums leave a step later, before the next rows are asked for: a store behind them would be waited for with them.
  float* own = held + wave * p.tokens * 64 + lane;
  float* out = p.out + (static_cast<int64_t>(b) * p.T + t0) * p.out_stride + k0;
  auto leave = [&](int at) {
    const int key = at + 16 * (lane >> 5) + col;
    if (at >= 0 && key < keys && !(g & 1))
      for (int t = 0; t < tokens; ++t) out[t * p.out_stride + key] = own[t * 64];
  };
  for (; k < keys; k += kWaves * kTile) {
    V8 key[kSub][NP][2];
    uint32_t top[kSub];
    hold(raw), hold(byte);
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      top[s] = 0;
      if constexpr (M::kRowScale) top[s] = row_top<NP, FULL>(byte[s], raw[s], g);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float f = M::scale(KS::byte(byte[s], i, g), top[s]);
        key[s][i][0] = M::keys(raw[s][i][0], raw[s][i][1], f);
        key[s][i][1] = M::keys(raw[s][i][2], raw[s][i][3], f);
      }
    }
    leave(k - kWaves * kTile);
    fetch(k + kWaves * kTile);
    const bool seen = slots[k + 16 * (lane >> 5) + col] >= 0;
    float size = 1.0f;
    if (M::kRowScale) size = __uint_as_float((lane < 32 ? top[0] : top[1]) << 23);
    int tile = 0;
    for (int t = 0; t < tokens; ++t) {
      float part[kSub] = {};
      for (int i = 0; i < p.head_tiles; ++i, ++tile) {
        f32x4 acc[kSub] = {};
#pragma unroll
        for (int j = 0; j < NP; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const V8 q = qs[((tile * NP + j) * 2 + h) * 64 + lane];
#pragma unroll
            for (int s = 0; s < kSub; ++s) acc[s] = M::mma(q, key[s][j][h], acc[s]);
          }
        }
        const f32x4 w = *reinterpret_cast<const f32x4*>(ws + tile * 16 + 4 * g);
#pragma unroll
        for (int s = 0; s < kSub; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            part[s] = fmaf(w[e], __builtin_elementwise_maximum(acc[s][e], 0.0f), part[s]);
      }
      // over the four lanes of a key: key col of the first half in lanes 0 to 31, of the second in the others
      const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(part[0]), __float_as_uint(part[1]), false, false);
      const uint32_t x = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
      const auto c = __builtin_amdgcn_permlane16_swap(x, x, false, false);
      const float sum = (__uint_as_float(c[0]) + __uint_as_float(c[1])) * size;
      own[t * 64] = seen ? sum : kNegInf;
    }
  }
  leave(k - kWaves * kTile);
    todo -= (keys + kUnit - 1) / kUnit;
    k0 += keys;
  }
}

template <class T, int NP>
void launch_pairs(const ScoreParams& p, dim3 grid, size_t lds, hipStream_t s) {
  if (p.D == 64 * NP) {
    hipLaunchKernelGGL((scores_kernel<T, NP, true>), grid, dim3(kThreads), lds, s, p);
  } else {
    hipLaunchKernelGGL((scores_kernel<T, NP, false>), grid, dim3(kThreads), lds, s, p);
  }
}

template <class T>
void launch_scores(const ScoreParams& p, int np, dim3 grid, size_t lds, hipStream_t s) {
  if (np == 1) {
    launch_pairs<T, 1>(p, grid, lds, s);
  } else if (np == 2) {
    launch_pairs<T, 2>(p, grid, lds, s);
  } else if (np == 3) {
    launch_pairs<T, 3>(p, grid, lds, s);
  } else {
    launch_pairs<T, 4>(p, grid, lds, s);
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
  if (B < 0 || B > 65535 || T < 0 || H < 1 || H > ETS_MAX_INDEX_HEADS || D < kCacheBlock || D % kCacheBlock ||
      D > ETS_MAX_INDEX_DIM || S < 0 || S > INT32_MAX || page_size < 1 || L < 0 || L > ETS_MAX_LENGTH || out_stride < L ||
      (dtype != ETS_BF16 && dtype != ETS_FP16) ||
      codes_s < 0 || codes_s > UINT32_MAX || scales_s < 0 || scales_s > UINT32_MAX || static_cast<int64_t>(B) * ((static_cast<int64_t>(L) + kFill - 1) / kFill) > INT32_MAX)
    return ETS_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || L == 0) return ETS_OK;
  if (!q || !weights || !page_table || !seq_lens || !out || (S && (!codes || !scales))) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int np = (D + 63) / 64;
  ScoreParams p{};
  p.q = static_cast<const char*>(q), p.q_b = 2 * q_b, p.q_t = 2 * q_t, p.q_h = 2 * q_h;
  p.w = weights, p.w_b = w_b, p.w_t = w_t;
  p.B = B, p.T = T, p.H = H, p.D = D, p.L = L;
  p.head_tiles = (H + 15) / 16;
  p.by_head_tiles = fast_div(p.head_tiles);
  const int room = kQueryBytes / (np * 2048) / p.head_tiles;
  p.tokens = T < room ? T : room;
  const int groups = (T + p.tokens - 1) / p.tokens;
  if (groups > 65535) return ETS_ERR_INVALID_ARG;
  p.codes = codes, p.codes_s = static_cast<uint32_t>(codes_s), p.scales = scales, p.scales_s = static_cast<uint32_t>(scales_s), p.S = S;
  p.table = page_table, p.pt_b = pt_b, p.lens = seq_lens;
  p.by_page = fast_div(page_size);
  p.out = out, p.out_stride = out_stride;
  p.by_fills = fast_div(static_cast<uint32_t>((static_cast<int64_t>(L) + kFill - 1) / kFill));
  // as many workgroups as the device holds at once (registers, LDS), over the groups of tokens
  const int tiles = p.tokens * p.head_tiles;
  const size_t lds = static_cast<size_t>(tiles) * np * 2048 + tiles * 64 + kPiece * 4 + p.tokens * kThreads * 4;
  const int64_t by_regs = np <= 2 ? 4 : np == 3 ? 3 : 2, by_lds = 160 * 1024 / (static_cast<int64_t>(lds) + 512);
  const int64_t most = (static_cast<int64_t>(L) + kUnit - 1) / kUnit * B;
  const int64_t fits = ((by_regs < by_lds ? by_regs : by_lds) * cu + groups - 1) / groups;
  const dim3 grid(static_cast<uint32_t>(most < fits ? most : fits), groups);
  auto s = static_cast<hipStream_t>(stream);
  if (dtype == ETS_BF16) {
    launch_scores<__bf16>(p, np, grid, lds, s);
  } else {
    launch_scores<_Float16>(p, np, grid, lds, s);
  }
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"
