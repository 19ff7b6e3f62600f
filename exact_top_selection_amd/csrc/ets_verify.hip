// ets_verify.hip -- which drafted tokens stand, and the token that follows
// (gfx950).
#include "ets_speculate.h"

#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 16;                  // values of a lane
constexpr int kChunk = kThreads * kEach;   // whose sums are kept
constexpr int kPerUnit = 4;                // workgroups of a compute unit

// What the walk over a sequence's nodes leaves.
struct Walk {
  int32_t node;     // where it ended
  int32_t count;    // nodes on the line; 0: an empty sequence
  uint64_t kids;    // drafted tokens that were refused there
};

struct VerifyParams {
  const char* probs;
  const char* draft;
  int64_t p_b, p_t, q_b, q_t;  // bytes
  int32_t B, T, V, chunks;
  int32_t each, groups;  // chunks of a workgroup, workgroups of a sequence
  uint32_t group;        // the launch's first workgroup
  const int32_t* tokens;
  int64_t tok_b;
  const float* uniform;
  int64_t u_b;
  const int64_t* mask;
  int64_t mask_b;
  const int32_t* lens;
  int32_t* out_tokens;
  int32_t* out_path;
  int32_t* out_counts;
  f64x2* sums;  // [B][chunks]: of the last draw's weights, of the target's
  Walk* walks;  // [B]
  FastDiv by_groups;
};

// A probability in 64 bits; negative ones, infinities and no numbers count as 0.
template <class T>
__device__ __forceinline__ double clean(T x) {
  const float v = static_cast<float>(x);
  return v > 0.0f && v < __builtin_inff() ? static_cast<double>(v) : 0.0;
}
__device__ __forceinline__ int lane_int(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ double lane_double(double x, int lane) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(bits), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(bits >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// One wave walks a sequence's line: lane t stands for node t and brings what its
// test needs at once; the walk then goes from child to child in registers.
template <class T>
__device__ __forceinline__ Walk walk(const VerifyParams& p, int b, uint64_t* line) {
  const int lane = threadIdx.x & 63;
  const int n = p.lens ? min(p.lens[b], p.T) : p.T;
  Walk w = {0, 0, 0};
  *line = 0;
  if (n <= 0) return w;
  const bool live = lane > 0 && lane < n;
  int parent = -1, token = -1;
  double target = 0.0, draft = 1.0, u = 0.0;
  if (live) {
    const uint64_t above = p.mask ? static_cast<uint64_t>(p.mask[b * p.mask_b + lane]) & ((1ull << lane) - 1) : 1ull << (lane - 1);
    parent = above ? 63 - __builtin_clzll(above) : -1;
    token = p.tokens[b * p.tok_b + lane];
    u = static_cast<double>(p.uniform[b * p.u_b + lane]);
    if (parent >= 0 && token >= 0 && token < p.V) {
      target = clean(load_any<T>(p.probs + b * p.p_b + parent * p.p_t + token * static_cast<int64_t>(sizeof(T))));
      if (p.draft) draft = clean(load_any<T>(p.draft + b * p.q_b + (lane - 1) * p.q_t + token * static_cast<int64_t>(sizeof(T))));
    } else if (p.draft) {
      draft = 0.0;
    }
  }
  uint64_t taken = 1;
  w.count = 1;
  for (;;) {
    const uint64_t kids = __ballot(live && parent == w.node);
    double rest = 1.0;
    int next = -1;
    for (uint64_t left = kids; left;) {
      const int c = __builtin_ctzll(left);
      left &= left - 1;
      const int x = lane_int(token, c);
      // a token that an earlier child had has nothing left
      const bool again = __ballot(live && token == x) & kids & ((1ull << c) - 1);
      const double share = again ? 0.0 : lane_double(target, c);
      if (lane_double(u, c) * (p.draft ? lane_double(draft, c) : rest) < share) {
        next = c;
        break;
      }
      rest -= share;
    }
    if (next < 0) {
      w.kids = kids;
      break;
    }
    w.node = next;
    ++w.count;
    taken |= 1ull << next;
  }
  *line = taken;
  return w;
}

// Tokens of refused children that lie in a chunk, as bits in LDS (where drafts have no probabilities).
__device__ __forceinline__ void mark_refused(const VerifyParams& p, int b, uint64_t kids, int base, uint32_t* bits) {
  for (int i = threadIdx.x; i < kChunk / 32; i += kThreads) bits[i] = 0;
  __syncthreads();
  if (threadIdx.x < 64 && (kids >> threadIdx.x & 1)) {
    const int64_t at = static_cast<int64_t>(p.tokens[b * p.tok_b + threadIdx.x]) - base;
    if (at >= 0 && at < kChunk) atomicOr(&bits[at >> 5], 1u << (at & 31));
  }
  __syncthreads();
}

// Weights of a lane's values base + 16 t .. + 15: of the last draw, and the target's own.
template <class T>
__device__ __forceinline__ void weights(const VerifyParams& p, int b, const Walk& w, int base, const uint32_t* refused,
                                        double (&last)[kEach], double (&whole)[kEach]) {
  const int first = base + static_cast<int>(threadIdx.x) * kEach;
  const char* target = p.probs + b * p.p_b + w.node * p.p_t;
  const char* draft = p.draft + b * p.q_b + w.node * p.q_t;
  const bool residue = p.draft && w.kids;
  T x[kEach], y[kEach];
  if (first + kEach <= p.V) {
    typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
    constexpr int n = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kEach / n; ++i) {
      const V v = load_any<V>(target + (first + i * n) * static_cast<int64_t>(sizeof(T)));
#pragma unroll
      for (int j = 0; j < n; ++j) x[i * n + j] = v[j];
    }
    if (residue) {
#pragma unroll
      for (int i = 0; i < kEach / n; ++i) {
        const V v = load_any<V>(draft + (first + i * n) * static_cast<int64_t>(sizeof(T)));
#pragma unroll
        for (int j = 0; j < n; ++j) y[i * n + j] = v[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      x[j] = y[j] = static_cast<T>(0.0f);
      if (first + j < p.V) {
        x[j] = load_any<T>(target + (first + j) * static_cast<int64_t>(sizeof(T)));
        if (residue) y[j] = load_any<T>(draft + (first + j) * static_cast<int64_t>(sizeof(T)));
      }
    }
  }
  const uint32_t gone = p.draft ? 0 : refused[threadIdx.x >> 1] >> (16 * (threadIdx.x & 1));
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    whole[j] = clean(x[j]);
    last[j] = whole[j];
    if (residue) {
      const double d = whole[j] - clean(y[j]);
      last[j] = d > 0.0 ? d : 0.0;
    }
    if (gone >> j & 1) last[j] = 0.0;
  }
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int i = 1; i < 64; i *= 2) x += __shfl_xor(x, i);
  return x;
}

// Sums of the last draw's weights, chunk by chunk; a workgroup takes a few chunks of one sequence, whose line it walks
// for itself (a launch of its own would cost more), and reads them side by side: lane t holds vectors t, t + 256, .. of
// a chunk.
//
// The walk is three loads in turn (line and tokens, probabilities, the row), so workgroups take as many chunks as leave
// about kPerUnit of them to a compute unit.
//
// Measured: 14 us for 64 sequences of 6 nodes over 128000 tokens with draft
// probabilities, fp32 (65 MB, 4.6 TB/s: the walk takes 4 of them); 6 us for 8 trees
// of 32 over 50001, bf16.
template <class T>
__global__ __launch_bounds__(kThreads) void weigh_kernel(VerifyParams p) {
  constexpr int n = 16 / sizeof(T), kVectors = kEach / n;
  typedef T V __attribute__((ext_vector_type(n)));
  __shared__ Walk shared;
  __shared__ uint32_t refused[kChunk / 32];
  __shared__ f64x2 part[2][kThreads / 64];
  const uint32_t at = p.group + blockIdx.x;
  const int b = static_cast<int>(div_by(at, p.by_groups)), group = static_cast<int>(at) - b * p.groups;
  const int first = group * p.each, end = min(first + p.each, p.chunks);
  if (threadIdx.x < 64) {
    uint64_t line;
    const Walk w = walk<T>(p, b, &line);
    if (threadIdx.x == 0) shared = w;
    if (group == 0) {
      if (threadIdx.x == 0) {
        p.walks[b] = w;
        p.out_counts[b] = w.count;
      }
      // lane i: the i-th node of the line, and the token behind it
      const int lane = threadIdx.x;
      if (lane < p.T) {
        uint64_t left = line;
        for (int i = 0; i < lane && left; ++i) left &= left - 1;
        const int node = left ? __builtin_ctzll(left) : -1;
        const uint64_t after = left & (left - 1);
        const int64_t to = static_cast<int64_t>(b) * p.T + lane;
        p.out_path[to] = node;
        p.out_tokens[to] = left && after ? p.tokens[b * p.tok_b + __builtin_ctzll(after)] : -1;
      }
    }
  }
  __syncthreads();
  const Walk w = shared;
  if (w.count == 0) return;
  const bool residue = p.draft && w.kids;
  const char* target = p.probs + b * p.p_b + w.node * p.p_t;
  const char* draft = p.draft + b * p.q_b + w.node * p.q_t;
  for (int chunk = first; chunk < end; ++chunk) {
    const int base = chunk * kChunk;
    const bool marks = !p.draft && w.kids;
    V x[kVectors], y[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int at = base + (i * kThreads + static_cast<int>(threadIdx.x)) * n;
      x[i] = y[i] = V{};
      if (at + n <= p.V) {
        x[i] = load_any<V>(target + at * static_cast<int64_t>(sizeof(T)));
        if (residue) y[i] = load_any<V>(draft + at * static_cast<int64_t>(sizeof(T)));
      } else {
#pragma unroll
        for (int j = 0; j < n; ++j) {
          if (at + j < p.V) {
            x[i][j] = load_any<T>(target + (at + j) * static_cast<int64_t>(sizeof(T)));
            if (residue) y[i][j] = load_any<T>(draft + (at + j) * static_cast<int64_t>(sizeof(T)));
          }
        }
      }
    }
    if (marks) mark_refused(p, b, w.kids, base, refused);
    double a = 0.0, c = 0.0;
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int in = (i * kThreads + static_cast<int>(threadIdx.x)) * n;
      const uint32_t gone = marks ? refused[in >> 5] >> (in & 31) : 0;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const double whole = clean(x[i][j]);
        double last = whole;
        if (residue) {
          const double d = whole - clean(y[i][j]);
          last = d > 0.0 ? d : 0.0;
        }
        if (gone >> j & 1) last = 0.0;
        a += last, c += whole;
      }
    }
    a = wave_sum(a), c = wave_sum(c);
    if ((threadIdx.x & 63) == 0) part[chunk & 1][threadIdx.x >> 6] = f64x2{a, c};
    __syncthreads();  // `part` of this chunk is there; that of the one before has been read, and so have its marks
    if (threadIdx.x == 0) {
      const f64x2* q = part[chunk & 1];
      p.sums[static_cast<int64_t>(b) * p.chunks + chunk] = (q[0] + q[1]) + (q[2] + q[3]);
    }
  }
}

// Exclusive running sums of x over the workgroup's lanes, and the total.
template <class V>
__device__ __forceinline__ V shift_up(V x, int by);
template <>
__device__ __forceinline__ double shift_up(double x, int by) { return __shfl_up(x, by); }
template <>
__device__ __forceinline__ f64x2 shift_up(f64x2 x, int by) { return f64x2{__shfl_up(x[0], by), __shfl_up(x[1], by)}; }
template <class V>
__device__ __forceinline__ V before_lane(V x, V* waves, V* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  V run = x;
#pragma unroll
  for (int i = 1; i < 64; i *= 2) {
    const V y = shift_up(run, i);
    if (lane >= i) run += y;
  }
  if (lane == 63) waves[wave] = run;
  __syncthreads();
  V base = {}, all = {};
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    if (i < wave) base += waves[i];
    all += waves[i];
  }
  __syncthreads();
  *total = all;
  const V up = shift_up(run, 1);
  return lane == 0 ? base : base + up;
}

// Draws a sequence's last token: the chunk in which the running sum passes the
// mark, and the value in it.  6 us, of loads in turn and barriers.
template <class T>
__global__ __launch_bounds__(kThreads) void draw_kernel(VerifyParams p) {
  __shared__ f64x2 both[kThreads / 64];
  __shared__ double waves[kThreads / 64];
  __shared__ uint32_t refused[kChunk / 32];
  __shared__ int found, fallback;
  __shared__ double found_base;
  const int b = static_cast<int>(p.group + blockIdx.x);
  Walk w = p.walks[b];
  if (w.count == 0) return;
  const f64x2* sums = p.sums + static_cast<int64_t>(b) * p.chunks;
  const int per = (p.chunks + kThreads - 1) / kThreads;  // chunks of a lane, one after another
  const int from = min(static_cast<int>(threadIdx.x) * per, p.chunks), to = min(from + per, p.chunks);
  f64x2 own = {}, totals;
  for (int i = from; i < to; ++i) own += sums[i];
  if (threadIdx.x == 0) found = INT32_MAX, fallback = -1;  // before the barriers below
  const f64x2 bases = before_lane(own, both, &totals);
  const int which = totals[0] > 0.0 ? 0 : 1;
  if (which) w.kids = 0;  // nothing is left to draw from but the target's own distribution
  const double base = bases[which], total = totals[which];
  int32_t* out = p.out_tokens + static_cast<int64_t>(b) * p.T + w.count - 1;
  if (!(total > 0.0)) return;  // stays -1
  const double u = static_cast<double>(p.uniform[b * p.u_b]);
  const double mark = u > 0.0 ? (u < 1.0 ? u * total : total) : u == u ? 0.0 : total;
  // the first chunk whose running sum passes the mark, else the last one that weighs something
  {
    double run = base;
    for (int i = from; i < to; ++i) {
      const double s = sums[i][which];
      run += s;
      if (s > 0.0 && run > mark) {
        atomicMin(&found, i);
        break;
      }
      if (s > 0.0) atomicMax(&fallback, i);
    }
  }
  __syncthreads();
  const bool passed = found != INT32_MAX;
  const int chunk = passed ? found : fallback;
  if (chunk >= from && chunk < to) {
    double run = base;
    for (int i = from; i < chunk; ++i) run += sums[i][which];
    found_base = run;
  }
  __syncthreads();
  const double start = found_base;
  if (threadIdx.x == 0) found = INT32_MAX, fallback = -1;
  if (!p.draft) {
    mark_refused(p, b, w.kids, chunk * kChunk, refused);
  } else {
    __syncthreads();
  }
  double last[kEach], whole[kEach], sum = 0.0, all;
  weights<T>(p, b, w, chunk * kChunk, refused, last, whole);
#pragma unroll
  for (int j = 0; j < kEach; ++j) sum += last[j];
  double run = start + before_lane(sum, waves, &all);
  int hit = INT32_MAX, some = -1;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    run += last[j];
    const int v = chunk * kChunk + static_cast<int>(threadIdx.x) * kEach + j;
    if (last[j] > 0.0) some = v;
    if (last[j] > 0.0 && run > mark) hit = min(hit, v);
  }
  if (hit != INT32_MAX) atomicMin(&found, hit);
  if (some >= 0) atomicMax(&fallback, some);
  __syncthreads();
  if (threadIdx.x == 0) *out = passed && found != INT32_MAX ? found : fallback;
}

int64_t chunks_of(int32_t V) { return (static_cast<int64_t>(V) + kChunk - 1) / kChunk; }

bool sizes_fit(int32_t B, int32_t T, int32_t V) {
  return B >= 0 && T >= 0 && T <= ETS_MAX_TREE && V >= 1 && V <= INT32_MAX - kChunk && chunks_of(V) * B <= INT32_MAX;
}

template <class T>
void launch(VerifyParams p, hipStream_t s) {
  launch_in_turn(static_cast<int64_t>(p.B) * p.groups, kThreads, [&](uint32_t first, uint32_t grid) {
    p.group = first;
    hipLaunchKernelGGL(weigh_kernel<T>, dim3(grid), dim3(kThreads), 0, s, p);
  });
  launch_in_turn(p.B, kThreads, [&](uint32_t first, uint32_t grid) {
    p.group = first;
    hipLaunchKernelGGL(draw_kernel<T>, dim3(grid), dim3(kThreads), 0, s, p);
  });
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_verify_workspace_size(int32_t B, int32_t T, int32_t V, size_t* bytes) {
  if (!bytes || !ets::sizes_fit(B, T, V)) return ETS_ERR_INVALID_ARG;
  *bytes = B && T ? static_cast<size_t>(B) * (ets::chunks_of(V) * sizeof(ets::f64x2) + sizeof(ets::Walk)) : 0;
  return ETS_OK;
}

ets_status ets_verify_drafts(const void* probs, int64_t p_b, int64_t p_t, const void* draft_probs, int64_t q_b, int64_t q_t,
                             int32_t B, int32_t T, int32_t V, const int32_t* tokens, int64_t tok_b, const float* uniform,
                             int64_t u_b, const int64_t* tree_mask, int64_t mask_b, const int32_t* lens, int32_t* out_tokens,
                             int32_t* out_path, int32_t* out_counts, int32_t dtype, void* workspace, size_t workspace_bytes,
                             void* stream) {
  using namespace ets;
  if (!sizes_fit(B, T, V) || !dtype_known(dtype) || (draft_probs && tree_mask)) return ETS_ERR_INVALID_ARG;
  if (B == 0) return ETS_OK;
  if (T == 0 || !probs || !tokens || !uniform || !out_tokens || !out_path || !out_counts) return ETS_ERR_INVALID_ARG;
  size_t need = 0;
  ets_verify_workspace_size(B, T, V, &need);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || workspace_bytes < need) return ETS_ERR_WORKSPACE;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const int64_t size = dtype == ETS_FP32 ? 4 : 2;
  VerifyParams p{};
  p.probs = static_cast<const char*>(probs), p.p_b = p_b * size, p.p_t = p_t * size;
  p.draft = static_cast<const char*>(draft_probs), p.q_b = q_b * size, p.q_t = q_t * size;
  p.B = B, p.T = T, p.V = V, p.chunks = static_cast<int32_t>(chunks_of(V));
  p.tokens = tokens, p.tok_b = tok_b, p.uniform = uniform, p.u_b = u_b;
  p.mask = tree_mask, p.mask_b = mask_b, p.lens = lens;
  p.out_tokens = out_tokens, p.out_path = out_path, p.out_counts = out_counts;
  p.sums = static_cast<f64x2*>(workspace);
  p.walks = reinterpret_cast<Walk*>(p.sums + static_cast<int64_t>(B) * p.chunks);
  const int64_t work = static_cast<int64_t>(B) * p.chunks, room = static_cast<int64_t>(cu) * kPerUnit;
  const int64_t each = (work + room - 1) / room;
  p.each = static_cast<int32_t>(each < p.chunks ? each : p.chunks);
  p.groups = (p.chunks + p.each - 1) / p.each;
  p.by_groups = fast_div(p.groups);
  auto s = static_cast<hipStream_t>(stream);
  if (dtype == ETS_BF16) {
    launch<__bf16>(p, s);
  } else if (dtype == ETS_FP16) {
    launch<_Float16>(p, s);
  } else {
    launch<float>(p, s);
  }
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"
