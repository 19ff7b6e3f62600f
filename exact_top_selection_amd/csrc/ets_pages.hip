// ets_pages.hip -- the pages of a pool: copied, taken, let go, branched and
// drawn together (gfx950).  Nothing is kept on the host: which pages are free
// is read from their counts, so calls can follow each other in a graph.
#include "ets_speculate.h"

#include "ets_cache_format.h"

namespace ets {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 8;                  // entries of a lane, kThreads apart
constexpr int kChunk = kThreads * kEach;  // of a workgroup
constexpr int64_t kMaxPages = static_cast<int64_t>(1) << 26;
constexpr int kPiece = 16384;             // bytes of a page that a workgroup moves at a time

struct Buffers {
  char* data[ETS_MAX_BUFFERS];
  int64_t page_bytes[ETS_MAX_BUFFERS];
  int32_t end[ETS_MAX_BUFFERS];  // pieces of a page of this buffer and those before it
  int32_t count, pieces;
};

enum Kind { kExtend, kFork, kCompact };

struct PoolParams {
  int32_t* refs;
  int32_t P;
  int32_t* table;  // fork: read only
  int64_t pt_b;
  int32_t B, M;
  const int32_t* lens;
  int32_t page_size;
  const int32_t* parents;  // fork
  int32_t* out;
  int64_t out_b;
  int32_t out_M;
  int32_t* lacking;
  int32_t* moved;  // compact
  int32_t page_chunks, entries, entry_chunks;
  uint32_t group;  // the launch's first workgroup, where a launch does not hold them all
  // workspace
  int32_t* head;        // [0]: free pages under the number in use (compact)
  int32_t* page_count;  // free pages of each chunk
  int32_t* entry_count; // entries of each chunk that want a page
  int32_t* free_list;   // free pages, lowest first
  int32_t* used_list;   // compact: pages in use, lowest first
  int32_t* rank;        // compact: a page's place among those in use
  FastDiv by_M, by_pieces, by_page;
};

__device__ __forceinline__ int pages_of(const PoolParams& p, int len) {
  return len <= 0 ? 0 : static_cast<int>(div_by(static_cast<uint32_t>(len - 1), p.by_page)) + 1;
}
__device__ __forceinline__ bool holds(const PoolParams& p, int entry) { return entry >= 0 && entry < p.P; }

// Whether branch i wants a page of its own.
__device__ __forceinline__ bool wants(const PoolParams& p, int i) {
  const int b = p.parents[i];
  if (b < 0 || b >= p.B) return false;
  const int len = max(p.lens[b], 0), full = static_cast<int>(div_by(len, p.by_page));
  return len != full * p.page_size && full < p.M && full < p.out_M && holds(p, p.table[b * p.pt_b + full]);
}

// Places of a workgroup's flags in order (entry j of lane t is number j * kThreads + t), and how many there are.
__device__ __forceinline__ int places(uint32_t flags, int (&place)[kEach], int* counts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kWaves = kThreads / 64, kParts = kEach * kWaves;
  static_assert(kParts <= 64, "one wave sums the parts");
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const uint64_t set = __ballot(flags >> j & 1);
    place[j] = __popcll(set & ((1ull << lane) - 1));
    if (lane == 0) counts[j * kWaves + wave] = __popcll(set);
  }
  __syncthreads();
  if (wave == 0) {
    const int mine = lane < kParts ? counts[lane] : 0;
    int run = mine;
#pragma unroll
    for (int i = 1; i < kParts; i *= 2) {
      const int y = __shfl_up(run, i);
      if (lane >= i) run += y;
    }
    if (lane < kParts) counts[lane] = run - mine;
    if (lane == kParts - 1) counts[kParts] = run;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j) place[j] += counts[j * kWaves + wave];
  const int total = counts[kParts];
  __syncthreads();
  return total;
}

// Sums of the counts before `mine`, and of all.
__device__ __forceinline__ void chunk_base(const int32_t* counts, int n, int mine, int* base, int* total, int* shared) {
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int c = counts[i];
    all += c;
    before += i < mine ? c : 0;
  }
#pragma unroll
  for (int i = 1; i < 64; i *= 2) before += __shfl_xor(before, i), all += __shfl_xor(all, i);
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = before, shared[4 + (threadIdx.x >> 6)] = all;
  __syncthreads();
  *base = shared[0] + shared[1] + shared[2] + shared[3];
  *total = shared[4] + shared[5] + shared[6] + shared[7];
  __syncthreads();
}

__device__ __forceinline__ uint32_t free_flags(const PoolParams& p, int chunk) {
  uint32_t flags = 0;
  int refs[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int64_t i = static_cast<int64_t>(chunk) * kChunk + j * kThreads + threadIdx.x;
    refs[j] = i < p.P ? p.refs[i] : 1;
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) flags |= refs[j] <= 0 ? 1u << j : 0;
  return flags;
}
template <int KIND>
__device__ __forceinline__ uint32_t want_flags(const PoolParams& p, int chunk) {
  uint32_t flags = 0;
  if constexpr (KIND == kExtend) {
    // all loads first, those of entries behind the last from the last
    int len[kEach], entry[kEach], column[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t at = static_cast<int64_t>(chunk) * kChunk + j * kThreads + threadIdx.x;
      const int i = at < p.entries ? static_cast<int>(at) : p.entries - 1;
      const int b = static_cast<int>(div_by(i, p.by_M));
      column[j] = i - b * p.M;
      len[j] = p.lens[b];
      entry[j] = p.table[b * p.pt_b + column[j]];
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t at = static_cast<int64_t>(chunk) * kChunk + j * kThreads + threadIdx.x;
      if (at < p.entries && column[j] < pages_of(p, len[j]) && !holds(p, entry[j])) flags |= 1u << j;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t i = static_cast<int64_t>(chunk) * kChunk + j * kThreads + threadIdx.x;
      if (i < p.entries && wants(p, static_cast<int>(i))) flags |= 1u << j;
    }
  }
  return flags;
}

// Three launches put entries and pages together (four with fork's copies): counts
// by chunk, lists, then what they say.  4 + 4 + 5 us for 256 rows of 256 entries on
// 32768 pages: a launch and two loads in turn each.  The flags' loads all go out
// before the first test (24 us in all where each waited for its own).

// First launch: how many pages of each chunk are free, how many entries want one.
template <int KIND>
__global__ __launch_bounds__(kThreads) void count_kernel(PoolParams p) {
  __shared__ int counts[kThreads / 64 * kEach + 1];
  const int chunk = static_cast<int>(blockIdx.x), entry = chunk - p.page_chunks;
  int place[kEach];
  const int n = places(entry < 0 ? free_flags(p, chunk) : want_flags<KIND>(p, entry), place, counts);
  if (threadIdx.x == 0) (entry < 0 ? p.page_count[chunk] : p.entry_count[entry]) = n;
  if (KIND == kExtend && entry < 0) {
    // rows' counts of missing pages start at zero
    for (int64_t i = static_cast<int64_t>(chunk) * kThreads + threadIdx.x; i < p.B; i += static_cast<int64_t>(p.page_chunks) * kThreads)
      p.lacking[i] = 0;
  }
}

// Second launch: free pages by their place; those that are wanted are taken.
template <int KIND>
__global__ __launch_bounds__(kThreads) void list_kernel(PoolParams p) {
  __shared__ int counts[kThreads / 64 * kEach + 1];
  __shared__ int sums[8];
  const int chunk = static_cast<int>(blockIdx.x);
  int base, total, before, wanted = 0;
  chunk_base(p.page_count, p.page_chunks, chunk, &base, &total, sums);
  if (KIND != kCompact) chunk_base(p.entry_count, p.entry_chunks, 0, &before, &wanted, sums);
  if (KIND != kCompact && base >= wanted) return;
  const uint32_t flags = free_flags(p, chunk);
  int place[kEach];
  places(flags, place, counts);
  const int used = p.P - total;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int64_t at = static_cast<int64_t>(chunk) * kChunk + j * kThreads + threadIdx.x;
    if (at >= p.P) continue;
    const int i = static_cast<int>(at), r = base + place[j];
    const bool free = flags >> j & 1;
    if (KIND != kCompact) {
      if (free && r < wanted) {
        p.free_list[r] = i;
        p.refs[i] = 1;
      }
    } else {
      const int order = i - r;  // among those in use
      if (free) {
        p.free_list[r] = i;
      } else {
        p.used_list[order] = i;
      }
      p.rank[i] = order;
      if (i == used) p.head[0] = r;  // free pages under that number; with no free page nothing asks
      p.moved[i] = free ? -1 : i;
    }
  }
}

// Third launch of extend: entries get their pages.
__global__ __launch_bounds__(kThreads) void extend_kernel(PoolParams p) {
  __shared__ int counts[kThreads / 64 * kEach + 1];
  __shared__ int sums[8];
  const int chunk = static_cast<int>(blockIdx.x);
  int base, total, before, available;
  chunk_base(p.entry_count, p.entry_chunks, chunk, &base, &total, sums);
  if (total == 0) return;
  chunk_base(p.page_count, p.page_chunks, 0, &before, &available, sums);
  const uint32_t flags = want_flags<kExtend>(p, chunk);
  int place[kEach];
  places(flags, place, counts);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (!(flags >> j & 1)) continue;
    const int i = chunk * kChunk + j * kThreads + static_cast<int>(threadIdx.x);  // flagged, so under p.entries
    const int b = static_cast<int>(div_by(i, p.by_M)), r = base + place[j];
    const bool there = r < available;
    p.table[b * p.pt_b + (i - b * p.M)] = there ? p.free_list[r] : -1;
    if (!there) atomicAdd(&p.lacking[b], 1);
  }
}

// Third launch of fork: a workgroup writes one branch's row.
__global__ __launch_bounds__(kThreads) void branch_kernel(PoolParams p) {
  __shared__ int sums[8];
  const int i = static_cast<int>(p.group + blockIdx.x);
  const int b = p.parents[i];
  int32_t* row = p.out + i * p.out_b;
  const bool there = b >= 0 && b < p.B;
  const int full = there ? static_cast<int>(div_by(max(p.lens[b], 0), p.by_page)) : 0;
  const bool want = wants(p, i);
  // branches before this one that want a page
  int before = 0;
  if (want) {
    const int chunk = i / kChunk;
    for (int k = threadIdx.x; k < chunk; k += kThreads) before += p.entry_count[k];
    for (int k = chunk * kChunk + static_cast<int>(threadIdx.x); k < i; k += kThreads) before += wants(p, k);
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) before += __shfl_xor(before, k);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = before;
  __syncthreads();
  const int place = sums[0] + sums[1] + sums[2] + sums[3];
  __syncthreads();
  int none, available = 0;
  if (want) chunk_base(p.page_count, p.page_chunks, 0, &none, &available, sums);
  const int fresh = want && place < available ? p.free_list[place] : -1;
  for (int j = threadIdx.x; j < p.out_M; j += kThreads) {
    int entry = -1;
    if (there && j < full && j < p.M) {
      const int held = p.table[b * p.pt_b + j];
      if (holds(p, held)) {
        entry = held;
        atomicAdd(&p.refs[held], 1);
      }
    } else if (j == full) {
      entry = fresh;
    }
    row[j] = entry;
  }
  if (threadIdx.x == 0) p.lacking[i] = want && fresh < 0;
}

// One piece of a page of some buffer.  Drawing 8192 pages of 131 KB together moves
// 250 to 300 MB in 100 us (5.3 TB/s, as a copy does); 128 branches' pages take 6.
__device__ __forceinline__ void move_piece(const Buffers& buffers, int piece, int64_t src, int64_t dst) {
  int k = 0, before = 0;
  while (piece >= buffers.end[k]) before = buffers.end[k++];
  const int64_t bytes = buffers.page_bytes[k], at = static_cast<int64_t>(piece - before) * kPiece;
  const char* from = buffers.data[k] + src * bytes + at;
  char* to = buffers.data[k] + dst * bytes + at;
  const int n = static_cast<int>(bytes - at < kPiece ? bytes - at : kPiece);
  u32v4 v[kPiece / kThreads / 16];
#pragma unroll
  for (int i = 0; i < kPiece / kThreads / 16; ++i) {
    const int o = (i * kThreads + static_cast<int>(threadIdx.x)) * 16;
    if (o + 16 <= n) v[i] = load_any<u32v4>(from + o);
  }
#pragma unroll
  for (int i = 0; i < kPiece / kThreads / 16; ++i) {
    const int o = (i * kThreads + static_cast<int>(threadIdx.x)) * 16;
    if (o + 16 <= n) store_any(to + o, v[i]);
  }
  const int tail = n & ~15;
  if (static_cast<int>(threadIdx.x) < n - tail) to[tail + threadIdx.x] = from[tail + threadIdx.x];
}

__global__ __launch_bounds__(kThreads) void copy_kernel(Buffers buffers, const int32_t* src, const int32_t* dst, int64_t P, FastDiv by_pieces, uint32_t first) {
  const uint32_t group = first + blockIdx.x, pair = div_by(group, by_pieces);
  const int64_t s = src[pair], d = dst[pair];
  if (s < 0 || s >= P || d < 0 || d >= P) return;
  move_piece(buffers, static_cast<int>(group - pair * by_pieces.d), s, d);
}

// Fourth launch of fork: the pages that branches hold in part.
__global__ __launch_bounds__(kThreads) void branch_copy_kernel(PoolParams p, Buffers buffers) {
  const uint32_t group = p.group + blockIdx.x, i = div_by(group, p.by_pieces);
  if (!wants(p, static_cast<int>(i))) return;
  const int b = p.parents[i], full = static_cast<int>(div_by(p.lens[b], p.by_page));
  const int to = p.out[i * p.out_b + full];
  if (to < 0) return;
  move_piece(buffers, static_cast<int>(group - i * p.by_pieces.d), p.table[b * p.pt_b + full], to);
}

// Third launch of compact: page after page moves, the first workgroups' share, and table entries and counts follow.
__global__ __launch_bounds__(kThreads) void compact_kernel(PoolParams p, Buffers buffers, int movers) {
  __shared__ int sums[8];
  int none, available;
  chunk_base(p.page_count, p.page_chunks, 0, &none, &available, sums);
  const int used = p.P - available;
  const int moves = used < p.P ? p.head[0] : 0;  // as many as there are free pages under `used`
  const int above = used - moves;                // the first of used_list that moves
  if (static_cast<int>(blockIdx.x) < movers) {
    const int64_t all = static_cast<int64_t>(moves) * buffers.pieces;
    for (int64_t i = blockIdx.x; i < all; i += movers) {
      const int k = static_cast<int>(i / buffers.pieces);
      move_piece(buffers, static_cast<int>(i - static_cast<int64_t>(k) * buffers.pieces), p.used_list[above + k], p.free_list[k]);
    }
    return;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x - movers) * kThreads;
  const int64_t start = (static_cast<int64_t>(blockIdx.x) - movers) * kThreads + threadIdx.x;
  for (int64_t k = start; k < moves; k += step) {
    const int from = p.used_list[above + k], to = p.free_list[k];
    p.moved[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  for (int64_t i = start; i < p.entries; i += step) {
    const int b = static_cast<int>(div_by(static_cast<uint32_t>(i), p.by_M));
    int32_t* at = p.table + b * p.pt_b + (i - static_cast<int64_t>(b) * p.M);
    const int entry = *at;
    if (!holds(p, entry)) continue;
    if (p.moved[entry] < 0) {
      *at = -1;  // a free page, which never gets another number
    } else if (entry >= used) {
      *at = p.free_list[p.rank[entry] - above];
    }
  }
}

bool pool_fits(int64_t P, int64_t entries) { return P >= 0 && P <= kMaxPages && entries >= 0 && entries <= INT32_MAX - kChunk; }
int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }
size_t pool_bytes(int64_t P, int64_t entries) {
  return 4 * static_cast<size_t>(32 + chunks_of(P) + chunks_of(entries) + 3 * P);
}

ets_status take_buffers(const ets_page_buffer* from, int32_t count, int64_t P, Buffers* to) {
  if (count < 0 || count > ETS_MAX_BUFFERS || (count && !from)) return ETS_ERR_INVALID_ARG;
  *to = Buffers{};
  int64_t pieces = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (from[i].page_bytes < 0 || (!from[i].data && from[i].page_bytes && P)) return ETS_ERR_INVALID_ARG;
    pieces += (from[i].page_bytes + kPiece - 1) / kPiece;
    if (pieces > INT32_MAX) return ETS_ERR_INVALID_ARG;
    to->data[i] = static_cast<char*>(from[i].data);
    to->page_bytes[i] = from[i].page_bytes;
    to->end[i] = static_cast<int32_t>(pieces);
  }
  to->count = count, to->pieces = static_cast<int32_t>(pieces);
  return ETS_OK;
}

ets_status pool_params(PoolParams* p, int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, int64_t entries,
                       void* workspace, size_t workspace_bytes) {
  if (B < 0 || M < 0 || !pool_fits(P, entries) || (P && !refs) || (B && M && !table)) return ETS_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || workspace_bytes < pool_bytes(P, entries)) return ETS_ERR_WORKSPACE;
  *p = PoolParams{};
  p->refs = refs, p->P = static_cast<int32_t>(P), p->table = table, p->pt_b = pt_b, p->B = B, p->M = M;
  p->entries = static_cast<int32_t>(entries);
  p->page_chunks = static_cast<int32_t>(chunks_of(P)), p->entry_chunks = static_cast<int32_t>(chunks_of(entries));
  p->head = static_cast<int32_t*>(workspace);
  p->page_count = p->head + 16;
  p->entry_count = p->page_count + p->page_chunks;
  p->free_list = p->entry_count + p->entry_chunks;
  p->used_list = p->free_list + P;
  p->rank = p->used_list + P;
  p->by_M = fast_div(M ? M : 1);
  p->by_pieces = fast_div(1), p->by_page = fast_div(1);
  return ETS_OK;
}

// Whether rows of two tables share an entry: `n` rows of `width` entries, `pitch` apart.
struct Rows {
  const int32_t* data;
  int64_t pitch, n, width;
};
bool rows_meet(Rows a, Rows b) {
  if (a.n < 1 || b.n < 1 || a.width < 1 || b.width < 1) return false;
  for (Rows* r : {&a, &b}) {
    if (r->pitch < 0) r->data += r->pitch * (r->n - 1), r->pitch = -r->pitch;
    if (r->pitch == 0) r->n = 1;
  }
  if (b.n < a.n) {
    const Rows c = a;
    a = b, b = c;
  }
  // in bytes, from b's first row
  const int64_t start = static_cast<int64_t>(reinterpret_cast<intptr_t>(a.data) - reinterpret_cast<intptr_t>(b.data));
  const int64_t wide = 4 * a.width, other = 4 * b.width, step = 4 * b.pitch;
  if (start >= step * (b.n - 1) + other || start + 4 * a.pitch * (a.n - 1) + wide <= 0) return false;
  for (int64_t i = 0; i < a.n; ++i) {
    // b's first row that ends behind the start of this one
    const int64_t at = start + 4 * a.pitch * i, j = at < other ? 0 : (at - other) / step + 1;
    if (j < b.n && j * step < at + wide) return true;
  }
  return false;
}

uint32_t grid_of(int64_t n) { return static_cast<uint32_t>(n < 1 ? 1 : n); }

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_pages_workspace_size(int64_t P, int64_t rows, size_t* bytes) {
  if (!bytes || !ets::pool_fits(P, rows)) return ETS_ERR_INVALID_ARG;
  *bytes = ets::pool_bytes(P, rows);
  return ETS_OK;
}

ets_status ets_pages_copy(const ets_page_buffer* buffers, int32_t count, int64_t P, const int32_t* src, const int32_t* dst, int64_t n,
                          void* stream) {
  using namespace ets;
  Buffers to;
  if (P < 0 || P > kMaxPages || n < 0 || (n && (!src || !dst))) return ETS_ERR_INVALID_ARG;
  if (ets_status st = take_buffers(buffers, count, P, &to); st != ETS_OK) return st;
  if (n == 0 || P == 0 || to.pieces == 0) return ETS_OK;
  if (n > INT32_MAX / to.pieces) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  const FastDiv by_pieces = fast_div(to.pieces);
  launch_in_turn(n * to.pieces, kThreads, [&](uint32_t first, uint32_t grid) {
    hipLaunchKernelGGL(copy_kernel, dim3(grid), dim3(kThreads), 0, static_cast<hipStream_t>(stream), to, src, dst, P, by_pieces, first);
  });
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

ets_status ets_pages_extend(int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, const int32_t* lens,
                            int32_t page_size, int32_t* lacking, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ets;
  if (page_size < 1 || B < 0 || M < 0 || (B && (!lens || !lacking))) return ETS_ERR_INVALID_ARG;
  PoolParams p;
  if (ets_status st = pool_params(&p, refs, P, table, pt_b, B, M, static_cast<int64_t>(B) * M, workspace, workspace_bytes); st != ETS_OK)
    return st;
  if (B == 0) return ETS_OK;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  p.lens = lens, p.page_size = page_size, p.by_page = fast_div(page_size), p.lacking = lacking;
  if (p.page_chunks == 0) p.page_chunks = 1;  // an empty chunk: the counts of missing pages are cleared all the same
  auto s = static_cast<hipStream_t>(stream);
  p.entry_count = p.page_count + p.page_chunks;
  p.free_list = p.entry_count + p.entry_chunks;
  hipLaunchKernelGGL(count_kernel<kExtend>, dim3(grid_of(p.page_chunks + p.entry_chunks)), dim3(kThreads), 0, s, p);
  hipLaunchKernelGGL(list_kernel<kExtend>, dim3(grid_of(p.page_chunks)), dim3(kThreads), 0, s, p);
  if (p.entry_chunks) hipLaunchKernelGGL(extend_kernel, dim3(grid_of(p.entry_chunks)), dim3(kThreads), 0, s, p);
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"

namespace ets {
namespace {

__global__ __launch_bounds__(kThreads) void free_kernel(PoolParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.entries) return;
  const int b = static_cast<int>(div_by(static_cast<uint32_t>(i), p.by_M)), j = static_cast<int>(i - static_cast<int64_t>(b) * p.M);
  if (j < pages_of(p, p.lens[b])) return;
  int32_t* at = p.table + b * p.pt_b + j;
  const int entry = *at;
  if (entry == -1) return;
  *at = -1;
  if (holds(p, entry)) atomicSub(&p.refs[entry], 1);
}

}  // namespace
}  // namespace ets

extern "C" {

ets_status ets_pages_free(int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, const int32_t* lens,
                          int32_t page_size, void* stream) {
  using namespace ets;
  const int64_t entries = static_cast<int64_t>(B) * M;
  if (page_size < 1 || B < 0 || M < 0 || !pool_fits(P, entries) || (P && !refs) || (B && (!lens || (M && !table))))
    return ETS_ERR_INVALID_ARG;
  if (entries == 0) return ETS_OK;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  PoolParams p{};
  p.refs = refs, p.P = static_cast<int32_t>(P), p.table = table, p.pt_b = pt_b, p.B = B, p.M = M, p.lens = lens;
  p.page_size = page_size, p.by_page = fast_div(page_size), p.by_M = fast_div(M), p.entries = static_cast<int32_t>(entries);
  hipLaunchKernelGGL(free_kernel, dim3(static_cast<uint32_t>((entries + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), p);
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

ets_status ets_pages_fork(int32_t* refs, int64_t P, const int32_t* table, int64_t pt_b, int32_t B, int32_t M, const int32_t* lens,
                          int32_t page_size, const int32_t* parents, int32_t n, int32_t* out, int64_t out_b, int32_t out_M,
                          int32_t* lacking, const ets_page_buffer* buffers, int32_t count, void* workspace, size_t workspace_bytes,
                          void* stream) {
  using namespace ets;
  if (page_size < 1 || n < 0 || out_M < 0 || (n && (!parents || !lacking || (out_M && !out))) || (B > 0 && !lens)) return ETS_ERR_INVALID_ARG;
  PoolParams p;
  if (ets_status st = pool_params(&p, refs, P, const_cast<int32_t*>(table), pt_b, B, M, n, workspace, workspace_bytes); st != ETS_OK)
    return st;
  Buffers held;
  if (ets_status st = take_buffers(buffers, count, P, &held); st != ETS_OK) return st;
  if (n == 0) return ETS_OK;
  if (held.pieces && n > INT32_MAX / held.pieces) return ETS_ERR_INVALID_ARG;
  // rows are read while others are written
  if (rows_meet({table, pt_b, B, M}, {out, out_b, n, out_M})) return ETS_ERR_INVALID_ARG;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  p.lens = lens, p.page_size = page_size, p.by_page = fast_div(page_size);
  p.parents = parents, p.out = out, p.out_b = out_b, p.out_M = out_M, p.lacking = lacking;
  auto s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(count_kernel<kFork>, dim3(grid_of(p.page_chunks + p.entry_chunks)), dim3(kThreads), 0, s, p);
  if (p.page_chunks) hipLaunchKernelGGL(list_kernel<kFork>, dim3(grid_of(p.page_chunks)), dim3(kThreads), 0, s, p);
  launch_in_turn(n, kThreads, [&](uint32_t first, uint32_t grid) {
    p.group = first;
    hipLaunchKernelGGL(branch_kernel, dim3(grid), dim3(kThreads), 0, s, p);
  });
  p.by_pieces = fast_div(held.pieces ? held.pieces : 1);
  launch_in_turn(static_cast<int64_t>(n) * held.pieces, kThreads, [&](uint32_t first, uint32_t grid) {
    p.group = first;
    hipLaunchKernelGGL(branch_copy_kernel, dim3(grid), dim3(kThreads), 0, s, p, held);
  });
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

ets_status ets_pages_compact(int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, int32_t* moved,
                             const ets_page_buffer* buffers, int32_t count, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace ets;
  if (B < 0 || M < 0 || (P && !moved)) return ETS_ERR_INVALID_ARG;
  PoolParams p;
  if (ets_status st = pool_params(&p, refs, P, table, pt_b, B, M, static_cast<int64_t>(B) * M, workspace, workspace_bytes); st != ETS_OK)
    return st;
  Buffers held;
  if (ets_status st = take_buffers(buffers, count, P, &held); st != ETS_OK) return st;
  if (P == 0) return ETS_OK;
  int32_t cu = 0;
  if (ets_status st = device_ready(&cu); st != ETS_OK) return st;
  p.moved = moved;
  auto s = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(count_kernel<kCompact>, dim3(grid_of(p.page_chunks)), dim3(kThreads), 0, s, p);
  hipLaunchKernelGGL(list_kernel<kCompact>, dim3(grid_of(p.page_chunks)), dim3(kThreads), 0, s, p);
  const int64_t most = P / 2 * held.pieces, movers = held.pieces ? (most < 8 * cu ? most : 8 * cu) : 0;
  const int64_t longest = p.entries > P ? p.entries : P, follow = (longest + 4 * kThreads - 1) / (4 * kThreads);
  hipLaunchKernelGGL(compact_kernel, dim3(static_cast<uint32_t>(movers + (follow < cu ? follow : cu))), dim3(kThreads), 0, s, p, held,
                     static_cast<int>(movers));
  return hipGetLastError() == hipSuccess ? ETS_OK : ETS_ERR_HIP;
}

}  // extern "C"
