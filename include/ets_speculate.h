/*
 * ets_speculate.h -- C ABI of the operators of a speculative decode step over
 * a pool of cache pages, for AMD MI355X (gfx950); part of libets_topk.so.
 *
 *   ets_block_write    quantises new rows into a block cache
 *   ets_block_keep     moves the rows of accepted drafts to where they belong
 *   ets_attend_blocks  attention over a block cache: single tokens, trees of
 *                      drafted tokens, pieces of prompts
 *   ets_verify_drafts  which drafted tokens stand, and the next one
 *   ets_pages_copy, ets_pages_extend, ets_pages_free, ets_pages_fork,
 *   ets_pages_compact  the pages of a pool
 *
 * Block cache.  A cache is codes[S][H][D] (e4m3, as in ets_decode.h) and
 * scales[S / N][H]: one byte s for the N slots of a block and a head; the value
 * of a code c is c * 2^(s - 127).  N divides S and the page size, so that a
 * block lies in one page.  Scale bytes are 1 to 246.  D is a multiple of 32.
 * A scale grows with the values that come into its block.  Being a power of
 * two it re-rounds only those older codes that fall beneath 2^-6 of the new
 * scale's unit.
 *
 * Positions.  Position p of sequence b is slot page_table[b][p / page_size] *
 * page_size + p % page_size.  A position that is negative or behind the table,
 * or whose page is not inside [0, S / page_size), is not there: it is skipped
 * by the writes and not seen by attention.
 *
 * Pool.  refs[P] counts the table entries that hold each page; a page with
 * refs <= 0 is free.  Table entries outside [0, P) hold no page.
 *
 * Conventions are those of ets_decode.h: device pointers of the caller, nothing
 * allocated, the host never synchronised, arguments checked before anything is
 * enqueued, strides in elements, no alignment beyond the element's needed, and
 * results that do not change from run to run.  Workspaces need no particular
 * contents, and calls ordered on one stream may share one.
 */
#ifndef ETS_SPECULATE_H
#define ETS_SPECULATE_H

#include "ets_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ETS_MAX_BLOCK_DIM 256 /* largest D and Dv of a block cache */
#define ETS_MAX_BUFFERS 64    /* most buffers of a pool that one call moves */

/*
 * x[b][t] of `dtype`, t < min(counts[b], T), to position first[b] + t.  With m
 * the largest finite magnitude of a block and head's new rows, its exponent e
 * is the smallest in [-126, 119] with m <= 448 * 2^e (-126 where m = 0), and
 * not less than the one before where the block holds rows of earlier positions
 * than first[b]; those rows' codes are rounded to the new exponent.  New values
 * are x * 2^-e, rounded to nearest even and limited to +-448; NaN stays NaN,
 * infinities become +-448 * 2^e.  Rows of the block behind the new ones keep
 * their bytes and are taken for nothing.  A sequence with first[b] < 0 or
 * counts[b] <= 0 is left alone.  The pages that one call writes belong to one
 * sequence each.  H * D <= 2^28, D <= ETS_MAX_BLOCK_DIM; T, and B * H times
 * the blocks that T rows may touch, up to 2^31 - 1.  Rows of table_pages
 * entries, pt_b apart.
 */
ets_status ets_block_write(const void* x, int64_t x_b, int64_t x_t, int64_t x_h, int32_t B, int32_t T, int32_t H,
                           int32_t D, uint8_t* codes, int64_t codes_s, int64_t codes_h, uint8_t* scales,
                           int64_t scales_s, int64_t scales_h, int64_t S, int32_t block, const int32_t* page_table,
                           int64_t pt_b, int32_t table_pages, int32_t page_size, const int32_t* first,
                           const int32_t* counts, int32_t dtype, void* stream);

/*
 * The rows at positions first[b] + path[b][i], i < min(counts[b], T), move to
 * first[b] + i: all are read before any is written, and written as
 * ets_block_write writes their values.  Rows from the start with path[b][i] =
 * i stay as they are, and count as rows of earlier positions.  An entry of path
 * outside [0, T), or whose position is not there, leaves its place a row of
 * zeros.  T <= ETS_MAX_TREE.
 */
ets_status ets_block_keep(int32_t B, int32_t T, int32_t H, int32_t D, uint8_t* codes, int64_t codes_s, int64_t codes_h,
                          uint8_t* scales, int64_t scales_s, int64_t scales_h, int64_t S, int32_t block,
                          const int32_t* page_table, int64_t pt_b, int32_t table_pages, int32_t page_size,
                          const int32_t* first, const int32_t* path, int64_t path_b, const int32_t* counts, void* stream);

/*
 * Attention of q[b][t][hq] over the first n = min(seq_lens[b], L) positions of
 * its sequence, hq = hk * (Hq / Hkv) + i sharing head hk of the cache:
 *   x_p = D^-1/2 q . k_p over the positions p < n that (b, t) sees,
 *   out = sum_p softmax(x)_p v_p,  lse = log sum_p exp(x_p).
 * It sees
 *   - first == NULL: all of them;
 *   - first != NULL: token t stands at position first[b] + t.  Where that is
 *     not below n the token is padding and sees nothing.  Others see p <
 *     first[b], and first[b] + j for j <= t, or, with tree_mask, for j < T with
 *     bit j of tree_mask[b][t] set (T <= ETS_MAX_TREE then).
 * A row that sees nothing has out = 0 and lse = -inf.  Numerics are those of
 * ets_attend; products of keys are exact for bf16 and fp16 queries.  The
 * probabilities' 16 bits show where an exact result lies next to a border of the
 * output type: one bf16 result in a thousand is the other neighbour of what 32-bit
 * probabilities give, as near to the exact one over all.  One launch
 * takes a call, a workgroup of 256 or 512 lanes 16 to 256 rows of a list: sizes
 * that need 2^32 lanes or more (16 million workgroups) are refused.
 */
typedef struct ets_attend_blocks_args {
  int32_t B, T, Hq, Hkv, D, Dv;
  int32_t dtype;          /* of q and out: ETS_BF16 or ETS_FP16 */
  int32_t block;          /* slots that share a scale */
  int32_t L;              /* positions of a sequence at most */
  int32_t page_size;
  int64_t S;              /* slots of the cache */
  const void* q;          /* [B][T][Hq][D] */
  int64_t q_b, q_t, q_h;
  const uint8_t* k_codes; /* [S][Hkv][D] */
  int64_t k_s, k_h;
  const uint8_t* k_scales; /* [S / block][Hkv] */
  int64_t ks_s, ks_h;
  const uint8_t* v_codes; /* [S][Hkv][Dv] */
  int64_t v_s, v_h;
  const uint8_t* v_scales;
  int64_t vs_s, vs_h;
  const int32_t* page_table; /* [B][>= ceil(L / page_size)] */
  int64_t pt_b;
  const int32_t* seq_lens;   /* [B] */
  const int32_t* first;      /* [B] or NULL */
  const int64_t* tree_mask;  /* [B][T] or NULL */
  int64_t mask_b;
  void* out;                 /* contiguous [B][T][Hq][Dv] */
  float* lse;                /* contiguous [B][T][Hq] */
} ets_attend_blocks_args;

ets_status ets_attend_blocks_workspace_size(const ets_attend_blocks_args* args, size_t* bytes);
ets_status ets_attend_blocks(const ets_attend_blocks_args* args, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Which drafted tokens of a sequence stand, and the token that follows.  Nodes
 * 0 .. n - 1, n = min(lens[b], T) (T without lens): node 0 is the last token
 * that stands already, the others were drafted.  Node t's parent is the
 * highest bit under t of tree_mask[b][t], or t - 1 without a mask; a node
 * without one is never reached.  p(a, .) = probs[b][a] is the target's
 * distribution after node a, u_t = uniform[b][t] in [0, 1).  From a = 0 on, the
 * children c of a are tried in order, with x = tokens[b][c], w = p(a, x) (0
 * for a token outside [0, V), or that a child before it had):
 *   - with draft_probs (a chain: no mask), q = draft_probs[b][c - 1][x]: c is
 *     taken if u_c * q < w;
 *   - without, c is taken if u_c * rest < w, else rest (1 at first) loses w.
 * The taken child is the next a; where none is, the last token is drawn from
 *   max(p(a, v) - draft_probs[b][a][v], 0) if a drafted token was refused,
 *   or p(a, v) without the tokens of a's children,
 *   or p(a, v) where that has no positive value:
 * the lowest v whose running sum is over u_0 * total (u_0 limited to [0, 1];
 * the last v of positive weight if none is).  Everything is in 64 bits.
 * Probabilities that are negative, infinite or no number count as 0.
 *   out_tokens, out_path  int32 [B][T], contiguous: the taken tokens and the
 *     drawn one (-1 if all weights are 0); the nodes 0, .. that led there.  -1
 *     behind them.
 *   out_counts int32 [B]: how many nodes (and tokens) that is; 0 where n <= 0.
 * T <= ETS_MAX_TREE, draft_probs [B][T - 1][V].
 */
ets_status ets_verify_workspace_size(int32_t B, int32_t T, int32_t V, size_t* bytes);
ets_status ets_verify_drafts(const void* probs, int64_t p_b, int64_t p_t, const void* draft_probs, int64_t q_b, int64_t q_t,
                             int32_t B, int32_t T, int32_t V, const int32_t* tokens, int64_t tok_b, const float* uniform,
                             int64_t u_b, const int64_t* tree_mask, int64_t mask_b, const int32_t* lens,
                             int32_t* out_tokens, int32_t* out_path, int32_t* out_counts, int32_t dtype,
                             void* workspace, size_t workspace_bytes, void* stream);

/* A buffer of a pool: P pages of page_bytes each, one after another. */
typedef struct ets_page_buffer {
  void* data;
  int64_t page_bytes;
} ets_page_buffer;

/* Page dst[i] of every buffer becomes page src[i], i < n.  Pairs with a number
 * outside [0, P) are skipped; the destinations of one call differ from each
 * other and from its sources.  n times the buffers' pieces of 16 KB of a page is
 * at most 2^31 - 1, here and for the branches of a fork. */
ets_status ets_pages_copy(const ets_page_buffer* buffers, int32_t count, int64_t P, const int32_t* src, const int32_t* dst,
                          int64_t n, void* stream);

/* Row b of the table [B][M] needs pages for positions [0, lens[b]): its first
 * ceil(lens[b] / page_size) entries, M at most.  Those that hold none get the
 * free pages, lowest first, in the order of the rows and their entries, and
 * refs 1.  Where no page is left they are -1, and lacking[b] counts them. */
ets_status ets_pages_workspace_size(int64_t P, int64_t rows, size_t* bytes);
ets_status ets_pages_extend(int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, const int32_t* lens,
                            int32_t page_size, int32_t* lacking, void* workspace, size_t workspace_bytes, void* stream);

/* Row b keeps its pages for positions [0, lens[b]); its other entries become
 * -1, and the pages they held lose one from refs. */
ets_status ets_pages_free(int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, const int32_t* lens,
                          int32_t page_size, void* stream);

/* Row i < n of out [n][out_M] becomes a branch of row b = parents[i] of the table: it
 * shares the pages that lens[b] positions fill, which gain one in refs each.
 * A last page that they fill in part is copied, in every buffer, to a free one
 * (lowest first, in order of i); lacking[i] is 1 where there was none, else
 * 0.  The other entries are -1, and so are those whose parent's hold no page,
 * and all where parents[i] is outside [0, B).  A branch has its first out_M
 * pages alone: what lies behind them is not shared, not copied, and lacking
 * does not count it.  What out held before is not looked at; an out that shares
 * an entry with the table's rows is refused (ETS_ERR_INVALID_ARG). */
ets_status ets_pages_fork(int32_t* refs, int64_t P, const int32_t* table, int64_t pt_b, int32_t B, int32_t M,
                          const int32_t* lens, int32_t page_size, const int32_t* parents, int32_t n, int32_t* out,
                          int64_t out_b, int32_t out_M, int32_t* lacking, const ets_page_buffer* buffers, int32_t count,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Draws the pool together: of the u pages in use, those numbered u or more
 * move, lowest first, to the free ones under u, lowest first, in every buffer,
 * with their refs; the table's entries follow (those that hold a free page
 * become -1).  moved int32 [P]: each page's new number, -1 for free ones. */
ets_status ets_pages_compact(int32_t* refs, int64_t P, int32_t* table, int64_t pt_b, int32_t B, int32_t M, int32_t* moved,
                             const ets_page_buffer* buffers, int32_t count, void* workspace, size_t workspace_bytes,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ETS_SPECULATE_H */
