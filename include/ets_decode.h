/*
 * ets_decode.h -- C ABI of the operators around the selection in a sparse
 * decode step, for AMD MI355X (gfx950); part of libets_topk.so.
 *
 *   ets_rope          rotary positions of queries and keys
 *   ets_cache_write   quantises rows into an 8-bit cache
 *   ets_cache_read    reads rows of the cache back
 *   ets_index_scores  the indexer scores that the selection ranks
 *   ets_attend        attention over selected slots, or over whole paged
 *                     sequences, plus a tree of drafted tokens
 *
 * Cache format.  A cache is codes[S][H][D] (e4m3: sign, 4 bits of exponent
 * with bias 7, 3 of fraction, 0x7f and 0xff are NaN) and scales[S][H][D / 32]
 * (one byte a block of 32 values).  The value of a code c in a block with
 * scale byte s is c * 2^(s - 127).  ets_cache_write makes scale bytes from 1
 * to 246 and the other calls take no others.  D is a multiple of 32.
 *
 * Conventions shared by every call (those of ets_topk.h):
 *   - Array pointers are device memory of the caller; nothing is allocated,
 *     the host is never synchronised, work is enqueued on `stream`.
 *   - Arguments are checked on the host before anything is enqueued.  Slots
 *     are checked on the device: one outside [0, S) is skipped by the write,
 *     read as zeros, and not seen by scores and attention.
 *   - Strides are in elements (bytes for codes and scales); the innermost
 *     dimension is contiguous.  Strides from slot to slot of a cache that
 *     scores and attention read are at most 2^32 - 1.  No alignment beyond the element's is needed;
 *     rows that start at multiples of 16 bytes are the fast ones.
 *   - Results do not change from run to run.
 */
#ifndef ETS_DECODE_H
#define ETS_DECODE_H

#include "ets_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define ETS_BF16 0
#define ETS_FP16 1
#define ETS_FP32 2

/* pairs of a rotation */
#define ETS_ROPE_INTERLEAVED 0 /* channels (2i, 2i + 1) */
#define ETS_ROPE_HALF 1        /* channels (i, R / 2 + i) */

#define ETS_MAX_ROPE_DIM 4096   /* largest D of a rotation */
#define ETS_MAX_HEAD_DIM 576    /* largest D and Dv of attention */
#define ETS_MAX_INDEX_DIM 256   /* largest D of index scores */
#define ETS_MAX_INDEX_HEADS 128 /* largest H of index scores */
#define ETS_MAX_TREE 64         /* most drafted tokens of a sequence */
#define ETS_MAX_LENGTH 0x7ffff000 /* most positions of a sequence, slots of a list */

/*
 * Rotates channels [offset, offset + R) of x[N][H][D] and copies the others.
 * Pair i of row n, channels (a, b), turns by the angle positions[n] *
 * inv_freq[i]:
 *   out_a = scale * (x_a cos - x_b sin),  out_b = scale * (x_b cos + x_a sin).
 * `inverse` turns by the negative angle (and still multiplies by scale): the
 * transposed map, which takes a gradient with respect to out to the gradient
 * with respect to x.
 *   x, out     [N][H][D] of `dtype`, strides of n and h given; out may be x
 *              (the same pointer and strides), and must not overlap otherwise.
 *   positions  int32 [N].   inv_freq  double [R / 2], radians a position.
 *   R          even, 0 <= offset, offset + R <= D.
 * Angles, cosines and sines times scale are formed in 64 bits and rounded to
 * 32 once; products and sums are 32 bits.
 */
ets_status ets_rope(const void* x, int64_t x_n, int64_t x_h, void* out, int64_t out_n, int64_t out_h,
                    int64_t N, int32_t H, int32_t D, const int32_t* positions, const double* inv_freq,
                    int32_t R, int32_t offset, int32_t layout, double scale, int32_t inverse,
                    int32_t dtype, void* stream);

/*
 * codes[slots[n]][h], scales[slots[n]][h] <- x[n][h].  A block of largest
 * finite magnitude m gets the smallest exponent e in [-126, 119] with m <=
 * 448 * 2^e (-9 for a block of zeros) and the byte e + 127; its values are
 * x * 2^-e, rounded to nearest even and limited to +-448.  NaN stays NaN;
 * infinities become +-448 * 2^e.  Slots outside [0, S) are skipped; the slots
 * of one call are distinct.
 */
ets_status ets_cache_write(const void* x, int64_t x_n, int64_t x_h, int64_t N, int32_t H, int32_t D,
                           const int32_t* slots, uint8_t* codes, int64_t codes_s, int64_t codes_h,
                           uint8_t* scales, int64_t scales_s, int64_t scales_h, int64_t S,
                           int32_t dtype, void* stream);

/* out[n][h] (contiguous [N][H][D] of `dtype`) <- the values of
 * codes[slots[n]][h], rounded once; zeros for slots outside [0, S). */
ets_status ets_cache_read(const uint8_t* codes, int64_t codes_s, int64_t codes_h, const uint8_t* scales,
                          int64_t scales_s, int64_t scales_h, int64_t S, const int32_t* slots, int64_t N,
                          int32_t H, int32_t D, void* out, int32_t dtype, void* stream);

/*
 * out[b * T + t][p] = sum_h weights[b][t][h] * max(0, q[b][t][h] . key(b, p))
 * for positions p < min(seq_lens[b], L), minus infinity for the other p < L.
 * key(b, p) is the row of the cache's head 0 at slot page_table[b][p /
 * page_size] * page_size + p % page_size; a slot outside [0, S) scores minus
 * infinity.  Sums are held in 32 bits; products are exact, but with fp16
 * queries what lies beneath 2^-26 of a key's largest value (2^-33 in rows that
 * ets_cache_write made) is rounded.
 *   q        [B][T][H][D], bf16 or fp16.   weights  float [B][T][H].
 *   codes    row of slot s at s * codes_s.  D <= ETS_MAX_INDEX_DIM,
 *            H <= ETS_MAX_INDEX_HEADS, B <= 65535, L <= ETS_MAX_LENGTH.
 *   page_table int32 [B][>= ceil(L / page_size)], rows pt_b apart.
 *   out      float [B * T][out_stride >= L].
 */
ets_status ets_index_scores(const void* q, int64_t q_b, int64_t q_t, int64_t q_h, const float* weights,
                            int64_t w_b, int64_t w_t, int32_t B, int32_t T, int32_t H, int32_t D,
                            const uint8_t* codes, int64_t codes_s, const uint8_t* scales,
                            int64_t scales_s, int64_t S, const int32_t* page_table, int64_t pt_b,
                            const int32_t* seq_lens, int32_t page_size, int32_t L, float* out,
                            int64_t out_stride, int32_t dtype, void* stream);

/*
 * Attention of q[b][t][hq] over cached rows, hq = hk * (Hq / Hkv) + i sharing
 * head hk of the cache:
 *   x_j = D^-1/2 q . k_j over the rows j that (b, t) sees,
 *   out = sum_j softmax(x)_j v_j,  lse = log sum_j exp(x_j).
 * A row (b, t) that sees nothing has out = 0 and lse = -inf.  It sees
 *   - slots != NULL: the rows slots[b][t][0 .. K) (any order; a slot outside
 *     [0, S) is not seen); or
 *   - slots == NULL: positions p < min(seq_lens[b], L) of the sequence, at
 *     page_table[b][p / page_size] * page_size + p % page_size;
 *   - tree_slots != NULL: also tree_slots[b][j] for each j < T with bit j of
 *     tree_mask[b][t] set.
 * Scores (with products as in ets_index_scores), softmax statistics and output
 * sums are held in 32 bits: sums of p_j v_j with 0 <= p_j <= 1 and the largest
 * p_j at least 2^-24, so that they are finite where the sum of the values is,
 * and lose what lies beneath 2^-100 in values.  The p_j of these sums have 16
 * bits (two bf16 numbers).  A value or key that is NaN reaches the rows that
 * see it and no others.
 */
typedef struct ets_attend_args {
  int32_t B, T, Hq, Hkv, D, Dv;
  int32_t dtype;          /* of q and out: ETS_BF16 or ETS_FP16 */
  int32_t K;              /* selected: slots of a token, at most ETS_MAX_LENGTH */
  int32_t L;              /* paged: capacity of a sequence, at most ETS_MAX_LENGTH */
  int32_t page_size;      /* paged */
  int64_t S;              /* slots of the cache */
  const void* q;          /* [B][T][Hq][D] */
  int64_t q_b, q_t, q_h;
  const uint8_t* k_codes; /* [S][Hkv][D] */
  int64_t k_s, k_h;
  const uint8_t* k_scales;
  int64_t ks_s, ks_h;
  const uint8_t* v_codes; /* [S][Hkv][Dv] */
  int64_t v_s, v_h;
  const uint8_t* v_scales;
  int64_t vs_s, vs_h;
  const int32_t* slots;      /* [B][T][K] */
  int64_t slots_b, slots_t;
  const int32_t* page_table; /* [B][>= ceil(L / page_size)] */
  int64_t pt_b;
  const int32_t* seq_lens;   /* [B] */
  const int32_t* tree_slots; /* [B][T] */
  int64_t tree_b;
  const int64_t* tree_mask;  /* [B][T] */
  int64_t mask_b;
  void* out;                 /* contiguous [B][T][Hq][Dv] */
  float* lse;                /* contiguous [B][T][Hq] */
} ets_attend_args;

/* Bytes of workspace that the call needs on the current device (0 is
 * possible).  The contents do not matter before the call, and calls ordered
 * on one stream may share it. */
ets_status ets_attend_workspace_size(const ets_attend_args* args, size_t* bytes);
ets_status ets_attend(const ets_attend_args* args, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ETS_DECODE_H */
