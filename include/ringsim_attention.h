/*
 * ringsim_attention.h -- C ABI of libringsim's attention-step operators: what
 * a rank runs between the norm in front of its projections and the all-reduce
 * behind them, on device tensors of one MI355X (gfx950).
 *
 *   - ringsim_rotary: rotary positions of queries and keys, and, with
 *     `inverse`, their gradient;
 *   - ringsim_kv_append: keys, turned on the way, and values into a paged
 *     cache held in 4 bits; ringsim_kv_read: the values that it holds;
 *   - ringsim_paged_attention: softmax attention over that cache, for single
 *     tokens, several tokens a sequence, and prompts.
 *
 * The conventions are those of ringsim_ops.h: arguments are checked on the
 * host and refused before anything is enqueued; calls are asynchronous on
 * `stream`, allocate nothing, enqueue kernel launches only (so they may be
 * captured), and give the same bits for the same call on the same values.
 * What lies in device memory cannot be checked on the host: indices there
 * that lead outside their tensor are left out by the kernels, as said at each
 * call, and never followed.
 *
 * Element types are RINGSIM_FLOAT32, RINGSIM_BFLOAT16 and RINGSIM_FLOAT16;
 * index types RINGSIM_INT32 and RINGSIM_INT64. Tokens are an [outer, inner]
 * array; rows of a token's heads are a [outer, inner, heads, dim] array whose
 * last dimension is contiguous, with strides {outer, inner, head} in elements.
 */
#ifndef RINGSIM_ATTENTION_H
#define RINGSIM_ATTENTION_H

#include "ringsim_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest head that is turned. */
#define RINGSIM_ROTARY_MAX_DIM 2048

/* Arguments of ringsim_rotary. */
typedef struct {
  const void* x;             /* dtype */
  void* out;                 /* dtype; may be x itself (same address, same strides) */
  const void* positions;     /* position_dtype, [outer, inner] */
  const double* frequencies; /* `pairs` of them, in radians a position, contiguous */
  int64_t x_stride[3];
  int64_t out_stride[3];
  int64_t position_stride[2];
  int64_t outer;
  int64_t inner;
  int64_t heads;
  int64_t dim;               /* 1 .. RINGSIM_ROTARY_MAX_DIM */
  int64_t pairs;             /* 0 .. dim / 2: the first 2 * pairs columns are turned */
  int dtype;
  int position_dtype;
  int interleaved;           /* 0: column i goes with i + pairs; 1: 2 i with 2 i + 1 */
  int inverse;               /* 1: the transposed rotation, which is the gradient */
  float scale;               /* of the turned columns, finite */
} ringsim_rotary_t;

/* Turns pair i of every head of a token at position p by the angle
 * t = p * frequencies[i]:
 *     a' = scale * (a cos t - b sin t)
 *     b' = scale * (b cos t + a sin t)
 * (with `inverse` by -t) and copies the columns behind the pairs. Angles are
 * formed and reduced in 64 bits, so that far positions keep their places on
 * the circle, and then rounded to fp32; the rotation is in fp32, rounded once. */
ringsim_result_t ringsim_rotary(const ringsim_rotary_t* args, ringsim_stream_t stream);

/* Tokens a page holds at most; pages hold a power of two of at least 16. */
#define RINGSIM_KV_MAX_PAGE 1024
/* Positions of a sequence that attention reads at most: 2^31 - 1024. */
#define RINGSIM_ATTENTION_MAX_LENGTH 2147482624

/* A paged cache of keys and values in 4 bits, in device memory. Of every
 * page, head and token the values of two neighbouring columns share a byte,
 * the even column in its low half, as sign, two bits of exponent and one of
 * mantissa (0, 0.5, 1, 1.5, 2, 3, 4, 6); each 32 columns have one exponent
 * byte s and stand for their values times 2^(s - 127). s is 1 to 252, or 255
 * where the 32 are NaN; what a token sees of other bytes is undefined, finite
 * or not, and what it does not see may be anything.
 *   keys, values             [pages, heads, page_size, dim / 2]
 *   key_scales, value_scales [pages, heads, dim / 32, page_size]
 * The last two dimensions of each are contiguous; pages and heads are strides
 * apart, in bytes and multiples of 16. */
typedef struct {
  uint8_t* keys;
  uint8_t* values;
  uint8_t* key_scales;
  uint8_t* value_scales;
  int64_t stride[2];         /* {page, head} of keys and values */
  int64_t scale_stride[2];   /* {page, head} of the scales */
  int64_t pages;
  int64_t heads;
  int64_t page_size;         /* a power of two, 16 .. RINGSIM_KV_MAX_PAGE */
  int64_t dim;               /* 64, 96, 128, 192 or 256 */
} ringsim_kv_cache_t;

/* Arguments of ringsim_kv_append. Slot n is token n % page_size of page n /
 * page_size. */
typedef struct {
  ringsim_kv_cache_t cache;
  const void* k;             /* dtype, [outer, inner, heads, dim] */
  const void* v;
  const void* slots;         /* slot_dtype, [outer, inner] */
  const void* positions;     /* position_dtype, [outer, inner]; not read where pairs is 0 */
  const double* frequencies; /* as in ringsim_rotary_t */
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t slot_stride[2];
  int64_t position_stride[2];
  int64_t outer;
  int64_t inner;
  int64_t pairs;             /* 0: keys are stored as they are */
  int dtype;
  int slot_dtype;
  int position_dtype;
  int interleaved;
  float scale;
} ringsim_kv_append_t;

/* Turns every token's keys as ringsim_rotary does, and stores them and the
 * values in their slot. Of each 32 columns w the exponent is the least e >=
 * -126 with max|w| <= 7 * 2^e, at most 125, and each value becomes the nearest
 * to w / 2^e that 4 bits hold, halfway cases going to the even mantissa: below
 * 7 none is further away than half the step there. A NaN or an infinity makes
 * its 32 columns NaN. Keys are turned in 64 bits and rounded to fp32 before
 * that, since a last bit may decide between two codes. A token whose slot is
 * negative or beyond the cache is left out. No slot may be given twice in a
 * call: what it holds afterwards would be parts of either token. */
ringsim_result_t ringsim_kv_append(const ringsim_kv_append_t* args, ringsim_stream_t stream);

/* Arguments of ringsim_kv_read. */
typedef struct {
  ringsim_kv_cache_t cache;
  void* k;                   /* dtype, [outer, inner, heads, dim]; NULL: not wanted */
  void* v;
  const void* slots;
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t slot_stride[2];
  int64_t outer;
  int64_t inner;
  int dtype;
  int slot_dtype;
} ringsim_kv_read_t;

/* The values that the cache holds for each token's slot; zeros for slots that
 * are negative or beyond the cache. fp32 and bf16 hold every value of the
 * cache; fp16 rounds, and overflows to infinity above 65504. */
ringsim_result_t ringsim_kv_read(const ringsim_kv_read_t* args, ringsim_stream_t stream);

/* Arguments of ringsim_paged_attention. */
typedef struct {
  ringsim_kv_cache_t cache;  /* read only */
  const void* q;             /* dtype, [tokens, heads, dim] */
  void* out;                 /* dtype, like q; must not overlap q */
  float* lse;                /* fp32, [tokens, heads], contiguous; NULL: not wanted */
  const int32_t* pages;      /* [seqs, max_pages]: where a sequence's tokens lie, rows page_stride apart */
  const int32_t* lengths;    /* [seqs]: a sequence's tokens in the cache, those of this call among them */
  const int32_t* starts;     /* [seqs + 1]: a sequence's tokens in q; NULL: tokens / seqs each */
  void* workspace;           /* ringsim_paged_attention_workspace bytes, 16-byte aligned */
  size_t workspace_bytes;
  int64_t q_stride[2];       /* {token, head} */
  int64_t q_seq_stride;      /* between the first tokens of sequences, read without `starts` */
  int64_t out_stride[2];
  int64_t out_seq_stride;
  int64_t page_stride;       /* between rows of `pages`, in elements */
  int64_t tokens;            /* of all sequences, padding behind them included */
  int64_t heads;             /* a multiple of cache.heads: neighbouring ones share a key head */
  int64_t seqs;
  int64_t max_pages;
  int64_t max_length;        /* no sequence is longer; 0: max_pages * page_size */
  int64_t window;            /* > 0: a token sees the last `window` positions, its own among them */
  int dtype;
  int causal;                /* 1: a token sees no position behind its own */
  float scale;               /* of the products q k, above 0 and below 2^119 */
} ringsim_paged_attention_t;

/* Attention of the last tokens of every sequence over its cached keys and
 * values. Token i of the n that sequence b has in q stands at position p =
 * lengths[b] - n + i and sees the positions j < lengths[b] with j <= p if
 * `causal` and j > p - window with a window; for each of its heads
 *     out = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q k_j)
 *     lse = log(sum_j w_j)
 * A token that sees nothing gets zeros and an lse of minus infinity. Rows of
 * q that belong to no sequence (before starts[0], from starts[seqs] on) are
 * not read, and their outputs stay as they are. `starts` must not decrease;
 * what leads outside q in it is cut off. Positions whose page is negative,
 * beyond the cache or beyond the table, and those from max_length (or
 * RINGSIM_ATTENTION_MAX_LENGTH) on, are left out. What the cache holds in
 * positions that a token does not see does not reach it, NaN and infinities
 * included.
 *
 * Products of keys with queries are taken in two to five parts of a query and
 * summed in fp32, infinite from 2^136 on; where the call's sizes give each key
 * many rows of bf16 or fp16 queries, products below 2^-13 of the largest one of
 * neighbouring columns may be left out, else and in fp32 below 2^-18 of it (also
 * with many rows where `lse` is wanted and max_length, or with `causal` the
 * window, leaves a token no more than 128 positions). Statistics and sums are
 * fp32, of weights up to 2^8: outputs of a token that sees n positions are finite
 * where their values are below 2^119 / n, and may be infinite or NaN beyond. The
 * weights go into the second product in bf16: for bf16 outputs rounded to it
 * where the call's sizes give each key many rows of queries, else in two parts;
 * in two parts for fp16, in three for fp32. lse is formed of the weights before
 * that, in fp32. */
ringsim_result_t ringsim_paged_attention(const ringsim_paged_attention_t* args, ringsim_stream_t stream);

/* Bytes of workspace that the call needs, which depend on its sizes only (0
 * where no context is split). Pointers are not read. Host only. */
ringsim_result_t ringsim_paged_attention_workspace(const ringsim_paged_attention_t* args, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* RINGSIM_ATTENTION_H */
