/*
 * qmv_cache.h -- a key / value cache of 8-bit or 4-bit blocks and the attention
 * that reads it: what stands between a decoder's q / k / v products and its o
 * product (qmv.h, qmv_layer.h).  Same library (libqmv.so), same conventions as
 * qmv.h: device pointers, caller-owned buffers, status codes and qmv_last_error,
 * streams, no allocation, no synchronization, graph capture.
 *
 * The cache.  Keys and values are held in the blocks of qmv.h's formats
 * QMV_Q8_0 (w = d q, q in -127 .. 127) or QMV_Q4_0 (w = d q, q in -8 .. 7, kept as
 * q + 8), a block being 32 values of one head of one token, d its f16 scale.
 * The cache is an array of pages of `page` tokens; page p of head h is the record
 * p * heads + h of qmv_kv_cache_bytes / (pages * heads) bytes.
 *
 * Layout, version 1: a record is page / 16 records of 16 tokens, in order, each
 * of four planes: K codes, V codes (C bytes per block, C = 512 for Q8_0, 256 for
 * Q4_0), K scales, V scales (32 bytes per block).  With nb = D / 32 blocks a head,
 * for token t of the 16 and dimension 32 b + e:
 *   K, Q8_0   byte 512 b + 8 (16 (e / 8) + t) + e % 8                     = q + 128
 *   K, Q4_0   byte 256 b + 4 (16 (e / 8) + t) + e % 4,                      q + 8 in its
 *             low (e % 8 < 4) or high four bits
 *   V, Q8_0   byte 512 b + 4 (2 (16 (t / 4) + e % 16) + e / 16) + t % 4    = q + 128
 *   V, Q4_0   byte 256 b + 4 (16 (t / 4) + e % 16) + t % 4,                 q + 8 in its
 *             low (e < 16) or high four bits
 *   scales    f16 number 4 (nb (t / 4) + b) + t % 4
 * (the order in which the matrix cores take them: 16 tokens and 32 dimensions of K,
 * or 16 dimensions and 4 tokens of V, are what a wave reads in one load).
 *
 * Quantising a block x (f32, round to nearest even, in this order):
 *   d = f16(min(max |x| / 127, 65504)), q = clamp(rint(x * (1 / d)), -127, 127)  (Q8_0)
 *   d = f16(min(max |x| / 7.5, 65504)), q = clamp(rint(x * (1 / d)), -8, 7)      (Q4_0)
 * and q = 0 where d = 0.  A block that holds a NaN or an infinity gets d = NaN:
 * it reads back as NaN, and so does the attention that sees its token.
 *
 * The batch.  The T rows of a call are tokens of B sequences: rows q_start[b] ..
 * q_start[b + 1] - 1 are the last ones of sequence b, which is kv_len[b] tokens long
 * with them (its kv_len[b] - 1 is the last row's position).  Position p of sequence
 * b is token p % page of page table[b][p / page].  q_start, kv_len and table lie on
 * the device and are read when the call runs, so a captured call follows them.
 * Rows before q_start[0] and from q_start[B] on belong to no sequence and are left as they are.  What does
 * not fit is absent, not read and not written: a page id outside 0 .. pages - 1, a
 * position past the table's columns, a position below 0 (more rows than kv_len).
 * q_start must not decrease (rows and positions are checked against T all the same).
 */
#ifndef QMV_CACHE_H_
#define QMV_CACHE_H_

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qmv_kv_cache {
  int32_t fmt;    /* QMV_Q8_0 or QMV_Q4_0 */
  int32_t page;   /* tokens of a page: a multiple of 16, <= 1024 */
  int64_t pages;  /* >= 1, <= 2^31 - 1 */
  int64_t heads;  /* of k and of v, >= 1, <= 65535 */
  int64_t D;      /* values of a head: a multiple of 32, <= 256 */
  void* data;     /* qmv_kv_cache_bytes bytes, device, 16-byte aligned */
} qmv_kv_cache;

typedef struct qmv_kv_batch {
  int64_t T;               /* rows of the call, >= 1 */
  int64_t B;               /* sequences, >= 1 */
  const int32_t* q_start;  /* [B + 1], device */
  const int32_t* kv_len;   /* [B], device */
  const int32_t* table;    /* page ids, device: row b starts at table + b * stride */
  int64_t columns;         /* entries of a row, >= 1; columns * page <= 2^30 */
  int64_t stride;          /* >= columns (or B = 1) */
} qmv_kv_batch;

/* Bytes of a cache; cache->data is not looked at.  Host only.  Errors: NULL,
 * FORMAT, SHAPE, OVERFLOW. */
int qmv_kv_cache_bytes(const qmv_kv_cache* cache, size_t* out_bytes);

/*
 * Writes the keys and values of T new tokens to their places in the cache,
 * quantised as above.  Nothing else of the cache changes.
 *   k, v   [T][heads][D] of dtype QMV_F32, QMV_F16 or QMV_BF16, aligned to the
 *          element, with strides in elements (values of a head adjacent)
 * A place that two sequences of the batch name in one call (pages that they share)
 * holds a mixture of both tokens afterwards.  Sequences that share pages write
 * behind them.
 * Errors: FORMAT, SHAPE, NULL, ALIGN, DTYPE, UNSUPPORTED (Q8X; k or v that is the
 * cache's buffer), OVERFLOW, DEVICE, LAUNCH.
 */
int qmv_kv_write(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const void* k, int64_t k_token, int64_t k_head,
                 const void* v, int64_t v_token, int64_t v_head, int dtype, void* stream);

/*
 * Reads the rows' keys and values back, d * q rounded once to dtype (whole
 * sequences with q_start the running sum of kv_len).  A row whose place is
 * absent gives zeros.  k and v as in qmv_kv_write; either may be NULL.
 * Errors: as qmv_kv_write; UNSUPPORTED also for outputs that hold values twice or
 * are one buffer.
 */
int qmv_kv_read(const qmv_kv_cache* cache, const qmv_kv_batch* batch, void* k, int64_t k_token, int64_t k_head, void* v,
                int64_t v_token, int64_t v_head, int dtype, void* stream);

typedef struct qmv_kv_attention_args {
  const void* q;      /* [T][q_heads][D] of dtype */
  void* out;          /* the same shape and dtype; no overlap with q unless it is q with q's strides */
  float* lse;         /* [T][q_heads], contiguous: ln(sum exp(s)) of each row, -inf where it is empty; NULL: not wanted */
  int64_t q_heads;    /* a multiple of the cache's heads; q head h reads head h / (q_heads / heads) */
  int64_t q_token, q_head, out_token, out_head; /* strides in elements */
  int32_t dtype;      /* QMV_F32, QMV_F16 or QMV_BF16 */
  float scale;        /* finite */
  int64_t window;     /* a row at position p sees p - window + 1 .. p; 0: 0 .. p */
  int64_t prefix;     /* the first `prefix` positions are the same pages in every sequence: they are read
                         once for all rows, through row 0 of the table; 0: nothing is shared */
  int64_t max_q;      /* the most rows and tokens that a sequence is expected to have: they shape the */
  int64_t max_kv;     /* launch (any value >= 1 gives right results, to f32 rounding) */
} qmv_kv_attention_args;

/*
 * Attention over the cache, causal by position: for every row, at position p of
 * its sequence, and q head h
 *   s_t = scale * q . K_t,  out = sum_t softmax(s)_t V_t
 * over the positions t <= p that the window leaves and that are there; a row
 * that sees nothing gives zeros.  The rows' own keys and values are read from the
 * cache too: write them first.  Scores, maxima, sums and accumulators are f32; the
 * products run on the 16-bit matrix cores:
 *   f32 and f16 calls: with K, V and the probabilities in operands of 22 bits (exact for K
 *   and V; two f16 parts), f32 queries too;
 *   bf16 calls: with the probabilities, and from 65 queries of a k / v head on (max_q rows of a
 *   sequence, or all rows over a prefix, times q_heads / heads) d * q of K and V, rounded
 *   once to f16 (11 bits against the result's 8; with an exponent of its own for
 *   every 32 tokens).
 * A row whose q holds a NaN or an infinity is NaN, and one that sees a block which reads
 * back as NaN (in K altogether; in V in that block's dimensions at least).  Masked and
 * absent positions do not enter, whatever the cache holds there.
 *   ws, ws_bytes   scratch memory, 16-byte aligned, of at least
 *                  qmv_kv_attention_bytes bytes (NULL if that is 0); calls that overlap
 *                  in time need a ws of their own
 * Calls repeat bit for bit with the same sizes, max_q, max_kv and prefix.
 * Errors: FORMAT, SHAPE, NULL, ALIGN, DTYPE, UNSUPPORTED, OVERFLOW, DEVICE, LAUNCH.
 */
int qmv_kv_attention(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const qmv_kv_attention_args* args, void* ws,
                     size_t ws_bytes, void* stream);

/* Bytes of scratch memory that qmv_kv_attention needs for these sizes; pointers,
 * strides, scale and window are not looked at.  Host only.  Errors: NULL, FORMAT,
 * SHAPE, DTYPE, UNSUPPORTED, OVERFLOW. */
int qmv_kv_attention_bytes(const qmv_kv_cache* cache, const qmv_kv_batch* batch, const qmv_kv_attention_args* args,
                           size_t* out_bytes);

#ifdef __cplusplus
}
#endif

#endif /* QMV_CACHE_H_ */
