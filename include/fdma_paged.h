/*
 * fdma_paged.h -- C ABI of libfdma's paged key/value cache: writing new tokens
 * into the cache (bf16, or quantised to e4m3), reading sequences back, and
 * attention of the newest tokens of each sequence over its pages.
 *
 * The conventions of fdma.h hold: device pointers are the caller's, nothing is
 * allocated or retained, every call is asynchronous on `stream`, argument errors
 * return a status before anything is launched, no function throws or aborts.
 *
 * The cache.  Position p of sequence b is slot p % page_size of page
 * page_table[b][p / page_size].  A page holds page_size tokens' K and V rows of
 * every kv head, addressed by strides, so (page, token, head, d) and
 * (page, head, token, d) memory orders are both possible.
 *
 *   FDMA_CACHE_BF16   rows of d bf16 values
 *   FDMA_CACHE_E4M3   rows of d e4m3 codes and one byte e per (token, kv head)
 *                     and tensor: the row's values are code * 2^(e - 127).
 *                     A row x is written with the least e for which
 *                     max |x| <= 448 * 2^(e - 127), 1 <= e <= 246 (the largest
 *                     finite |x| where x has infinities, which become
 *                     +-448 * 2^(e - 127); NaN stays NaN), each value rounded
 *                     once, to nearest even.  The scale is a power of two, so
 *                     the values read back are exact in bf16 where they are multiples of its least
 *                     step, 2^-133, as all are from e = 3 on (else rounded once more).  Bytes that
 *                     are not written (0, 247 to 255) read as the nearest one that is.
 *
 * Several sequences are packed along one token axis: sequence b owns tokens
 * cu[b] .. cu[b+1]-1 (cu is non-decreasing, cu[0] >= 0).  k_len[b] counts the
 * sequence's keys INCLUDING its new tokens, in every call: new token i of n is at
 * position k_len[b] - n + i.  One set of cu, k_len and page_table so serves the
 * write of a step's tokens and the attention over them.
 *
 * What only the device sees (cu, k_len, page_table) is checked there: a page
 * number outside [0, num_pages), a k_len outside [0, max_pages * page_size], a
 * token range outside [0, T) or a position outside the sequence's pages is never
 * dereferenced; the tokens it stands for are left out (their rows or slots stay as they are, all
 * other tokens keep their positions), keys of a page that is not
 * there read as zeros, and fdma_get_device_error() returns FDMA_ERR_INVALID.  Entries of page_table that
 * no position below k_len needs are not looked at.
 */
#ifndef FDMA_PAGED_H_
#define FDMA_PAGED_H_

#include "fdma.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FDMA_CACHE_BF16 = 0, FDMA_CACHE_E4M3 = 1 } fdma_cache_type;

typedef struct fdma_kv_cache {
  int32_t B;          /* sequences (at most 2^30): rows of page_table, entries of k_len */
  int32_t Hkv, d;     /* kv heads (at most 2^20); head dim, a multiple of 8 (bf16) or 16 (e4m3), at most 128 */
  int32_t cache_type; /* fdma_cache_type */
  int32_t num_pages;  /* pages of k and v */
  int32_t page_size;  /* tokens of a page: a power of two, 16 to 4096 */
  int32_t max_pages;  /* entries of a page_table row */

  /* rows of d contiguous elements; strides (page, token, head) in ELEMENTS, multiples of 16
     bytes, none negative; base 16-byte aligned */
  void* k;
  int64_t k_stride[3];
  void* v;
  int64_t v_stride[3];
  /* FDMA_CACHE_E4M3: scale bytes; strides (page, token, head) in bytes, none negative */
  uint8_t* k_exp;
  int64_t k_exp_stride[3];
  uint8_t* v_exp;
  int64_t v_exp_stride[3];

  const int32_t* page_table; /* (B, max_pages), rows table_stride entries apart */
  int64_t table_stride;
  const int32_t* k_len; /* (B) */
} fdma_kv_cache;

typedef struct fdma_paged_args {
  fdma_kv_cache cache;

  /* q (T, Hq, d) bf16: strides (token, head) in elements, multiples of 8, d contiguous, base
     16-byte aligned.  Query head h reads kv head h / (Hq / Hkv).  T may exceed cu_q[B]: the
     rows behind the last sequence are neither read nor written. */
  int32_t T, Hq;
  const void* q;
  int64_t q_stride[2];
  const int32_t* cu_q; /* (B + 1) */
  int32_t max_q;       /* at least the longest sequence's new tokens (rows past it are left out and
                          reported as FDMA_ERR_INVALID by fdma_get_device_error; 0: nothing is done) */

  int32_t causal; /* 1: the row at position p sees keys j <= p; 0: all k_len[b] keys */
  int32_t window; /* > 0 (causal only): of those, j > p - window or j < sinks; 0: no window */
  int32_t sinks;  /* first tokens that stay visible to every later row (ignored without a window) */
  float scale;    /* multiplies q.k; > 0, and finite times log2(e) */

  void* workspace; /* >= fdma_paged_workspace_size() bytes, 256-byte aligned; holds nothing between
                      calls.  Calls that may run at the same time (two streams, two captured graphs)
                      need one each. */
  size_t workspace_bytes;
} fdma_paged_args;

/* Writes k_new and v_new ((T, Hkv, d) bf16; strides (token, head) in elements, multiples of 8, d
   contiguous, bases 16-byte aligned) of the tokens cu[0] .. cu[B]-1 into the cache.  The slots of
   one call must be distinct (a page that several sequences share is written by none of them), and
   none may hold a row of k_new or v_new.
   All else in the cache is left as it is. */
FDMA_API int fdma_kv_append(const fdma_kv_cache* cache, const void* k_new, const int64_t k_new_stride[2],
                            const void* v_new, const int64_t v_new_stride[2], const int32_t* cu, int T, void* stream);

/* Reads positions first[b] + i (i = 0 .. cu[b+1]-cu[b]-1; first NULL: 0) of every sequence into
   rows cu[b] + i of k_out and v_out, (T, Hkv, d) bf16 contiguous, 16-byte aligned.  Positions
   outside [0, k_len[b]) read as zeros (so cu = b * N gives sequences padded to N rows), as do, where
   k_len[b] is out of range, positions that the table does not reach; rows behind cu[B] are left as they are. */
FDMA_API int fdma_kv_gather(const fdma_kv_cache* cache, const int32_t* cu, const int32_t* first, int T, void* k_out,
                            void* v_out, void* stream);

/* Bytes of workspace that fdma_paged_fwd needs for these sizes (0: invalid sizes).  It depends on
   B, T, Hq, Hkv, d and max_q alone, not on what the device arrays hold. */
FDMA_API size_t fdma_paged_workspace_size(const fdma_paged_args* args);

/* Attention of the tokens cu_q[0] .. cu_q[B]-1 over the cache:
     S = scale * <q, k_j> for the visible keys j,  out = softmax(S) V  (bf16 (T, Hq, d) contiguous),
     lse = log sum exp S  (fp32 (Hq, T) contiguous).
   A row that sees no key gets out = 0 and lse = -inf.  Keys that a row does not see do not reach
   it, whatever they hold.  Precision: products in fp32 from the bf16 (or exact e4m3) values, the
   softmax in fp32; for the product with V the weights are rounded to bf16.  With an e4m3 cache and at most 16 rows
   (max_q * Hq / Hkv) they are rounded to f16, relative to the row's largest: to 11 bits or 2^-24; or, for a row that
   sees value scales more than 2^16 apart, not at all.
   Sums of weights (up to 2^8 in a chunk) times values are divided at the end: they have to stay finite in fp32.
   (A sequence's rounding so depends on max_q, the longest one's tokens in a serving batch.)
   Deterministic: the same call gives the same bits.  A call of more than 2^30 steps of 128 keys an SM does
   nothing, and fdma_get_device_error() returns FDMA_ERR_UNSUPPORTED. */
FDMA_API int fdma_paged_fwd(const fdma_paged_args* args, void* out, float* lse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FDMA_PAGED_H_ */
