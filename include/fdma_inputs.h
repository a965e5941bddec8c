/*
 * fdma_inputs.h -- C ABI of libfdma's operators on what goes into attention:
 * the norm of queries and keys for each head with the rotation of their
 * positions (forward, backward, and with the write into a paged cache for
 * serving), and a learned bias by buckets of the distance between query and key
 * with the gradient of its table.
 *
 * The conventions of fdma.h hold: device pointers are the caller's, nothing is
 * allocated or retained, every call is asynchronous on `stream`, argument errors
 * return a status before anything is launched, no function throws or aborts.
 */
#ifndef FDMA_INPUTS_H_
#define FDMA_INPUTS_H_

#include "fdma_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FDMA_FP32 = 0, FDMA_BF16 = 1 } fdma_param_type;

/* Rows of d contiguous bf16 values; strides (batch, token, head) in ELEMENTS, multiples of 8, none
   negative; base 16-byte aligned.  A batch stride is not looked at with one batch, and so on.  Rows that are
   written must not overlap: sorted, each stride has to step over all that the smaller ones reach. */
typedef struct fdma_rows {
  void* p;
  int64_t stride[3];
} fdma_rows;

/* With x a row (one token, one head), w its weight and t the angles of the token's position:
     y = x / sqrt(mean(x^2) + eps) * w                     (norm 0: y = x, and no weights)
     (a, b) -> (a cos t_i - b sin t_i, b cos t_i + a sin t_i)   for the rot / 2 pairs of y's first rot values:
   pair i is (y[i], y[i + rot / 2]), or (y[2 i], y[2 i + 1]) if interleaved; the others stay as they are.
   Everything is computed in fp32 and rounded once, to bf16. */
typedef struct fdma_norm_rope_args {
  int32_t B, N;   /* batches and tokens of each (packed tokens: B = 1); B * N at most 2^31 - 1 */
  int32_t Hq, Hk; /* heads of q (> 0) and of k (0: no k); at most 2^20 each */
  int32_t d;      /* a multiple of 8 from 8 to 256 */
  int32_t norm;   /* 1: norm, 0: rotation alone */
  float eps;      /* norm: > 0, finite */

  int32_t weight_type; /* fdma_param_type of both weights */
  /* d values, 16-byte aligned, or NULL (ones); (H, d) with the head stride in elements (a multiple of 8,
     at least d), or d for all heads with head stride 0.  Both weights are of one form, or one of them is NULL */
  const void* q_weight;
  int64_t q_weight_head;
  const void* k_weight;
  int64_t k_weight_head;

  const float* rope; /* (rope_len, 2, rot / 2) contiguous, 16-byte aligned: cosines and sines of each position's
                        angles.  NULL: no rotation */
  int32_t rope_len;
  int32_t rot;         /* a multiple of 8, at most d */
  int32_t interleaved; /* pairs: 0 halves, 1 adjacent */

  /* Positions.  NULL: token n of every batch is at first + n (checked against rope_len on the host).  Else int32 with
     strides (batch, token) in elements.  A token at a negative position is padding: it is left out (its rows of the outputs
     stay as they are; its gradients are 0).  So is one at or behind rope_len, and
     fdma_get_device_error() returns FDMA_ERR_INVALID. */
  int32_t first;
  const int32_t* positions;
  int64_t pos_stride[2];
} fdma_norm_rope_args;

/* q_out and k_out may be q and k themselves (same base and strides); other overlaps are the caller's mistake. */
FDMA_API int fdma_norm_rope(const fdma_norm_rope_args* args, const fdma_rows* q, const fdma_rows* k,
                            const fdma_rows* q_out, const fdma_rows* k_out, void* stream);

/* Bytes of workspace that fdma_norm_rope_bwd needs (0: invalid sizes). */
FDMA_API size_t fdma_norm_rope_bwd_workspace_size(const fdma_norm_rope_args* args);

/* From the gradients of the outputs: dq, dk (bf16; may be dq_out and dk_out themselves), and, where not NULL, the
   gradients of the weights, fp32, (d) or (H, d) contiguous like the weight (all written, zeros included; a weight
   that is NULL has none).  q and k are the forward's inputs (not read without norm, and may be NULL then).
   workspace: 256-byte aligned; calls that may run at the same time need one each.  It is not needed (size 0
   passes) where no weight's gradient is wanted.  Deterministic: sums run in a fixed order. */
FDMA_API int fdma_norm_rope_bwd(const fdma_norm_rope_args* args, const fdma_rows* q, const fdma_rows* k,
                                const fdma_rows* dq_out, const fdma_rows* dk_out, const fdma_rows* dq,
                                const fdma_rows* dk, float* dq_weight, float* dk_weight, void* workspace,
                                size_t workspace_bytes, void* stream);

/* fdma_norm_rope of packed new tokens (B = 1, N = T), q into q_out, and the keys, with v as it is, into the cache: as
   fdma_norm_rope followed by fdma_kv_append, in one launch.  positions NULL: each token's place in its sequence
   (first is not looked at).  An e4m3 cache takes its codes from the fp32 values of y, rounded once.  Tokens that the
   cache's plan or their position leaves out (see fdma_kv_append; a negative position is padding) leave q_out and the
   cache as they are.  Hk = Hkv of the cache, d as the cache's.  v, k and q must not lie in the slots that are
   written. */
FDMA_API int fdma_norm_rope_append(const fdma_norm_rope_args* args, const fdma_kv_cache* cache, const fdma_rows* q,
                                   const fdma_rows* k, const fdma_rows* v, const fdma_rows* q_out, const int32_t* cu,
                                   void* stream);

#define FDMA_MAX_BUCKETS 256 /* of one side */

/* A learned bias by distance: bias[h, i, j] = table[bucket(j - i - offset), h] for query row i at position i + offset
   and key j; h runs over kv heads, as in the bias that fdma_fwd takes.  One side (two_sided 0): the bucket of delta is that of the distance max(-delta, 0); two_sided: that of
   |delta|, plus num_starts where delta > 0.  A distance a is in the last bucket s with starts[s] <= a.  starts is a HOST
   array of num_starts values, copied by the call: starts[0] = 0, none smaller than the one before. */
typedef struct fdma_rel_args {
  int32_t H, Nq, Nk;  /* Nq, Nk at most 131072; Nk a multiple of 8 (as fdma_fwd wants it with a bias) */
  int32_t num_starts; /* buckets of a side, at most FDMA_MAX_BUCKETS; the table has them once, or twice if two_sided */
  int32_t two_sided;
  int32_t offset; /* position of query row 0 in the key sequence; |offset| <= 2^30 */
} fdma_rel_args;

/* table: (buckets, H) of table_type, element strides table_stride (bucket, head), none negative.  out: (H, Nq, Nk)
   bf16, element strides (head, row), multiples of 8, rows not overlapping, base 16-byte aligned. */
FDMA_API int fdma_rel_bias(const fdma_rel_args* args, const int32_t* starts, const void* table, int table_type,
                           const int64_t table_stride[2], void* out, const int64_t out_stride[2], void* stream);

/* Bytes of workspace that fdma_rel_bias_bwd needs for B batches (0: invalid sizes). */
FDMA_API size_t fdma_rel_bias_bwd_workspace_size(const fdma_rel_args* args, int B);

/* The table's gradient from that of the bias: dtable (buckets, H) fp32 contiguous, all written:
     dtable[s, h] = sum of dbias[b, h, i, j] over b and the (i, j) in bucket s.
   dbias: (B, H, Nq, Nk) bf16, element strides (batch, head, row), multiples of 8, none negative (0 repeats), base
   16-byte aligned.  causal 1: keys j > i + offset count as zeros, whatever is there, and most of them are not read
   (fdma_bwd writes zeros there for is_causal).  workspace: 256-byte aligned; calls that may run at the same time need one each.  Sums in fp32, in a
   fixed order: the same call gives the same bits. */
FDMA_API int fdma_rel_bias_bwd(const fdma_rel_args* args, const int32_t* starts, int B, const void* dbias,
                               const int64_t dbias_stride[3], int causal, float* dtable, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FDMA_INPUTS_H_ */
