/*
 * infini_attn_packed.h -- C ABI of the packed-sequence operators: causal
 * softmax attention with grouped heads, and the gated delta rule. They stand
 * beside the layer of infini_attn.h (whose segments are equal and whose q, k, v
 * have the same heads): a batch here is any number of sequences of any lengths
 * laid end to end, with fewer key heads than query (or value) heads allowed.
 *
 * Rows. A tensor of T tokens and H heads is an infini_rows: element c of token
 * t and head h is ptr[t * stride_t + h * stride_h + c], strides in elements, so
 * q, k and v may be slices of one projection's output and the heads may lie
 * outside the tokens. Every (t, h) of [0, T) x [0, H) must be inside the
 * allocation. Pointers are 16-byte aligned and strides positive multiples of 16
 * bytes (the stride of a dimension of size 1 is not used).
 *
 * Sequences. Sequence s has the rows off[s] .. off[s + 1] - 1 (int32, DEVICE,
 * n_seq + 1 values); with len not NULL (int32, DEVICE, n_seq values) only the
 * first len[s] of them, as in a padded batch or a cache. Lengths of zero are
 * fine. Rows of no sequence are not written, and nothing that they hold enters a
 * result; but they may be read (tiles run past a sequence's end), so they belong
 * to the allocation. An offset out of range (negative, behind T) leaves out the
 * sequences on both its sides, a length out of range (negative, longer than its
 * room) its own: their rows stay as they were in every output (a state is handed
 * through), the other sequences are computed as ever. Offsets that decrease may
 * leave out further sequences, or rows of them; what is computed is right all the
 * same. Each of these makes infini_attn_device_status() return INFINI_ERR_OFFSETS,
 * and none leads to an access out of range. Sequences that overlap in the outputs
 * are unspecified.
 *
 * Calls follow infini_attn.h: DEVICE pointers, asynchronous on `stream`, checked
 * on the host before anything is launched, no state between calls, no allocation
 * (a workspace of the size that the *_workspace_size functions give, 256-byte
 * aligned, not shared by calls in flight at the same time: two captured graphs
 * that may run at once need one each; a size of 256 stands for none needed, and
 * workspace may be NULL then). Shapes and infini_rows are HOST pointers,
 * read during the call only. Nothing a call writes may overlap its other
 * buffers (INFINI_ERR_ALIAS), except where a function says so; views that
 * interleave in one buffer ([T][n][H][d], [T][H][n][d], [H][T][n][d], [H][n][T][d])
 * are fine. No atomics enter a result: the same call gives the same bits.
 */
#ifndef INFINI_ATTN_PACKED_H
#define INFINI_ATTN_PACKED_H

#include "infini_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* More return codes. */
enum {
  INFINI_ERR_OFFSETS = -12 /* offsets or lengths on the device are out of range
                              (from infini_attn_device_status)                 */
};

/* More paths for the functions below. */
enum {
  INFINI_PATH_SPLIT = 4 /* attention only: the keys of a sequence split over CTAs and joined, for
                           few queries against many keys                                       */
};

typedef struct {
  void* ptr;
  int64_t stride_t;
  int64_t stride_h;
} infini_rows;

typedef struct {
  int64_t n_seq; /* sequences                                            >= 0 */
  int64_t Tq;    /* rows of q, out (and their gradients)                 >= 0 */
  int64_t Tk;    /* rows of k, v                                         >= 0 */
  int64_t Hq;    /* query heads, a multiple of Hkv                       >= 1 */
  int64_t Hkv;   /* key / value heads; query head h reads h / (Hq / Hkv) >= 1 */
  int64_t d;     /* 64 or 128                                                 */
  int64_t max_q; /* longest sequence's queries and keys, as the caller knows  */
  int64_t max_k; /* them (the choice of path and grid; results do not depend
                    on them beyond rounding)                                  */
  int32_t dtype; /* infini_dtype of all rows                                  */
  float scale;   /* of the scores, finite and > 0 (commonly 1 / sqrt(d))      */
} infini_packed_shape;

/* ------------------------------------------------------------ attention
 * Query i of a sequence with nq queries and nk keys sees the keys
 * j <= i + nk - nq (the last query sees every key: a whole prompt has nq == nk,
 * a step against a cache nq == 1):
 *   x_ij = scale q_i . k_j,  lse_i = log sum_j exp(x_ij),
 *   out_i = sum_j exp(x_ij - lse_i) v_j
 * A query that sees no key has out = 0 and lse = -inf (nq > nk, or nk == 0).
 * NaN scores are not that: a NaN in a query, or in a key that it sees, gives NaN
 * in its out and lse.
 *   q, out  rows [Tq][Hq][d];  k, v  rows [Tk][Hkv][d], in shp->dtype
 *   lse     [Hq][Tq] fp32, or NULL
 *   q_off, q_len, k_off, k_len  the sequences (q_len, k_len may be NULL)
 *   path    INFINI_PATH_AUTO, _SIMT (any shape), _TC (bf16) or _SPLIT
 * Scores, softmax statistics and sums are fp32. With bf16 rows the products run
 * on the tensor cores (exp(x - m) is rounded to bf16 for the product with v).
 * A non-finite element of v at a key that a query does not see may still reach
 * that query if the two lie in one tile of a sequence (in the gradients one of q, k,
 * v or dout); rows behind a sequence's length never do. */
INFINI_API size_t infini_attn_packed_workspace_size(const infini_packed_shape* shp, int path);
INFINI_API int infini_attn_packed_select_path(const infini_packed_shape* shp);
INFINI_API int infini_attn_packed_forward(const infini_packed_shape* shp, const infini_rows* q, const infini_rows* k,
                                          const infini_rows* v, const int32_t* q_off, const int32_t* k_off,
                                          const int32_t* q_len, const int32_t* k_len, const infini_rows* out,
                                          float* lse, void* workspace, size_t workspace_bytes, int path,
                                          infini_stream_t stream);

/* Gradients, with out and lse as the forward gave them:
 *   D_i = dout_i . out_i,  p_ij = exp(x_ij - lse_i),  ds_ij = scale p_ij (dout_i . v_j - D_i)
 *   dq_i = sum_j ds_ij k_j,  dk_j = sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i
 * dk and dv are summed over the query heads of their group in a fixed order. dq,
 * dk, dv: rows in shp->dtype, written for every row of a sequence (zero where
 * nothing is seen). path: INFINI_PATH_AUTO, _SIMT or _TC (bf16; p and ds are
 * rounded to bf16 for their products). */
INFINI_API size_t infini_attn_packed_backward_workspace_size(const infini_packed_shape* shp);
INFINI_API int infini_attn_packed_backward(const infini_packed_shape* shp, const infini_rows* q, const infini_rows* k,
                                           const infini_rows* v, const infini_rows* out, const float* lse,
                                           const infini_rows* dout, const int32_t* q_off, const int32_t* k_off,
                                           const int32_t* q_len, const int32_t* k_len, const infini_rows* dq,
                                           const infini_rows* dk, const infini_rows* dv, void* workspace,
                                           size_t workspace_bytes, int path, infini_stream_t stream);

/* ------------------------------------------------------ gated delta rule
 * A memory that forgets by a gate and overwrites what a key held before: per
 * sequence and value head h (key head h / (Hv / Hk)), with a_t = exp(g_t),
 *   S' = a_t S_{t-1},  u_t = beta_t (v_t - S'^T k_t),
 *   S_t = S' + k_t u_t^T,  out_t = scale S_t^T q_t
 *   q, k     rows [T][Hk][d];  v, out  rows [T][Hv][d], in shp->dtype
 *   g, beta  [T][Hv] in shp->dtype (infini_rows with d = 1: any positive
 *            strides, element alignment). g is the log of the decay (<= 0 as a
 *            rule; below -200, -inf included, it counts as -200: the state is
 *            dropped; NaN does not, it makes the state NaN). The keys are used
 *            as they are: for a memory that stays bounded they have norm 1 and
 *            0 <= beta <= 1.
 *   S_in, S_out  [n_seq][Hv][d][d] fp32 (S[i][j]: key dimension i, value
 *            dimension j); S_in NULL = zero, S_out NULL = not wanted, S_out may
 *            equal S_in. A sequence of length 0 hands its state through.
 *   off, len the sequences (len may be NULL)
 *   path     INFINI_PATH_AUTO, _SIMT or _TC (bf16, the chunked form on the
 *            tensor cores)
 * States, decays and the solve inside a chunk are fp32 (logs of decays are
 * summed in 64 bits). With INFINI_PATH_SIMT so are all products; with _TC those that
 * enter a state have 16 or more bits in each factor (states 4e-6 off by norm, 1e-7
 * with _SIMT). An element that is not finite may reach every row of its
 * sequence, the ones before it too, and no other sequence. At most 65535
 * sequences, and states of a one-token step, to a call. */
typedef struct {
  int64_t n_seq;   /* sequences                          >= 0 */
  int64_t T;       /* rows                               >= 0 */
  int64_t Hk;      /* query / key heads                  >= 1 */
  int64_t Hv;      /* value heads, a multiple of Hk      >= 1 */
  int64_t d;       /* 64 or 128, of keys and values           */
  int64_t max_len; /* longest sequence, as the caller knows it (the choice of path;
                      results do not depend on it beyond rounding)            */
  int32_t dtype;
  float scale;     /* of the output, finite */
} infini_delta_shape;

INFINI_API size_t infini_attn_delta_workspace_size(const infini_delta_shape* shp, int path);
INFINI_API int infini_attn_delta_forward(const infini_delta_shape* shp, const infini_rows* q, const infini_rows* k,
                                         const infini_rows* v, const infini_rows* g, const infini_rows* beta,
                                         const int32_t* off, const int32_t* len, const float* S_in,
                                         const infini_rows* out, float* S_out, void* workspace,
                                         size_t workspace_bytes, int path, infini_stream_t stream);

/* Gradients of the above for dout and dS_out (NULL = zero): dq, dk, dv, dg,
 * dbeta in shp->dtype and dS_in fp32 (NULL = not wanted; may equal dS_out). The
 * states are computed again. Where g is cut at -200 dg is that of the decay
 * e^-200. With INFINI_PATH_TC a |beta| below 2^-110 counts as 2^-110 with its sign,
 * and as 0 in dv. */
INFINI_API size_t infini_attn_delta_backward_workspace_size(const infini_delta_shape* shp, int path);
INFINI_API int infini_attn_delta_backward(const infini_delta_shape* shp, const infini_rows* q, const infini_rows* k,
                                          const infini_rows* v, const infini_rows* g, const infini_rows* beta,
                                          const int32_t* off, const int32_t* len, const float* S_in,
                                          const infini_rows* dout, const float* dS_out, const infini_rows* dq,
                                          const infini_rows* dk, const infini_rows* dv, const infini_rows* dg,
                                          const infini_rows* dbeta, float* dS_in, void* workspace,
                                          size_t workspace_bytes, int path, infini_stream_t stream);

/* One token for each of shp->T sequences (n_seq and max_len are not used): row b
 * of q, k, v, g, beta with state b. S_in, S_out: [T][Hv][d][d] fp32, S_out may
 * equal S_in (and then updates it in place). */
INFINI_API int infini_attn_delta_step(const infini_delta_shape* shp, const infini_rows* q, const infini_rows* k,
                                      const infini_rows* v, const infini_rows* g, const infini_rows* beta,
                                      const float* S_in, const infini_rows* out, float* S_out,
                                      infini_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* INFINI_ATTN_PACKED_H */
