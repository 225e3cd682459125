/*
 * dlrm_history.h -- C ABI of the event-history operators (GB300, sm_103a).
 *
 * Beside the sum-pooled bags of dlrm_sparse.h a recommendation model reads a
 * user's past events by attention: keys and values of the stored events lie
 * in a paged cache, and new events (in order, each seeing those before it) or
 * candidate items (each seeing the whole history) attend over it; the
 * attended vectors enter the interaction like pooled ones.  The operators:
 *   1. per-head norm of queries and keys with the position rotation in the
 *      same pass, and its gradient (training);
 *   2. appending new keys and values to the cache, normed and rotated on the
 *      way (serving);
 *   3. attention of the new tokens over the cache, from one token per
 *      sequence to long chunks.
 *
 * The conventions are those of dlrm_sparse.h: device pointers owned by the
 * caller, no device allocation, asynchronous on the caller's stream, host
 * checks before any launch, data-dependent errors as bits in an optional
 * device flag (read with dlrm_read_error), no kernel faults on bad data.
 * The structs below are host structs, read during the call.  Strides are in
 * elements; the d elements of a head row are contiguous.  Inputs may share
 * rows (a stride of 0); the rows of an output lie apart (strides of at least d
 * where there is more than one; DLRM_ERR_INVALID_ARG otherwise) and must not
 * overlap the inputs, but for the norms, their gradient and the append's queries
 * in place: q_out may be q and k_out may be k, dq may be q or dq_out and dk may
 * be k or dk_out, with the same pointer and strides.
 */
#ifndef DLRM_HISTORY_H
#define DLRM_HISTORY_H

#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head width of these calls. */
#define DLRM_MAX_HEAD_DIM 256

/* Rows of heads: row (token i, head h) starts at
 * ptr + i*token_stride + h*head_stride. */
typedef struct dlrm_heads {
    void *ptr;            /* device */
    int64_t token_stride; /* >= 0 */
    int64_t head_stride;  /* >= 0 */
    int32_t heads;        /* >= 1 */
} dlrm_heads;

/* Which elements turn together: i and i + rot/2, or 2i and 2i + 1. */
#define DLRM_ROPE_HALF 0
#define DLRM_ROPE_INTERLEAVED 1

/* The position rotation.  Row p of the table holds the cosines of position
 * p's rot/2 angles, then their sines; the caller makes it once.  Elements
 * from rot on are not turned. */
typedef struct dlrm_rope {
    const float *table;       /* device [length][rot], 4-byte aligned */
    int64_t length;           /* positions in the table */
    const int64_t *positions; /* device [n]; may be NULL in dlrm_kv_append */
    int32_t rot;              /* even, 2 .. d */
    int32_t layout;           /* DLRM_ROPE_HALF or DLRM_ROPE_INTERLEAVED */
} dlrm_rope;

/* A paged cache.  Slot t of page p holds, for head h, the key at
 * k + p*page_stride + t*slot_stride + h*head_stride (the value at the same
 * place from v), so both [pages][page_size][heads][d] and
 * [pages][heads][page_size][d] are described. */
typedef struct dlrm_kv_cache {
    void *k, *v;          /* device */
    int64_t pages;        /* 1 .. 2^31 - 1 */
    int64_t page_stride, slot_stride, head_stride;
    int32_t page_size;    /* slots of a page, 1 .. 65536 */
    int32_t heads;        /* key/value heads */
} dlrm_kv_cache;

/* A ragged batch of S sequences with n new tokens in all.  The new tokens of
 * sequence s are offsets[s] .. offsets[s+1]; lengths[s] tokens are (or, for
 * dlrm_kv_append, will be) stored; position j of the history lies in slot
 * j % page_size of page page_table[s*table_stride + j / page_size].  A length
 * beyond table_width * page_size or below 0, or offsets that are not monotone
 * within 0 .. n, raise DLRM_FLAG_BAD_OFFSETS and that sequence is left out
 * (nothing of it is written), whether it has new tokens or not.  offsets[0] is 0
 * and offsets[S] is n: else the flag is raised too, and what no sequence owns is
 * left out.  Where offsets fall, a token's sequence may not be found, and sequences
 * that are sound by themselves may be left out too, in part.  (A call with n = 0
 * launches nothing and checks none of this.) */
typedef struct dlrm_kv_batch {
    int64_t S;                 /* sequences, 0 .. 2^24 */
    int64_t n;                 /* new tokens, 0 .. 2^31 - 1 */
    const int64_t *offsets;    /* device [S + 1] */
    const int64_t *lengths;    /* device [S] */
    const int32_t *page_table; /* device, rows of table_width page numbers */
    int64_t table_stride, table_width; /* at most 2^30 positions in a row */
} dlrm_kv_batch;

/*
 * Norm and rotation of query and key heads.  For each row x (d elements):
 *
 *   z = x * w / sqrt(mean(x^2) + eps)      (z = x where the weight is NULL)
 *   y = z, with each pair (a, b) of its first rot elements turned:
 *       (a c - b s, b c + a s),  c, s from rope row positions[i]
 *
 * all in fp32, rounded once to dtype.
 * q, k            inputs; k and k_out may be NULL (queries alone).
 * n, d            tokens; head width, 1 .. DLRM_MAX_HEAD_DIM.
 * dtype           DLRM_F32, DLRM_F16 or DLRM_BF16, of q, k, q_out and k_out.
 * q_weight, k_weight  device fp32 [d], or NULL: no norm.
 * eps             >= 0 and finite.  Without one, rows whose mean square is
 *                 subnormal in fp32 count as zeros.
 * rope            NULL: no rotation.
 * A position outside the table raises DLRM_FLAG_INDEX_OOB and that token's
 * outputs are zeros.  Rows of a multiple of 8 elements whose pointers and
 * strides are multiples of 4 elements, with rot a multiple of 8 and a 16-byte
 * aligned table, take the vector path.
 */
int dlrm_qk_norm_rope_fwd(const dlrm_heads *q, const dlrm_heads *k, int64_t n, int d, int dtype,
                          const float *q_weight, const float *k_weight, float eps, const dlrm_rope *rope,
                          const dlrm_heads *q_out, const dlrm_heads *k_out, int32_t *err_flag,
                          dlrm_stream_t stream);

/* Bytes of workspace of the gradient below; 0 for invalid sizes. */
size_t dlrm_qk_norm_rope_bwd_workspace_size(int64_t n, int q_heads, int k_heads, int d);

/*
 * Its gradient.  With dz = dy turned back, r = 1/sqrt(mean(x^2) + eps) and
 * g = dz * w:
 *
 *   dx = r (g - x r^2 mean(g x))           (dx = dz where the weight is NULL)
 *   dw = sum over tokens and heads of dz * x * r
 *
 * dq_out, dk_out   gradients of the outputs (dtype);  q, k  the inputs.
 * dq, dk           gradients of the inputs (dtype), overwritten.
 * dq_weight, dk_weight  device fp32 [d], overwritten; NULL: not computed.
 *                  They need their weight.
 * workspace        device, 16-byte aligned, of at least
 *                  dlrm_qk_norm_rope_bwd_workspace_size bytes.
 * The sums have a fixed order: results are the same bits from run to run.
 * A token whose position is outside the table gets zero gradients and adds
 * nothing to the weights' (flagged as above).
 */
int dlrm_qk_norm_rope_bwd(const dlrm_heads *dq_out, const dlrm_heads *dk_out, const dlrm_heads *q,
                          const dlrm_heads *k, int64_t n, int d, int dtype, const float *q_weight,
                          const float *k_weight, float eps, const dlrm_rope *rope, const dlrm_heads *dq,
                          const dlrm_heads *dk, float *dq_weight, float *dk_weight, void *workspace,
                          size_t workspace_bytes, int32_t *err_flag, dlrm_stream_t stream);

/*
 * Appends the batch's new tokens to the cache: new token i of sequence s goes
 * to position p = lengths[s] - (offsets[s+1] - offsets[s]) + i; its key heads
 * are normed (k_weight) and turned as above and stored in dtype, its value
 * heads are stored as they are.  The rotation uses position p, or
 * rope->positions[token] where given.
 * k, v             [n] tokens, as many heads as the cache.
 * q, q_out         optional (NULL): queries normed (q_weight) and turned in
 *                  the same launch.
 * dtype            of k, v, q, q_out and the cache.
 * More new tokens than the length raise DLRM_FLAG_BAD_OFFSETS and the
 * sequence is left out.  A page number outside 0 .. pages - 1 or a rotation
 * position outside the table raises DLRM_FLAG_INDEX_OOB and the token is not
 * stored (q_out is zeros in the second case).  Two tokens of one call must not
 * share a slot.
 */
int dlrm_kv_append(const dlrm_heads *k, const dlrm_heads *v, const dlrm_kv_batch *batch,
                   const dlrm_kv_cache *cache, int d, int dtype, const float *k_weight, float eps,
                   const dlrm_rope *rope, const dlrm_heads *q, const float *q_weight, const dlrm_heads *q_out,
                   int32_t *err_flag, dlrm_stream_t stream);

/* Bytes of workspace of dlrm_kv_attn_fwd for these sizes; 0 for invalid ones. */
size_t dlrm_kv_attn_workspace_size(int64_t S, int64_t n, int q_heads, int kv_heads, int d, int64_t max_new,
                                   int64_t max_len);

/*
 * Attention of the batch's new tokens over the cache.  Query i of sequence s
 * (c new tokens, length L) sees the positions lo <= j < hi:
 *
 *   hi = L - c + i + 1 with causal, else L;   lo = max(0, hi - window), 0 without a window
 *   p_j = softmax over j of scale * (q_i . k_j);   out_i = sum_j p_j v_j
 *   lse_i = log sum_j exp(scale * (q_i . k_j))                (natural logarithm)
 *
 * Query head h reads cache head h / (q_heads / cache heads).  A query that
 * sees nothing gets out = 0 and lse = -infinity; one with a NaN gets NaN in both.
 *
 * q, out     heads a multiple of the cache's; dtype is that of q, out and the
 *            cache.
 * scale      > 0, at most 2e38.
 * causal     0 or 1;  window  >= 0, 0 for none.
 * max_new, max_len  host bounds of the batch's new tokens per sequence and
 *            lengths, for the launch's shape; a sequence beyond them raises
 *            DLRM_FLAG_BAD_OFFSETS and its rows are not written.  The shape is
 *            one for all: long chunks and single tokens are faster in a call each
 *            (one of 2048 new and 256 of one, on 2000: 480 us, in two calls 236).
 * lse        optional (NULL) device fp32 [n][q_heads].
 * workspace  device, 16-byte aligned, dlrm_kv_attn_workspace_size bytes.
 *
 * Slots that no query sees (past the length, before the window, whole pages
 * outside it) may hold anything, NaN included, and their page numbers may be
 * invalid; stored tokens that some query sees are taken to be finite.  A page
 * number outside the cache in the seen range reads as a page of zeros and
 * raises DLRM_FLAG_INDEX_OOB.
 *
 * Scores, the softmax's maxima and sums and the output's sums are fp32.  The
 * products run on the tensor cores for heads of at most 256 16-bit or 128 fp32
 * elements whose widths, strides and pointers are multiples of 16 bytes; others
 * take a general kernel in fp32.  16-bit types: for up to 8 rows (max_new times the query heads
 * of a cache head) each weight p (relative to the row's running maximum) is carried in two
 * parts of that type, for more it is rounded to it, an error as large as the rounding of the
 * output itself; f16 weights are scaled to use that type's range, so this holds
 * down to 2^-25 of the row's largest weight, and smaller ones are rounded to
 * steps of at most 2^-35 of it.  fp32: operands are split in two TF32 parts, which carries
 * each product to about 2^-22 of its magnitude.  Results are the same bits from
 * run to run of one batch; a sequence's last bits may depend on which other
 * sequences are in its batch.  Every wait inside a kernel is bounded; one that
 * runs out raises DLRM_FLAG_WAIT_TIMEOUT (results then invalid).
 */
int dlrm_kv_attn_fwd(const dlrm_heads *q, const dlrm_kv_batch *batch, const dlrm_kv_cache *cache, int d, int dtype,
                     float scale, int causal, int64_t window, int64_t max_new, int64_t max_len,
                     const dlrm_heads *out, float *lse, void *workspace, size_t workspace_bytes,
                     int32_t *err_flag, dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_HISTORY_H */
