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
 *      sequence to long chunks;
 *   4. the same cache in 8 bits: an append that encodes, and attention that reads
 *      the codes;
 *   5. pages and slots of a step's new tokens, given out on the device.
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

/*
 * A paged cache in 8 bits.  Keys and values are E4M3 codes (a sign, 4 bits of exponent, 3 of
 * mantissa; at most 448), laid out like those of dlrm_kv_cache, a byte an
 * element.  For each head, each `block` consecutive slots of a page share one exponent for their
 * keys and one for their values: the value of slot t's code c is
 * c * 2^(e - 127), with e the byte at k_exp (or v_exp)
 * + p*exp_page_stride + (t / block)*exp_block_stride + h*exp_head_stride.  0 stands for a block of zeros;
 * 248 .. 255 are never written, and what is read with them may overflow.
 */
typedef struct dlrm_kv_cache8 {
    void *k, *v;            /* device, codes */
    uint8_t *k_exp, *v_exp; /* device, exponents */
    int64_t pages;          /* 1 .. 2^31 - 1 */
    int64_t page_stride, slot_stride, head_stride;             /* of the codes */
    int64_t exp_page_stride, exp_block_stride, exp_head_stride; /* of the exponents */
    int32_t page_size;      /* slots of a page, 1 .. 65536 */
    int32_t heads;          /* key/value heads */
    int32_t block;          /* slots that share an exponent; divides page_size */
} dlrm_kv_cache8;

/*
 * Appends the batch's new tokens to a cache in 8 bits, at the places that
 * dlrm_kv_append says.  Keys are stored as they are given: dlrm_qk_norm_rope_fwd
 * norms and turns them first (with dlrm_kv_reserve's positions).
 *
 * Of each block that new tokens enter, with m the largest finite |x| of its new tokens in a
 * head and e the smallest exponent, at least 1, with m <= 448 * 2^(e - 127) (0 for m = 0):
 * - a block whose first slot is among the new ones gets e, whatever it held;
 * - one that holds older tokens of its sequence keeps the larger of e and its own; where e
 *   is larger, the older codes are rounded again.
 * A code is x * 2^(127 - e) rounded to nearest, ties to even.  Infinities become the
 * largest code and NaN its own code; neither counts for m.  The products with powers of two are exact, so
 * results are the same bits as those of this definition.
 *
 * k, v        [n] tokens, as many heads as the cache; dtype DLRM_F32, DLRM_F16 or DLRM_BF16.
 * Errors in the data are flagged and left out as by dlrm_kv_append.  Two sequences of a call must not add to
 * one block (pages that sequences share are read only).  Rows of a multiple of 8 elements, on 16 bytes, with
 * codes on 8, take the vector path.
 */
int dlrm_kv8_append(const dlrm_heads *k, const dlrm_heads *v, const dlrm_kv_batch *batch,
                    const dlrm_kv_cache8 *cache, int d, int dtype, int32_t *err_flag, dlrm_stream_t stream);

/* Bytes of workspace of dlrm_kv8_attn_fwd for these sizes, of any dtype; 0 for invalid ones.  The copy of long chunks'
 * codes (below) is among them, which may be large.  Calls that cannot make it (fp32, heads that are no multiple of 16 or
 * above 128, rows or codes that do not lie on 16 bytes) do without: for heads of up to 128 they need
 * dlrm_kv_attn_workspace_size bytes alone. */
size_t dlrm_kv8_attn_workspace_size(int64_t S, int64_t n, int q_heads, int kv_heads, int d, int64_t max_new,
                                    int64_t max_len);

/*
 * dlrm_kv_attn_fwd over a cache in 8 bits: the same masks, rows, outputs, bounds and errors;
 * dtype is that of q and out.  Slots that no query sees may hold any code and any exponent.
 *
 * Scores, the softmax's maxima and sums and the output's sums are fp32.  Where widths are multiples of
 * 8 and the rows of q, out and codes begin on 16 bytes, the products run on the tensor cores, 16-bit
 * types for heads of at most 256 elements, fp32 for at most 128, but on pages of no multiple of 8 slots
 * only 16-bit types with widths of multiples of 16.  Others take a general kernel in fp32.  On the tensor cores:
 * - a code is an fp16 value as it is; the power of its block multiplies scores and weights
 *   in fp32, or the code where that stays exact but for what lies 2^-41 below the largest value near by;
 * - 16-bit queries enter exactly (bf16 lifted by a power of two a row, but for what lies 2^-38 below the
 *   row's largest), fp32 ones in two parts, 22 bits;
 * - weights are rounded to fp16, in two parts for fp32 and for fp16 with up to 8 rows; relative to the
 *   largest weight times the largest power of the values so far, what lies below 2^-36 may be lost;
 * - long chunks of 16-bit types (of at least 1536 rows of heads of 65 to 128, 2048 of up to 64, widths of multiples
 *   of 16) are converted once to a 16-bit cache in the workspace (four bytes for each code up to max_len, where that
 *   is at most 2 GiB; exact as above), and go on in the tiles of dlrm_kv_attn_fwd, bf16 with fp16 weights too.  Where
 *   the batch has fewer than 512 rows a sequence, sequences of up to 16 rows beside them do not: they go as single
 *   tokens do.
 * A value or a sum beyond the range of dtype is infinite.  Results are the same bits from run to run of one
 * batch; a sequence's last bits may depend on which other sequences are in its batch.
 *
 * It reads half of the bytes, so single tokens are faster than over a 16-bit cache (one event of 256 users with up to
 * 8192: 177 us against 322).  Many rows are bound by products instead and pay for the conversion (4 chunks of 2048
 * on 8192 378 us against 341, 64 users' 200 candidates on up to 2000 68 against 53).  Codes of contiguous heads lie on
 * 16 bytes where d is a multiple of 16; heads of 40, 72 and the like want slots or heads padded to that, or take the
 * general kernel (one event of 256 users, heads of 72: 2062 us against 367).
 */
int dlrm_kv8_attn_fwd(const dlrm_heads *q, const dlrm_kv_batch *batch, const dlrm_kv_cache8 *cache, int d, int dtype,
                      float scale, int causal, int64_t window, int64_t max_new, int64_t max_len,
                      const dlrm_heads *out, float *lse, void *workspace, size_t workspace_bytes,
                      int32_t *err_flag, dlrm_stream_t stream);

/*
 * Pages and slots for a step's new tokens, for either cache, without the host.
 * Sequence s stores L = lengths[s] tokens and gets c = counts[s] more; c < 0: it has
 * ended, and its pages are given back.  The free pages are a ring of `pages` entries:
 * those at places state[0] .. state[1] - 1 (modulo pages) are free.
 *
 * offsets      device [S + 1]: sums of the counts above 0, the batch's offsets.
 * new_lengths  device [S]: L + c, the batch's lengths; 0 for a sequence that has
 *              ended; ~L (below 0, so that append and attention leave it out) for one that
 *              does not get its pages.  A length below 0 is read as its complement, so the next
 *              call tries again.
 * page_table   device, rows of table_width entries, table_stride apart (at least table_width):
 *              the ceil((L + c) / page_size) - ceil(L / page_size) pages that s needs are
 *              written behind those it has; nothing else is.
 * ring, state  pages are taken from state[0] on, in the order of sequences and of their
 *              pages, and given back from state[1] on, in the same order; they can be taken from the
 *              next call on.  new_state[0 .. 1]: the state afterwards.
 * slots, positions  device [n] or NULL: of each new token its slot
 *              (page * page_size + slot of the page) and its place in its history, -1
 *              where its sequence is left out.  Rows behind the last token are left as they were.
 * n            new tokens at most: rows of slots and positions.
 * new_lengths may be lengths and new_state may be state; nothing else may overlap.
 *
 * A sequence whose pages, with those that the sequences before it need, are more than the ring has is left
 * out (DLRM_FLAG_CAPACITY), and so is every later one that needs a page; so is one that does not fit its row
 * of the table, which takes no pages, or whose tokens go beyond n (DLRM_FLAG_BAD_OFFSETS).  A page number outside 0 .. pages - 1 raises
 * DLRM_FLAG_INDEX_OOB: of a sequence that has ended it is passed over, so it does not become a free page; of one that
 * goes on, in its row or in the ring as the caller filled it, its tokens' slots are -1.  A state that is not 0 <= state[0] <= state[1] <=
 * state[0] + pages raises DLRM_FLAG_BAD_OFFSETS: no page is taken or given back.  More pages given back than the
 * ring has room for raise DLRM_FLAG_CAPACITY and are dropped.
 * Every launch sums up all S sequences in each of its CTAs: made for steps of some thousands of them.
 */
int dlrm_kv_reserve(const int64_t *counts, const int64_t *lengths, int64_t S, int64_t n, int32_t *page_table,
                    int64_t table_stride, int64_t table_width, int page_size, int32_t *ring, int64_t pages,
                    const int64_t *state, int64_t *new_state, int64_t *offsets, int64_t *new_lengths, int64_t *slots,
                    int64_t *positions, int32_t *err_flag, dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_HISTORY_H */
