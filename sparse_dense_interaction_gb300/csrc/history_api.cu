// C ABI of the event-history operators: argument checks and dispatch, all on
// the host before anything is launched.
#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

size_t norm_bwd_workspace(int64_t, int, int, int);
int launch_norm_rope(const HeadsView &, const HeadsView &, int64_t, int, int, const float *, const float *, float,
                     const RopeView &, const HeadsView &, const HeadsView &, int32_t *, cudaStream_t);
int launch_norm_rope_bwd(const HeadsView &, const HeadsView &, const HeadsView &, const HeadsView &, int64_t, int, int,
                         const float *, const float *, float, const RopeView &, const HeadsView &, const HeadsView &,
                         float *, float *, float *, int32_t *, cudaStream_t);
int launch_kv_append(const HeadsView &, const HeadsView &, const BatchView &, const CacheView &, int, int,
                     const float *, float, const RopeView &, const HeadsView &, const float *, const HeadsView &,
                     int32_t *, cudaStream_t);
size_t attn_workspace(int64_t, int64_t, int, int, int, int64_t, int64_t);
int launch_kv_attn(AttnParams &, int, void *, cudaStream_t);

static const int64_t kMaxTokens = 0x7fffffffLL, kMaxPositions = (int64_t)1 << 30, kMaxSequences = (int64_t)1 << 24;
static const int kMaxHeads = 65536;
static const float kMaxScale = 2.0e38f;  // times log2(e) it is still finite

static bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

static int elem_bytes(int dtype) { return dtype == DLRM_F32 ? 4 : 2; }

static int check_row_type(int64_t n, int d, int dtype)
{
    if (n < 0 || d <= 0 || (dtype != DLRM_F32 && dtype != DLRM_F16 && dtype != DLRM_BF16))
        return DLRM_ERR_INVALID_ARG;
    return n > kMaxTokens || d > DLRM_MAX_HEAD_DIM ? DLRM_ERR_UNSUPPORTED : DLRM_OK;
}

static int check_heads(const dlrm_heads *h, int64_t n, int dtype, HeadsView &v)
{
    if (!h || h->heads < 1 || h->token_stride < 0 || h->head_stride < 0 || (n > 0 && !h->ptr) ||
        !aligned(h->ptr, elem_bytes(dtype)))
        return DLRM_ERR_INVALID_ARG;
    if (h->heads > kMaxHeads)
        return DLRM_ERR_UNSUPPORTED;
    v.ptr = static_cast<char *>(h->ptr);
    v.ts = h->token_stride;
    v.hs = h->head_stride;
    v.heads = h->heads;
    return DLRM_OK;
}

// Rows that are written lie apart (an input's may be the same: a stride of 0).
static bool apart(int64_t count, int64_t stride, int d) { return count <= 1 || stride >= d; }

// An input and an output of the same heads; both null: no heads.
static int check_pair(const dlrm_heads *in, const dlrm_heads *out, int64_t n, int d, int dtype, HeadsView &vi,
                      HeadsView &vo)
{
    vi = vo = HeadsView{nullptr, 0, 0, 0};
    if (!in && !out)
        return DLRM_OK;
    int s = check_heads(in, n, dtype, vi);
    if (s == DLRM_OK)
        s = check_heads(out, n, dtype, vo);
    return s == DLRM_OK && (vi.heads != vo.heads || !apart(n, vo.ts, d) || !apart(vo.heads, vo.hs, d))
               ? DLRM_ERR_INVALID_ARG
               : s;
}

static int check_rope(const dlrm_rope *r, int64_t n, int d, bool needs_positions, RopeView &v)
{
    v = RopeView{nullptr, 0, nullptr, 0, false};
    if (!r)
        return DLRM_OK;
    if (r->rot < 2 || r->rot > d || r->rot % 2 != 0 || r->length < 0 || !r->table || !aligned(r->table, 4) ||
        (r->layout != DLRM_ROPE_HALF && r->layout != DLRM_ROPE_INTERLEAVED) || !aligned(r->positions, 8) ||
        (needs_positions && n > 0 && !r->positions))
        return DLRM_ERR_INVALID_ARG;
    v = RopeView{r->table, r->length, r->positions, r->rot, r->layout == DLRM_ROPE_INTERLEAVED};
    return DLRM_OK;
}

static int check_weights(const float *qw, const float *kw, float eps)
{
    if (!aligned(qw, 4) || !aligned(kw, 4) || !(eps >= 0.f) || !(eps <= 3.0e38f))
        return DLRM_ERR_INVALID_ARG;
    return DLRM_OK;
}

static int check_batch(const dlrm_kv_batch *b, int page_size, BatchView &v)
{
    if (!b || b->S < 0 || b->n < 0 || b->table_stride < 0 || b->table_width < 0 || (b->S == 0 && b->n > 0))
        return DLRM_ERR_INVALID_ARG;
    if (b->S > kMaxSequences || b->n > kMaxTokens || b->table_width > kMaxPositions / page_size)
        return DLRM_ERR_UNSUPPORTED;
    if (b->n > 0 && (!b->offsets || !b->lengths || (b->table_width > 0 && !b->page_table)))
        return DLRM_ERR_INVALID_ARG;
    if (!aligned(b->offsets, 8) || !aligned(b->lengths, 8) || !aligned(b->page_table, 4))
        return DLRM_ERR_INVALID_ARG;
    v = BatchView{b->S, b->n, b->offsets, b->lengths, b->page_table, b->table_stride, b->table_width * page_size};
    return DLRM_OK;
}

static int check_cache(const dlrm_kv_cache *c, int dtype, CacheView &v)
{
    if (!c || !c->k || !c->v || c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->page_stride < 0 ||
        c->slot_stride < 0 || c->head_stride < 0 || !aligned(c->k, elem_bytes(dtype)) ||
        !aligned(c->v, elem_bytes(dtype)))
        return DLRM_ERR_INVALID_ARG;
    if (c->pages > 0x7fffffffLL || c->page_size > 65536 || c->heads > kMaxHeads)
        return DLRM_ERR_UNSUPPORTED;
    v = CacheView{static_cast<char *>(c->k), static_cast<char *>(c->v), c->page_stride, c->slot_stride,
                  c->head_stride, (uint32_t)c->pages, FastDiv::make((uint32_t)c->page_size), c->heads};
    return DLRM_OK;
}

}  // namespace dlrm

using namespace dlrm;

extern "C" {

int dlrm_qk_norm_rope_fwd(const dlrm_heads *q, const dlrm_heads *k, int64_t n, int d, int dtype,
                          const float *q_weight, const float *k_weight, float eps, const dlrm_rope *rope,
                          const dlrm_heads *q_out, const dlrm_heads *k_out, int32_t *err_flag, dlrm_stream_t stream)
{
    HeadsView vq, vk, vqo, vko;
    RopeView vr;
    int s = check_row_type(n, d, dtype);
    if (s != DLRM_OK)
        return s;
    if (!q || (s = check_pair(q, q_out, n, d, dtype, vq, vqo)) != DLRM_OK)
        return s != DLRM_OK ? s : DLRM_ERR_INVALID_ARG;
    if ((s = check_pair(k, k_out, n, d, dtype, vk, vko)) != DLRM_OK ||
        (s = check_weights(q_weight, k_weight, eps)) != DLRM_OK || (s = check_rope(rope, n, d, true, vr)) != DLRM_OK)
        return s;
    if (n == 0)
        return DLRM_OK;
    return launch_norm_rope(vq, vk, n, d, dtype, q_weight, k_weight, eps, vr, vqo, vko, err_flag,
                            static_cast<cudaStream_t>(stream));
}

size_t dlrm_qk_norm_rope_bwd_workspace_size(int64_t n, int q_heads, int k_heads, int d)
{
    if (n < 0 || n > kMaxTokens || q_heads < 1 || k_heads < 0 || q_heads > kMaxHeads || k_heads > kMaxHeads || d < 1 ||
        d > DLRM_MAX_HEAD_DIM)
        return 0;
    return norm_bwd_workspace(n, q_heads, k_heads, d);
}

int dlrm_qk_norm_rope_bwd(const dlrm_heads *dq_out, const dlrm_heads *dk_out, const dlrm_heads *q,
                          const dlrm_heads *k, int64_t n, int d, int dtype, const float *q_weight,
                          const float *k_weight, float eps, const dlrm_rope *rope, const dlrm_heads *dq,
                          const dlrm_heads *dk, float *dq_weight, float *dk_weight, void *workspace,
                          size_t workspace_bytes, int32_t *err_flag, dlrm_stream_t stream)
{
    HeadsView vq, vk, vdq, vdk, vdqo, vdko = {nullptr, 0, 0, 0};
    RopeView vr;
    int s = check_row_type(n, d, dtype);
    if (s != DLRM_OK)
        return s;
    if (!q || (s = check_pair(q, dq, n, d, dtype, vq, vdq)) != DLRM_OK)
        return s != DLRM_OK ? s : DLRM_ERR_INVALID_ARG;
    if ((s = check_heads(dq_out, n, dtype, vdqo)) != DLRM_OK ||
        (s = check_pair(k, dk, n, d, dtype, vk, vdk)) != DLRM_OK ||
        (k && (s = check_heads(dk_out, n, dtype, vdko)) != DLRM_OK) ||
        (s = check_weights(q_weight, k_weight, eps)) != DLRM_OK || (s = check_rope(rope, n, d, true, vr)) != DLRM_OK)
        return s;
    if (vdqo.heads != vq.heads || !k != !dk_out || (k && vdko.heads != vk.heads))
        return DLRM_ERR_INVALID_ARG;
    if ((dq_weight && !q_weight) || (dk_weight && (!k_weight || !k)) || !aligned(dq_weight, 4) ||
        !aligned(dk_weight, 4) || !workspace || !aligned(workspace, 16))
        return DLRM_ERR_INVALID_ARG;
    if (workspace_bytes < norm_bwd_workspace(n, vq.heads, vk.heads, d))
        return DLRM_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n == 0) {
        for (float *w : {dq_weight, dk_weight})
            if (w && cudaMemsetAsync(w, 0, d * sizeof(float), st) != cudaSuccess)
                return DLRM_ERR_CUDA;
        return DLRM_OK;
    }
    return launch_norm_rope_bwd(vdqo, vdko, vq, vk, n, d, dtype, q_weight, k_weight, eps, vr, vdq, vdk, dq_weight,
                                dk_weight, static_cast<float *>(workspace), err_flag, st);
}

int dlrm_kv_append(const dlrm_heads *k, const dlrm_heads *v, const dlrm_kv_batch *batch, const dlrm_kv_cache *cache,
                   int d, int dtype, const float *k_weight, float eps, const dlrm_rope *rope, const dlrm_heads *q,
                   const float *q_weight, const dlrm_heads *q_out, int32_t *err_flag, dlrm_stream_t stream)
{
    HeadsView vk, vv, vq, vqo;
    RopeView vr;
    BatchView vb;
    CacheView vc;
    if (!batch)
        return DLRM_ERR_INVALID_ARG;
    const int64_t n = batch->n;
    int s = check_row_type(n, d, dtype);
    if (s != DLRM_OK || (s = check_cache(cache, dtype, vc)) != DLRM_OK ||
        (s = check_batch(batch, cache->page_size, vb)) != DLRM_OK || (s = check_heads(k, n, dtype, vk)) != DLRM_OK ||
        (s = check_heads(v, n, dtype, vv)) != DLRM_OK || (s = check_pair(q, q_out, n, d, dtype, vq, vqo)) != DLRM_OK ||
        (s = check_weights(q_weight, k_weight, eps)) != DLRM_OK || (s = check_rope(rope, n, d, false, vr)) != DLRM_OK)
        return s;
    if (vk.heads != vc.heads || vv.heads != vc.heads || !apart(cache->pages, vc.page_stride, d) ||
        !apart(cache->page_size, vc.slot_stride, d) || !apart(vc.heads, vc.head_stride, d))
        return DLRM_ERR_INVALID_ARG;
    if (n == 0)
        return DLRM_OK;
    return launch_kv_append(vk, vv, vb, vc, d, dtype, k_weight, eps, vr, vq, q_weight, vqo, err_flag,
                            static_cast<cudaStream_t>(stream));
}

size_t dlrm_kv_attn_workspace_size(int64_t S, int64_t n, int q_heads, int kv_heads, int d, int64_t max_new,
                                   int64_t max_len)
{
    if (S < 0 || S > kMaxSequences || n < 0 || n > kMaxTokens || kv_heads < 1 || kv_heads > kMaxHeads ||
        q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads != 0 || d < 1 || d > DLRM_MAX_HEAD_DIM ||
        max_new < 0 || max_new > kMaxTokens || max_len < 0 || max_len > kMaxPositions)
        return 0;
    return attn_workspace(S, n, q_heads, kv_heads, d, max_new, max_len);
}

int dlrm_kv_attn_fwd(const dlrm_heads *q, const dlrm_kv_batch *batch, const dlrm_kv_cache *cache, int d, int dtype,
                     float scale, int causal, int64_t window, int64_t max_new, int64_t max_len,
                     const dlrm_heads *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                     dlrm_stream_t stream)
{
    AttnParams p = {};
    if (!batch || !q)
        return DLRM_ERR_INVALID_ARG;
    const int64_t n = batch->n;
    int s = check_row_type(n, d, dtype);
    if (s != DLRM_OK || (s = check_cache(cache, dtype, p.cache)) != DLRM_OK ||
        (s = check_batch(batch, cache->page_size, p.batch)) != DLRM_OK ||
        (s = check_pair(q, out, n, d, dtype, p.q, p.out)) != DLRM_OK)
        return s;
    if (p.q.heads % p.cache.heads != 0 || !(scale > 0.f) || !(scale <= kMaxScale) || (causal != 0 && causal != 1) ||
        window < 0 || max_new < 0 || max_len < 0 || !aligned(lse, 4) || !workspace || !aligned(workspace, 16))
        return DLRM_ERR_INVALID_ARG;
    p.group = p.q.heads / p.cache.heads;
    p.max_new = max_new < n ? max_new : n;
    if (max_len > kMaxPositions || p.max_new * p.group > kMaxTokens)
        return DLRM_ERR_UNSUPPORTED;
    if (n > 0 && max_new == 0)
        return DLRM_ERR_INVALID_ARG;
    if (workspace_bytes < attn_workspace(p.batch.S, n, p.q.heads, p.cache.heads, d, max_new, max_len))
        return DLRM_ERR_WORKSPACE_TOO_SMALL;
    if (n == 0)
        return DLRM_OK;
    p.max_len = max_len;
    p.d = d;
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.causal = causal != 0;
    p.window = window < kMaxPositions ? (int)window : 0;  // as wide as any history: none
    p.lse = lse;
    p.wait_polls = wait_hooks(0, tc::kSpinLimit).copy_polls;  // the default unless a test shortens it
    p.err = err_flag;
    return launch_kv_attn(p, dtype, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
