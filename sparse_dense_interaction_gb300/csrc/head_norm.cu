// Norm and rotation of query and key heads, its gradient, and the append of
// keys and values to the paged cache.
//
// One row is the d elements of one head of one token.  With r = 1/sqrt(mean
// x^2 + eps):  z = x r w, then pairs of z are turned by the token's angles.
// Turning is orthogonal, so the gradient turns dy back (dz), and with
// g = dz w:  dx = r (g - x r^2 mean(g x)),  dw = sum of dz x r over all rows.
//
// The row kernels here serve every width, stride and alignment: a warp per row,
// lane l holds the elements l, l + 32, ...  Rows that can be moved as 4-element pieces
// take the vector path (head_norm.cuh).  Loads of single elements, few at a
// time, bound them: 20000 tokens of 8 query and 2 key heads of 250 bf16 elements
// take 180 us forward, 1.1 TB/s, 373 backward, 0.8 TB/s; of 17 fp32 elements 89
// and 123 us; the append of as many rows of 250 294 us.
#include <initializer_list>

#include "head_norm.cuh"

namespace dlrm {

size_t norm_bwd_vec_workspace(int64_t, int, int, int);
int launch_norm_rope_vec(const HeadsView &, const HeadsView &, int64_t, int, int, const float *, const float *, float,
                         const RopeView &, const HeadsView &, const HeadsView &, int32_t *, cudaStream_t);
int launch_norm_rope_bwd_vec(const HeadsView &, const HeadsView &, const HeadsView &, const HeadsView &, int64_t, int,
                             int, const float *, const float *, float, const RopeView &, const HeadsView &,
                             const HeadsView &, float *, float *, float *, int32_t *, cudaStream_t);
int launch_kv_append_vec(const HeadsView &, const HeadsView &, const BatchView &, const CacheView &, int, int,
                         const float *, float, const RopeView &, const HeadsView &, const float *, const HeadsView &,
                         int32_t *, cudaStream_t);

constexpr int kRowElems = DLRM_MAX_HEAD_DIM / 32;  // elements of a lane

// The partner of element e in its pair and whether e is the pair's first; -1
// for elements that are not turned.
__device__ __forceinline__ int pair_of(const RopeView &rope, int e, bool &first)
{
    if (!rope.table || e >= rope.rot)
        return -1;
    const int half = rope.rot >> 1;
    first = rope.interleaved ? (e & 1) == 0 : e < half;
    if (rope.interleaved)
        return e ^ 1;
    return first ? e + half : e - half;
}

// The angle's column of element e in a rope row.
__device__ __forceinline__ int angle_of(const RopeView &rope, int e)
{
    const int half = rope.rot >> 1;
    return rope.interleaved ? e >> 1 : (e < half ? e : e - half);
}

// 1/sqrt(mean x^2 + eps) of a row, from every lane's sum of squares.
__device__ __forceinline__ float inv_rms(float squares, int d, float eps)
{
    return 1.f / sqrtf(warp_sum(squares) / (float)d + eps);
}

// One row: norm (weight not null) and rotation (row not null) into y, which may
// be x: it is written when every lane has read.
template <typename T>
__device__ __forceinline__ void norm_rope_row(const T *x, T *y, int d, const float *weight, float eps,
                                              const RopeView &rope, const float *angles)
{
    const int lane = threadIdx.x & 31;
    float v[kRowElems], sq = 0.f, r = 1.f;
#pragma unroll
    for (int j = 0; j < kRowElems; j++) {
        const int e = lane + 32 * j;
        v[j] = e < d ? to_f32(x[e]) : 0.f;
        sq = fmaf(v[j], v[j], sq);
    }
    if (weight)
        r = inv_rms(sq, d, eps);
#pragma unroll
    for (int j = 0; j < kRowElems; j++) {
        const int e = lane + 32 * j;
        if (e >= d)
            continue;
        float z = weight ? v[j] * r * weight[e] : v[j];
        bool first;
        const int other = angles ? pair_of(rope, e, first) : -1;
        if (other >= 0) {
            const float xo = to_f32(x[other]), zo = weight ? xo * r * weight[other] : xo;
            const int a = angle_of(rope, e);
            const float c = angles[a], s = angles[a + (rope.rot >> 1)];
            z = first ? fmaf(z, c, -zo * s) : fmaf(z, c, zo * s);
        }
        v[j] = z;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kRowElems; j++)
        if (lane + 32 * j < d)
            y[lane + 32 * j] = from_f32<T>(v[j]);
}

template <typename T>
__device__ __forceinline__ void zero_row(T *y, int d)
{
    for (int e = threadIdx.x & 31; e < d; e += 32)
        y[e] = from_f32<T>(0.f);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_rows_kernel(HeadsView q, HeadsView k, int64_t n, int d, const float *__restrict__ qw,
                      const float *__restrict__ kw, float eps, RopeView rope, HeadsView qo, HeadsView ko, int32_t *err)
{
    const int heads = q.heads + k.heads;
    const int64_t rows = n * heads;
    for (int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < rows; row += (int64_t)gridDim.x * kWarps) {
        const int64_t token = row / heads;
        const int h = (int)(row - token * heads);
        const bool is_q = h < q.heads;
        const T *x = is_q ? q.row<T>(token, h) : k.row<T>(token, h - q.heads);
        T *y = is_q ? qo.row<T>(token, h) : ko.row<T>(token, h - q.heads);
        const float *angles = rope.table ? rope_row(rope, rope.positions[token], err) : nullptr;
        if (rope.table && !angles)
            zero_row(y, d);
        else
            norm_rope_row(x, y, d, is_q ? qw : kw, eps, rope, angles);
    }
}

// blockIdx.y: 0 the queries, 1 the keys.  part: [2][gridDim.x][d] sums of the
// weights' gradients.  dx may be x or dy: what is stored depends on sums of all that
// the warp reads of the row, but for rows that are only turned (kPlain: there are
// some), which wait for one another (in all rows that takes 418 us instead of 373
// for the bf16 gradient named above).
template <typename T, bool kPlain>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_bwd_rows_kernel(HeadsView dqo, HeadsView dko, HeadsView q, HeadsView k, int64_t n, int d,
                          const float *__restrict__ qw, const float *__restrict__ kw, float eps, RopeView rope,
                          HeadsView dq, HeadsView dk, float *__restrict__ part, int32_t *err)
{
    __shared__ float sums[kWarps][DLRM_MAX_HEAD_DIM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool is_q = blockIdx.y == 0;
    const HeadsView x_ = is_q ? q : k, dy_ = is_q ? dqo : dko, dx_ = is_q ? dq : dk;
    const float *weight = is_q ? qw : kw;
    float dw[kRowElems] = {};
    const int64_t rows = n * x_.heads;
    for (int64_t row = (int64_t)blockIdx.x * kWarps + warp; row < rows; row += (int64_t)gridDim.x * kWarps) {
        const int64_t token = row / x_.heads;
        const int h = (int)(row - token * x_.heads);
        const T *x = x_.row<T>(token, h), *dy = dy_.row<T>(token, h);
        T *dx = dx_.row<T>(token, h);
        const float *angles = rope.table ? rope_row(rope, rope.positions[token], err) : nullptr;
        if (rope.table && !angles) {
            zero_row(dx, d);
            continue;
        }
        float v[kRowElems], dz[kRowElems], sq = 0.f, gx = 0.f;
#pragma unroll
        for (int j = 0; j < kRowElems; j++) {
            const int e = lane + 32 * j;
            v[j] = dz[j] = 0.f;
            if (e >= d)
                continue;
            v[j] = to_f32(x[e]);
            dz[j] = to_f32(dy[e]);
            bool first;
            const int other = angles ? pair_of(rope, e, first) : -1;
            if (other >= 0) {
                const float o = to_f32(dy[other]);
                const int a = angle_of(rope, e);
                const float c = angles[a], s = angles[a + (rope.rot >> 1)];
                dz[j] = first ? fmaf(dz[j], c, o * s) : fmaf(dz[j], c, -o * s);
            }
            sq = fmaf(v[j], v[j], sq);
            if (weight)
                gx = fmaf(dz[j] * weight[e], v[j], gx);
        }
        if (weight) {
            const float r = inv_rms(sq, d, eps);
            const float m = warp_sum(gx) / (float)d * r * r;
#pragma unroll
            for (int j = 0; j < kRowElems; j++) {
                const int e = lane + 32 * j;
                if (e >= d)
                    continue;
                dw[j] = fmaf(dz[j], v[j] * r, dw[j]);
                dz[j] = r * fmaf(-v[j], m, dz[j] * weight[e]);
            }
        }
        if (kPlain)
            __syncwarp();
#pragma unroll
        for (int j = 0; j < kRowElems; j++)
            if (lane + 32 * j < d)
                dx[lane + 32 * j] = from_f32<T>(dz[j]);
    }
#pragma unroll
    for (int j = 0; j < kRowElems; j++)
        if (lane + 32 * j < d)
            sums[warp][lane + 32 * j] = dw[j];
    __syncthreads();
    for (int e = threadIdx.x; e < d; e += blockDim.x) {
        float s = 0.f;
        for (int w = 0; w < kWarps; w++)
            s += sums[w][e];
        part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * d + e] = s;
    }
}

// The CTAs' sums of the weights' gradients added up, in a fixed order: a warp per
// element.  A few hundred rows from L2: 3 us, latency.
// part: q_parts rows of d sums of the queries', then k_parts of the keys'.
__global__ void __launch_bounds__(kWarps * 32)
norm_weight_sum_kernel(const float *__restrict__ part, int64_t q_parts, int64_t k_parts, int d,
                       float *__restrict__ dqw, float *__restrict__ dkw)
{
    float *out = blockIdx.y == 0 ? dqw : dkw;
    const int64_t from = blockIdx.y == 0 ? 0 : q_parts, to = blockIdx.y == 0 ? q_parts : q_parts + k_parts;
    const int e = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (!out || e >= d)
        return;
    float s = 0.f;
    for (int64_t c = from + (threadIdx.x & 31); c < to; c += 32)
        s += part[c * d + e];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0)
        out[e] = s;
}

void launch_norm_weight_sum(const float *part, int64_t q_parts, int64_t k_parts, int d, float *dqw, float *dkw,
                            cudaStream_t st)
{
    norm_weight_sum_kernel<<<dim3((d + kWarps - 1) / kWarps, k_parts > 0 ? 2 : 1), kWarps * 32, 0, st>>>(
        part, q_parts, k_parts, d, dqw, dkw);
    count_launch(st);
}

// One warp per new token.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
kv_append_rows_kernel(HeadsView k, HeadsView v, BatchView batch, CacheView cache, int d,
                      const float *__restrict__ kw, float eps, RopeView rope, HeadsView q,
                      const float *__restrict__ qw, HeadsView qo, int32_t *err)
{
    const int lane = threadIdx.x & 31;
    check_sequences(batch, (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x, err);
    for (int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); token < batch.n;
         token += (int64_t)gridDim.x * kWarps) {
        const int64_t s = find_sequence(batch, token);
        Sequence seq;
        if (s < 0 || !read_sequence(batch, s, batch.n, batch.capacity, seq, err) ||
            !seq.has(token) || seq.count > seq.length) {
            raise_flag(err, DLRM_FLAG_BAD_OFFSETS);
            continue;
        }
        const int at = seq.length - seq.count + (int)(token - seq.first);
        const float *angles = nullptr;
        if (rope.table) {
            angles = rope_row(rope, rope.positions ? rope.positions[token] : at, err);
            if (!angles) {
                for (int h = 0; h < q.heads; h++)
                    zero_row(qo.row<T>(token, h), d);
                continue;
            }
        }
        for (int h = 0; h < q.heads; h++)
            norm_rope_row(q.row<T>(token, h), qo.row<T>(token, h), d, qw, eps, rope, angles);
        const int64_t slot = slot_offset<T>(cache, batch.table + s * batch.table_stride, at, 0);
        if (slot < 0) {
            raise_flag(err, DLRM_FLAG_INDEX_OOB);
            continue;
        }
        for (int h = 0; h < cache.heads; h++) {
            norm_rope_row(k.row<T>(token, h), reinterpret_cast<T *>(cache.k + slot) + h * cache.head_stride, d, kw,
                          eps, rope, angles);
            const T *x = v.row<T>(token, h);
            T *y = reinterpret_cast<T *>(cache.v + slot) + h * cache.head_stride;
            for (int e = lane; e < d; e += 32)
                y[e] = x[e];
        }
    }
}

// CTAs of the gradient: enough for every SM, and few enough that their sums
// are small.
constexpr int64_t kBwdCtas = 608;  // four for each of 152 SMs

static int64_t bwd_ctas(int64_t n, int heads)
{
    const int64_t need = div_up(n * heads, kWarps);
    return need < 1 ? 1 : (need < kBwdCtas ? need : kBwdCtas);
}

size_t norm_bwd_workspace(int64_t n, int qh, int kh, int d)
{
    const size_t rows = 2 * (size_t)bwd_ctas(n, qh > kh ? qh : kh) * d * sizeof(float);
    const size_t vec = norm_bwd_vec_workspace(n, qh, kh, d);
    return rows > vec ? rows : vec;
}

// Whether the vector path takes these rows.
static bool vec_ok(int d, int dtype, const RopeView &rope, std::initializer_list<const HeadsView *> heads)
{
    bool ok = d % 8 == 0 && rope_pieces_ok(rope);
    for (const HeadsView *h : heads)
        ok = ok && pieces_ok(*h, dtype == DLRM_F32 ? 4 : 2);
    return ok;
}

static int64_t row_ctas(int64_t rows)
{
    const int64_t need = div_up(rows, kWarps);
    return need < 65536 ? need : 65536;
}

template <typename T>
static int norm_fwd(const HeadsView &q, const HeadsView &k, int64_t n, int d, const float *qw, const float *kw,
                    float eps, const RopeView &rope, const HeadsView &qo, const HeadsView &ko, int32_t *err,
                    cudaStream_t st)
{
    norm_rope_rows_kernel<T><<<(unsigned)row_ctas(n * (q.heads + k.heads)), kWarps * 32, 0, st>>>(q, k, n, d, qw, kw, eps, rope,
                                                                                    qo, ko, err);
    count_launch(st);
    return launch_status();
}

int launch_norm_rope(const HeadsView &q, const HeadsView &k, int64_t n, int d, int dtype, const float *qw,
                     const float *kw, float eps, const RopeView &rope, const HeadsView &qo, const HeadsView &ko,
                     int32_t *err, cudaStream_t st)
{
    if (vec_ok(d, dtype, rope, {&q, &k, &qo, &ko}))
        return launch_norm_rope_vec(q, k, n, d, dtype, qw, kw, eps, rope, qo, ko, err, st);
    if (dtype == DLRM_F32)
        return norm_fwd<float>(q, k, n, d, qw, kw, eps, rope, qo, ko, err, st);
    if (dtype == DLRM_F16)
        return norm_fwd<__half>(q, k, n, d, qw, kw, eps, rope, qo, ko, err, st);
    return norm_fwd<__nv_bfloat16>(q, k, n, d, qw, kw, eps, rope, qo, ko, err, st);
}

template <typename T>
static int norm_bwd(const HeadsView &dqo, const HeadsView &dko, const HeadsView &q, const HeadsView &k, int64_t n,
                    int d, const float *qw, const float *kw, float eps, const RopeView &rope, const HeadsView &dq,
                    const HeadsView &dk, float *dqw, float *dkw, float *part, int32_t *err, cudaStream_t st)
{
    const int64_t ctas = bwd_ctas(n, q.heads > k.heads ? q.heads : k.heads);
    const unsigned sides = k.heads > 0 ? 2 : 1;
    const auto kernel = qw && (kw || sides == 1) ? norm_rope_bwd_rows_kernel<T, false> : norm_rope_bwd_rows_kernel<T, true>;
    kernel<<<dim3((unsigned)ctas, sides), kWarps * 32, 0, st>>>(dqo, dko, q, k, n, d, qw, kw, eps, rope, dq, dk, part, err);
    count_launch(st);
    if (dqw || dkw)
        launch_norm_weight_sum(part, ctas, sides == 2 ? ctas : 0, d, dqw, dkw, st);
    return launch_status();
}

int launch_norm_rope_bwd(const HeadsView &dqo, const HeadsView &dko, const HeadsView &q, const HeadsView &k,
                         int64_t n, int d, int dtype, const float *qw, const float *kw, float eps,
                         const RopeView &rope, const HeadsView &dq, const HeadsView &dk, float *dqw, float *dkw,
                         float *part, int32_t *err, cudaStream_t st)
{
    if (vec_ok(d, dtype, rope, {&dqo, &dko, &q, &k, &dq, &dk}))
        return launch_norm_rope_bwd_vec(dqo, dko, q, k, n, d, dtype, qw, kw, eps, rope, dq, dk, dqw, dkw, part, err,
                                        st);
    if (dtype == DLRM_F32)
        return norm_bwd<float>(dqo, dko, q, k, n, d, qw, kw, eps, rope, dq, dk, dqw, dkw, part, err, st);
    if (dtype == DLRM_F16)
        return norm_bwd<__half>(dqo, dko, q, k, n, d, qw, kw, eps, rope, dq, dk, dqw, dkw, part, err, st);
    return norm_bwd<__nv_bfloat16>(dqo, dko, q, k, n, d, qw, kw, eps, rope, dq, dk, dqw, dkw, part, err, st);
}

template <typename T>
static int append(const HeadsView &k, const HeadsView &v, const BatchView &batch, const CacheView &cache, int d,
                  const float *kw, float eps, const RopeView &rope, const HeadsView &q, const float *qw,
                  const HeadsView &qo, int32_t *err, cudaStream_t st)
{
    kv_append_rows_kernel<T><<<(unsigned)row_ctas(batch.n), kWarps * 32, 0, st>>>(k, v, batch, cache, d, kw, eps,
                                                                                  rope, q, qw, qo, err);
    count_launch(st);
    return launch_status();
}

int launch_kv_append(const HeadsView &k, const HeadsView &v, const BatchView &batch, const CacheView &cache, int d,
                     int dtype, const float *kw, float eps, const RopeView &rope, const HeadsView &q,
                     const float *qw, const HeadsView &qo, int32_t *err, cudaStream_t st)
{
    const HeadsView kc = {cache.k, cache.page_stride, cache.slot_stride, 0}, vc = {cache.v, cache.head_stride, 0, 0};
    if (vec_ok(d, dtype, rope, {&k, &v, &q, &qo, &kc, &vc}))
        return launch_kv_append_vec(k, v, batch, cache, d, dtype, kw, eps, rope, q, qw, qo, err, st);
    if (dtype == DLRM_F32)
        return append<float>(k, v, batch, cache, d, kw, eps, rope, q, qw, qo, err, st);
    if (dtype == DLRM_F16)
        return append<__half>(k, v, batch, cache, d, kw, eps, rope, q, qw, qo, err, st);
    return append<__nv_bfloat16>(k, v, batch, cache, d, kw, eps, rope, q, qw, qo, err, st);
}

}  // namespace dlrm
