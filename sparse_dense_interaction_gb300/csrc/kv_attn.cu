// Attention over the paged cache: the launch plan, the general kernel and the
// join of splits.
//
// The queries of one sequence and cache head are packed rows: row
// r = token * group + g is query head (head * group + g) of that token, so
// all heads that share a cache head share one pass over its keys and values.
// The softmax runs in one pass: with a running maximum m and sum l in base 2,
// a tile of scores s raises m, scales l and the output by 2^(m_old - m_new)
// and adds 2^(s - m_new).  Positions are split where there are few rows; a
// split leaves its normalised output and log2 of its sum, and the join weighs
// the splits by 2^(lse - max).
#include <type_traits>

#include "kv8.cuh"

namespace dlrm {

size_t few_workspace(int64_t, int, int64_t);
int launch_kv_attn_few(AttnParams &, int, void *, cudaStream_t);
int launch_kv_attn_tile(const AttnParams &, int, int64_t, cudaStream_t);
int launch_kv8_attn_tile(const AttnParams &, int, int64_t, cudaStream_t);
size_t widen_workspace(int64_t, int, int, int, int64_t, int64_t);
int launch_widen(AttnParams &, int, void *, cudaStream_t);
bool launch_kv8_attn_few(AttnParams &, int, void *, cudaStream_t, int &);

// ---------------------------------------------------------------- general kernel

// For every type, head width, stride and page size.  A CTA holds kGenRows
// rows; a tile of 32 positions is widened to fp32 in shared memory, a lane
// takes one position's score for two rows, then each thread sums its output
// columns.  Its loads wait for its sums and its products for shared memory: one
// event of each of 64 users with 2000, 16 heads on 4 of 17 fp32 elements, takes
// 141 us, 0.5 TB/s.
constexpr int kGenRows = 8, kGenTile = 32, kGenThreads = 128;
constexpr int kGenCols = kGenRows * DLRM_MAX_HEAD_DIM / kGenThreads;  // output elements of a thread

__host__ __device__ constexpr int gen_pad(int d) { return (d + 3) & ~3; }

static int general_smem(int d)
{
    const int dp = gen_pad(d);
    return (kGenRows * dp + kGenTile * (dp + 4) + kGenTile * dp + kGenRows * kGenTile + kGenRows) * 4;
}

// kCodes: the cache holds codes of 8 bits.
template <typename T, bool kCodes>
__global__ void __launch_bounds__(kGenThreads)
kv_attn_general_kernel(const __grid_constant__ AttnParams p)
{
    using Stored = typename std::conditional<kCodes, uint8_t, T>::type;
    extern __shared__ float4 smem4[];
    const int d = p.d, dp = gen_pad(d), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sq = reinterpret_cast<float *>(smem4), *sk = sq + kGenRows * dp, *sv = sk + kGenTile * (dp + 4);
    float *sp = sv + kGenTile * dp, *sf = sp + kGenRows * kGenTile;
    AttnWork w;
    if (!attn_work(p, blockIdx.x, w))
        return;
    const int32_t *pages = p.batch.table + w.s * p.batch.table_stride;
    const int heads = p.cache.heads * p.group;
    for (int i = threadIdx.x; i < kGenRows * dp; i += kGenThreads) {
        const int r = i / dp, e = i - r * dp;
        float x = 0.f;
        if (r < w.rows && e < d) {
            const int row = w.row0 + r, t = row / p.group;
            x = to_f32(p.q.row<T>(w.seq.first + t, w.head * p.group + row - t * p.group)[e]);
        }
        sq[i] = x;
    }
    float acc[kGenCols] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int lo[2], hi[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int r = warp * 2 + j;
        hi[j] = r < w.rows ? seen_hi(w.seq, p.causal, (w.row0 + r) / p.group) : 0;
        lo[j] = max(seen_lo(hi[j], p.window), w.lo);
        hi[j] = min(hi[j], w.hi);
    }
    for (int tile = w.lo; tile < w.hi; tile += kGenTile) {
        __syncthreads();
        for (int t = warp; t < kGenTile; t += kGenThreads / 32) {
            int64_t at = -1;
            if (tile + t < w.hi) {
                at = slot_offset<Stored>(p.cache, pages, tile + t, w.head);
                if (at < 0)
                    raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
            }
            if constexpr (kCodes) {
                float kp = 0.f, vp = 0.f;
                if (at >= 0) {
                    const uint32_t page = p.cache.page.div((uint32_t)(tile + t));
                    const int64_t x = exp_offset(p.exp, pages[page], tile + t - page * p.cache.page.d, w.head);
                    kp = exp_power(p.exp.k[x]);
                    vp = exp_power(p.exp.v[x]);
                }
                for (int e = lane; e < dp; e += 32) {
                    const bool there = at >= 0 && e < d;
                    const uint16_t c = there ? (uint8_t)p.cache.k[at + e] | (uint8_t)p.cache.v[at + e] << 8 : 0;
                    const float2 x = decode2_f32(c);
                    sk[t * (dp + 4) + e] = x.x * kp;
                    sv[t * dp + e] = x.y * vp;
                }
                continue;
            }
            const T *k = reinterpret_cast<const T *>(p.cache.k + at), *v = reinterpret_cast<const T *>(p.cache.v + at);
            for (int e = lane; e < dp; e += 32) {
                sk[t * (dp + 4) + e] = at >= 0 && e < d ? to_f32(k[e]) : 0.f;
                sv[t * dp + e] = at >= 0 && e < d ? to_f32(v[e]) : 0.f;
            }
        }
        __syncthreads();
        const float4 *k4 = reinterpret_cast<const float4 *>(sk + lane * (dp + 4));
        float s[2] = {0.f, 0.f};
        for (int e = 0; e < dp / 4; e++) {
            const float4 k = k4[e];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const float4 q = reinterpret_cast<const float4 *>(sq + (warp * 2 + j) * dp)[e];
                s[j] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[j]))));
            }
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int at = tile + lane;
            const float x = at >= lo[j] && at < hi[j] ? s[j] * p.scale_log2 : -INFINITY;
            const float top = fmaxf(m[j], warp_max(x)), base = top == -INFINITY ? 0.f : top;
            const float e = exp2_approx(x - base), f = exp2_approx(m[j] - base);
            l[j] = fmaf(l[j], f, warp_sum(e));
            m[j] = top;
            sp[(warp * 2 + j) * kGenTile + lane] = e;
            if (lane == 0)
                sf[warp * 2 + j] = f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kGenCols; i++) {
            const int idx = threadIdx.x + i * kGenThreads, r = idx / d, e = idx - r * d;
            if (r >= kGenRows)
                break;
            float a = acc[i] * sf[r];
            for (int t = 0; t < kGenTile; t++)
                a = fmaf(sp[r * kGenTile + t], sv[t * dp + e], a);
            acc[i] = a;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int r = warp * 2 + j;
        if (lane == 0) {
            sf[r] = l[j] == 0.f ? 0.f : 1.f / l[j];
            if (r < w.rows) {
                const int row = w.row0 + r, t = row / p.group, h = w.head * p.group + row - t * p.group;
                const float lse = m[j] + log2f(l[j]);  // -infinity where nothing was seen
                if (!w.whole)
                    p.part_lse[((int64_t)w.split * p.batch.n + w.seq.first + t) * heads + h] = lse;
                else if (p.lse)
                    p.lse[(w.seq.first + t) * heads + h] = lse * kLn2;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGenCols; i++) {
        const int idx = threadIdx.x + i * kGenThreads, r = idx / d, e = idx - r * d;
        if (r >= w.rows)
            break;
        const int row = w.row0 + r, t = row / p.group, h = w.head * p.group + row - t * p.group;
        const float x = acc[i] * sf[r];
        if (w.whole)
            p.out.row<T>(w.seq.first + t, h)[e] = from_f32<T>(x);
        else
            p.part_o[(((int64_t)w.split * p.batch.n + w.seq.first + t) * heads + h) * d + e] = x;
    }
}

// ---------------------------------------------------------------- join of splits

// A warp per (token, query head).
template <typename T>
__global__ void __launch_bounds__(256)
kv_attn_join_kernel(const __grid_constant__ AttnParams p)
{
    const int lane = threadIdx.x & 31, heads = p.cache.heads * p.group;
    const int64_t all = p.batch.n * heads;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < all; i += (int64_t)gridDim.x * 8) {
        const int64_t token = i / heads, s = find_sequence(p.batch, token);
        const int h = (int)(i - token * heads);
        Sequence seq;
        if (s < 0 || !read_sequence(p.batch, s, p.max_new, p.max_len, seq, nullptr) || !seq.has(token) ||
            !attn_takes(p, seq))
            continue;
        // the tile that held this row, and whether it was split
        const int t = (int)(token - seq.first), row = t * p.group + h % p.group, row0 = row / p.rows * p.rows;
        const int row1 = min(row0 + p.rows, seq.count * p.group) - 1;
        const int base = split_base(seq, p.causal, p.window, row0 / p.group);
        if (seen_hi(seq, p.causal, row1 / p.group) - base <= p.split_len)
            continue;
        const int hi = seen_hi(seq, p.causal, t), lo = seen_lo(hi, p.window);
        const int first = (lo - base) / p.split_len, last = hi > lo ? (hi - 1 - base) / p.split_len : first - 1;
        float top = -INFINITY;
        for (int k = first + lane; k <= last; k += 32)
            top = fmaxf(top, p.part_lse[(int64_t)k * all + i]);
        top = warp_max(top);
        const float base_top = top == -INFINITY ? 0.f : top;
        float total = 0.f, acc[DLRM_MAX_HEAD_DIM / 32] = {};
        for (int k0 = first; k0 <= last; k0 += 32) {
            // the weights by a lane each, then the parts, whose loads do not wait for one another
            const int n = min(last - k0 + 1, 32);
            const float mine = lane < n ? exp2_approx(p.part_lse[(int64_t)(k0 + lane) * all + i] - base_top) : 0.f;
            total += warp_sum(mine);
#pragma unroll 8
            for (int k = 0; k < n; k++) {
                const float f = __shfl_sync(0xffffffffu, mine, k);
                const float *o = p.part_o + ((int64_t)(k0 + k) * all + i) * p.d;
#pragma unroll
                for (int j = 0; j < DLRM_MAX_HEAD_DIM / 32; j++)
                    if (lane + 32 * j < p.d)
                        acc[j] = fmaf(o[lane + 32 * j], f, acc[j]);
            }
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;
        T *out = p.out.row<T>(token, h);
#pragma unroll
        for (int j = 0; j < DLRM_MAX_HEAD_DIM / 32; j++)
            if (lane + 32 * j < p.d)
                out[lane + 32 * j] = from_f32<T>(acc[j] * inv);
        if (p.lse && lane == 0)
            p.lse[i] = last >= first ? (top + log2f(total)) * kLn2 : -INFINITY;
    }
}

// ---------------------------------------------------------------- plan and launch

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kPlanSms = 152;   // the plan is this GPU's; it does not change with the device
constexpr int kMaxSplits = 256;

// Splits of a sequence's positions: enough CTAs to fill the GPU `waves` times
// over, none shorter than `least` positions.
static AttnPlan plan_splits(AttnKernel kernel, int rows, int64_t S, int kv_heads, int group, int64_t max_new,
                            int64_t max_len, int64_t ctas, int64_t least)
{
    AttnPlan a;
    a.kernel = kernel;
    a.rows = rows;
    a.tiles = ceil_div(max_new * group, rows);
    const int64_t have = S * kv_heads * a.tiles, longest = max_len + 127;
    int64_t want = ceil_div(ctas, have < 1 ? 1 : have);
    want = want < 1 ? 1 : (want < kMaxSplits ? want : kMaxSplits);
    int64_t len = ceil_div(ceil_div(longest, want), 128) * 128;
    if (len < least)
        len = least;
    a.split_len = (int)(len < 0x7fffff80 ? len : 0x7fffff80);
    a.splits = (int)ceil_div(longest, a.split_len);
    if (a.splits < 1)
        a.splits = 1;
    return a;
}

// The number of splits that ends soonest, for lengths that are all the longest
// (rounds of CTAs) and for lengths of any size up to it (the CTAs' positions
// shared out evenly, then the last CTA's own): the sum of both.  A CTA costs as
// much as 512 positions beside its share (its start and its end), 704 where its
// rows go through the join, which itself costs 512.  (24 sequences of up to 333
// rows on up to 95129 positions: 213 us with 16 splits, 401 with the 3 that one
// round takes; 8 of 1024 rows on 8192 each: 95 and 77, on up to 8192: 53 and 69.)
static AttnPlan plan_tile(int64_t S, int kv_heads, int group, int d, int64_t max_new, int64_t seen)
{
    const int rows = tile_rows(max_new * group, d);
    const int64_t have = S * kv_heads * ceil_div(max_new * group, rows), longest = seen + 127;
    const int64_t places = tile_places(rows, d);
    int64_t best = 1, least = INT64_MAX;
    // one, or as many as fill 1 to 16 rounds of places
    for (int64_t round = 0, last = 0; round <= (have < 2 * places ? 16 : 0); round++) {
        const int64_t most = round * places / (have < 1 ? 1 : have), s = most < 1 ? 1 : (most < 64 ? most : 64);
        if (s == last)
            continue;
        last = s;
        const int64_t cta = s > 1 ? 704 : 512, own = ceil_div(longest, s) + cta;
        const int64_t cost = ceil_div(have * s, places) * own + have * (longest / 2 + s * cta) / places + own +
                             (s > 1 ? 1024 : 0);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return plan_splits(kAttnTile, rows, S, kv_heads, group, max_new, seen, best > 1 ? have * best : 1, 512);
}

static AttnPlan plan(AttnKernel kernel, int64_t S, int kv_heads, int group, int d, int64_t max_new, int64_t max_len)
{
    if (kernel == kAttnTile)
        return plan_tile(S, kv_heads, group, d, max_new, max_len);
    return plan_splits(kAttnGeneral, kGenRows, S, kv_heads, group, max_new, max_len, kPlanSms * 8, 256);
}

static size_t part_floats(const AttnPlan &a, int64_t n, int heads, int d)
{
    return a.splits > 1 ? (size_t)a.splits * n * heads * (d + 1) : 0;
}

// The largest of the kernels' needs: which one runs depends on types and alignment too.  (Heads above 128 take tiles
// over a cache in 8 bits alone.)
static size_t workspace_of(bool codes, int64_t S, int64_t n, int q_heads, int kv_heads, int d, int64_t max_new,
                           int64_t max_len)
{
    const int group = q_heads / kv_heads;
    max_new = max_new < n ? max_new : n;
    size_t most = few_workspace(max_new * group, d, max_len);
    for (AttnKernel k : {kAttnGeneral, kAttnTile}) {
        if (k == kAttnTile && d > 128 && !codes)
            continue;
        const size_t b = part_floats(plan(k, S, kv_heads, group, d, max_new, max_len), n, q_heads, d) * sizeof(float);
        most = b > most ? b : most;
    }
    return most + 16;
}

size_t attn_workspace(int64_t S, int64_t n, int q_heads, int kv_heads, int d, int64_t max_new, int64_t max_len)
{
    return workspace_of(false, S, n, q_heads, kv_heads, d, max_new, max_len);
}

// Over a cache in 8 bits: a copy of it in 16 bits may come first, if the call may take tiles.
size_t attn8_workspace(int64_t S, int64_t n, int q_heads, int kv_heads, int d, int64_t max_new, int64_t max_len,
                       bool tiles)
{
    const int group = q_heads / kv_heads;
    return workspace_of(true, S, n, q_heads, kv_heads, d, max_new, max_len) +
           (tiles ? widen_workspace(S, kv_heads, group, d, max_new < n ? max_new : n, max_len) : 0);
}

template <typename T, bool kCodes>
static int launch_general(const AttnParams &p, int64_t ctas, cudaStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv_attn_general_kernel<T, kCodes>, general_smem(DLRM_MAX_HEAD_DIM), &done);
    if (s != DLRM_OK)
        return s;
    kv_attn_general_kernel<T, kCodes><<<(unsigned)ctas, kGenThreads, general_smem(p.d), st>>>(p);
    count_launch(st);
    return DLRM_OK;
}

template <typename T>
static int launch_attn_t(AttnParams &p, const AttnPlan &a, int dtype, cudaStream_t st)
{
    const int64_t ctas = p.batch.S * a.tiles * a.splits * p.cache.heads;
    if (ctas > 0x7fffffff)
        return DLRM_ERR_UNSUPPORTED;
    int s;
    if (a.kernel == kAttnTile)
        s = p.exp.k ? launch_kv8_attn_tile(p, dtype, ctas, st) : launch_kv_attn_tile(p, dtype, ctas, st);
    else
        s = p.exp.k ? launch_general<T, true>(p, ctas, st) : launch_general<T, false>(p, ctas, st);
    if (s != DLRM_OK)
        return s;
    if (a.splits > 1) {
        const int64_t need = ceil_div(p.batch.n * p.cache.heads * p.group, 8);
        kv_attn_join_kernel<T><<<(unsigned)(need < 65536 ? need : 65536), 256, 0, st>>>(p);
        count_launch(st);
    }
    return launch_status();
}

// The tensor-core kernels' copies are 16 bytes wide.  Heads of 129 to 256
// 16-bit elements take rows of 16 for any number of rows (one event of each of
// 64 users with 2000, 16 heads on 4 of 256: 100 us, the general kernel 823; 64
// new of 16: 293 and 4499).
static bool wide_rows(const AttnParams &p, int dtype)
{
    const int e = dtype == DLRM_F32 ? 4 : 8;
    auto ok = [e](const void *ptr, int64_t a, int64_t b) {
        return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && a % e == 0 && b % e == 0;
    };
    return p.d <= (dtype == DLRM_F32 ? 128 : 256) && p.d % e == 0 && ok(p.q.ptr, p.q.ts, p.q.hs) &&
           ok(p.out.ptr, p.out.ts, p.out.hs) &&
           ok(p.cache.k, p.cache.page_stride, p.cache.slot_stride) && ok(p.cache.v, p.cache.head_stride, 0);
}

// The part that a row sees at most, whatever the history's length: a window bounds it, and a sequence's rows.
static int64_t seen_bound(const AttnParams &p)
{
    const int64_t bound = p.window + (p.causal ? p.max_new : 0);
    return p.window > 0 && bound < p.max_len ? bound : p.max_len;
}

// A kernel that goes by tiles of rows and splits of positions, and the join.
static int launch_planned(AttnParams &p, AttnKernel kernel, int64_t seen, int dtype, void *workspace, cudaStream_t st)
{
    AttnPlan a = plan(kernel, p.batch.S, p.cache.heads, p.group, p.d, p.max_new, p.max_len);
    if (seen < p.max_len) {  // never more parts than the workspace, whose size knows no window
        const AttnPlan b = plan(kernel, p.batch.S, p.cache.heads, p.group, p.d, p.max_new, seen);
        if (b.splits <= a.splits)
            a = b;
    }
    p.rows = a.rows;
    p.tiles = a.tiles;
    p.split_len = a.split_len;
    p.splits = a.splits;
    p.part_o = static_cast<float *>(workspace);
    p.part_lse = p.part_o + (size_t)a.splits * p.batch.n * p.cache.heads * p.group * p.d;
    if (dtype == DLRM_F32)
        return launch_attn_t<float>(p, a, dtype, st);
    if (dtype == DLRM_F16)
        return launch_attn_t<__half>(p, a, dtype, st);
    return launch_attn_t<__nv_bfloat16>(p, a, dtype, st);
}

int launch_kv_attn(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    const bool cores = wide_rows(p, dtype);
    const int64_t rows = p.max_new * p.group, seen = seen_bound(p);
    // Rows of 16: for few of them a short history's keys and values stay in L2,
    // and more CTAs fit on an SM.  150 users, 8 heads of 128, 32 rows, rows of 16
    // against tiles: up to 100 events 51 and 73 us, up to 1000 105 and 113; 64
    // users, up to 2000: 101 and 37; 48 rows, up to 400: 90 and 88; heads of 64,
    // 32 rows, up to 100: 42 and 40.
    if (cores && (dtype == DLRM_F32 || p.d > 128 || rows <= 16 || (p.d > 64 && rows <= 32 && seen <= 1024)))
        return launch_kv_attn_few(p, dtype, workspace, st);
    return launch_planned(p, cores ? kAttnTile : kAttnGeneral, seen, dtype, workspace, st);
}

static bool even_rows(const HeadsView &h, int dtype)
{
    const int e = dtype == DLRM_F32 ? 4 : 8;
    return reinterpret_cast<uintptr_t>(h.ptr) % 16 == 0 && h.ts % e == 0 && h.hs % e == 0;
}

// What the tensor-core kernels over codes ask of rows and codes.
static bool kv8_even(const AttnParams &p, int dtype)
{
    const CacheView &c = p.cache;
    return p.d % 8 == 0 && even_rows(p.q, dtype) && even_rows(p.out, dtype) &&
           reinterpret_cast<uintptr_t>(c.k) % 16 == 0 && reinterpret_cast<uintptr_t>(c.v) % 16 == 0 &&
           c.page_stride % 16 == 0 && c.slot_stride % 16 == 0 && c.head_stride % 16 == 0;
}

// Whether a call may take tiles, and convert codes of long chunks.
bool kv8_tiles(const AttnParams &p, int dtype) { return dtype != DLRM_F32 && p.d % 16 == 0 && kv8_even(p, dtype); }

int launch_kv8_attn(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    const CacheView &c = p.cache;
    const int64_t rows = p.max_new * p.group, seen = seen_bound(p);
    const bool tile = kv8_tiles(p, dtype), few = kv8_even(p, dtype) && p.d <= (dtype == DLRM_F32 ? 128 : 256);
    int status;
    // Long chunks: the codes are converted once (heads of up to 128).  Sequences beside them that have up to 16 rows go in
    // rows of 16 instead, in a launch of their own, where the batch has fewer than 512 rows a sequence, so that there may be
    // many of them.  With that launch and without, us (bf16, 16 heads on 4 of 128, histories of 8192): one chunk of 2048
    // and 99 single events 352 and 870, and 31 192 and 367; 4 of 2048 and 60 users without new events (512 rows a
    // sequence) 397 and 392; 8 of up to 2048 on up to 8192 361 and 348; 16 of 300 to 500 on up to 4000 174 and 164.
    const size_t widened = widen_workspace(p.batch.S, c.heads, p.group, p.d, p.max_new, p.max_len);
    if (tile && widened > 0) {
        AttnParams others = p;
        others.most_new = 16 / p.group;
        if (others.most_new > 0 && p.batch.n * p.group < 512 * p.batch.S &&
            launch_kv8_attn_few(others, dtype, workspace, st, status)) {
            if (status != DLRM_OK)
                return status;
            p.from_new = others.most_new + 1;
        }
        status = launch_widen(p, dtype, workspace, st);
        return status != DLRM_OK ? status : launch_kv_attn(p, dtype, static_cast<char *>(workspace) + widened, st);
    }
    // Rows of 16, as with the 16-bit cache, but for heads above 128 too, rows of 16 against tiles (bf16, 8 heads on
    // 2 of 256): 96 users with 1500 and 12 rows 51 and 87 us; 16 with up to 4000 and 256 rows 113 and 72; 4 with
    // 4096 and 8192 rows 1678 and 280.
    if (few && (!tile || rows <= 16 || (p.d > 64 && p.d <= 128 && rows <= 32 && seen <= 1024)) &&
        launch_kv8_attn_few(p, dtype, workspace, st, status))
        return status;
    return launch_planned(p, tile ? kAttnTile : kAttnGeneral, seen, dtype, workspace, st);
}

}  // namespace dlrm
