// Attention over the paged cache for few rows: up to 16 (token, head of a
// group) rows of a sequence and cache head, as single tokens have.
//
// Such a call reads every key and value once and does little with each, so
// memory bounds it, and the design keeps loads in flight.  The positions of
// all (sequence, head) items are laid end to end in units of four warp blocks;
// a CTA takes an equal run of units, whatever the lengths, and its warps
// stream their blocks through rings of asynchronous 16-byte copies that do
// not stop between items.  Every lane reads back exactly the chunks it
// copied itself, so the rings need no barrier:
//  - scores: m16n8k16 MMAs, rows x 8 tokens.  The order of the summed elements is
//    free, so a lane's chunk of 8 elements of a key serves two MMA steps as
//    it is, with the query's chunks in the same order.
//  - output: m16n8k16 MMAs, rows x 8 columns, 16 tokens deep.  Which columns
//    form an MMA's 8 is free too: a lane's chunks of 8 columns of two tokens,
//    interleaved by byte permutes, are the operands of 8 MMAs.
// A warp keeps its own running maximum, sum and output; the four are joined
// in shared memory at an item's end.  An item that spans CTAs leaves
// normalised partial rows and log2 of their sums, which a second kernel joins.
#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

constexpr int kFewWarps = 4, kFewRows = 16, kFewStages = 3;
constexpr int kFewCtas = 304;      // two for each of 152 SMs
constexpr int kFewStageBytes = 8192;  // of a warp: keys and values of 16 tokens x 128 or 32 x 64
constexpr int kFewMinUnits = 4;    // of a CTA: less is not worth a join

template <typename T>
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One (sequence, head) item and its units [first, last).
struct FewItem {
    Sequence seq;
    int64_t s, first, last;
    int head, lo, hi;  // positions that its queries see
    const int32_t *pages;
};

// Positions that a sequence's queries see, and the units of one of its items
// (one at least where there are queries: their rows are written).
__device__ __forceinline__ int few_units(const AttnParams &p, const Sequence &q, int unit, int &lo, int &hi)
{
    lo = hi = 0;
    if (q.count == 0)
        return 0;
    hi = seen_hi(q, p.causal, q.count - 1);
    lo = seen_lo(seen_hi(q, p.causal, 0), p.window);
    return hi > lo ? (hi - lo + unit - 1) / unit : 1;
}

// Sets the item's sequence to s, the item to its head 0 from unit `first`;
// false where the sequence has no units.
__device__ __forceinline__ bool few_sequence(const AttnParams &p, FewItem &w, int64_t s, int64_t first, int unit)
{
    if (!read_sequence(p.batch, s, p.max_new, p.max_len, w.seq, nullptr))
        return false;
    const int units = few_units(p, w.seq, unit, w.lo, w.hi);
    w.s = s;
    w.head = 0;
    w.first = first;
    w.last = first + units;
    w.pages = p.batch.table + s * p.batch.table_stride;
    return units > 0;
}

__device__ __forceinline__ void few_next(const AttnParams &p, FewItem &w, int unit)
{
    if (++w.head < p.cache.heads) {
        const int64_t units = w.last - w.first;
        w.first = w.last;
        w.last += units;
        return;
    }
    const int64_t first = w.last;
    for (int64_t s = w.s + 1; s < p.batch.S; s++)
        if (few_sequence(p, w, s, first, unit))
            return;
    w.last = INT64_MAX;  // not reached: a CTA's units end with the last item's
}

// Units of a CTA when `total` are shared out.
__host__ __device__ __forceinline__ int64_t few_quota(int64_t total)
{
    const int64_t q = (total + kFewCtas - 1) / kFewCtas;
    return q < kFewMinUnits ? kFewMinUnits : q;
}

// The CTA's share of all units: sums every sequence's units (each thread a run
// of sequences), finds the item that holds the first unit of the share.  CTA
// 0 leaves the sums before each sequence in p.prefix for the join.
__device__ bool few_share(const AttnParams &p, FewItem &w, int64_t &u0, int64_t &u1, int unit)
{
    __shared__ int64_t sums[kFewWarps], found[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t run = (p.batch.S + kFewWarps * 32 - 1) / (kFewWarps * 32);
    const int64_t from = min(threadIdx.x * run, p.batch.S), to = min(from + run, p.batch.S);
    int64_t mine = 0;
    Sequence q;
    int lo, hi;
    for (int64_t s = from; s < to; s++)
        if (read_sequence(p.batch, s, p.max_new, p.max_len, q, blockIdx.x == 0 ? p.err : nullptr))
            mine += (int64_t)few_units(p, q, unit, lo, hi) * p.cache.heads;
    int64_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
        before += lane >= o ? x : 0;
    }
    if (lane == 31)
        sums[warp] = before;
    __syncthreads();
    int64_t total = 0;
    before -= mine;
    for (int i = 0; i < kFewWarps; i++) {
        before += i < warp ? sums[i] : 0;
        total += sums[i];
    }
    const int64_t quota = few_quota(total);
    u0 = min(blockIdx.x * quota, total);
    u1 = min(u0 + quota, total);
    const bool here = u0 < u1 && u0 >= before && u0 < before + mine;
    if (here || blockIdx.x == 0) {
        for (int64_t s = from; s < to; s++) {
            int64_t units = 0;
            if (read_sequence(p.batch, s, p.max_new, p.max_len, q, nullptr))
                units = (int64_t)few_units(p, q, unit, lo, hi) * p.cache.heads;
            if (here && u0 >= before && u0 < before + units) {
                found[0] = s;
                found[1] = before;
            }
            if (blockIdx.x == 0)
                p.prefix[s] = before;
            before += units;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0)
            p.prefix[p.batch.S] = total;
    }
    __syncthreads();
    if (u0 >= u1)
        return false;
    few_sequence(p, w, found[0], found[1], unit);
    while (u0 >= w.last)
        few_next(p, w, unit);
    return true;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kFewWarps * 32, 2)
kv_attn_few_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int TB = 2048 / DP, NB = TB / 16, UT = kFewWarps * TB;  // tokens of a warp's block, of a unit
    constexpr int KG = DP / 32, VS = DP / 64;  // 32-element groups of a key, 64-column sets of a value
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_m[kFewWarps][kFewRows], s_l[kFewWarps][kFewRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    uint8_t *ring = smem + warp * kFewStages * kFewStageBytes + lane * 16;
    float *merge = reinterpret_cast<float *>(smem + kFewWarps * kFewStages * kFewStageBytes);  // [2][DP/2][32]

    FewItem it;  // of the unit being computed; `is`: of the unit whose addresses come next
    int64_t u0 = 0, u1;
    bool split = p.splits > 1;
    if (split) {
        if (!few_share(p, it, u0, u1, UT))
            return;
    } else {
        const int64_t s = blockIdx.x / p.cache.heads;
        if (!read_sequence(p.batch, s, p.max_new, p.max_len, it.seq, p.err) || !few_sequence(p, it, s, 0, UT))
            return;
        it.head = (int)(blockIdx.x - s * p.cache.heads);
        u1 = it.last;
    }
    FewItem is = it;

    // this lane's token of the warp's block of unit u: its place in the cache,
    // -1 for a position that no query sees or an invalid page
    auto place = [&](int64_t u) -> int64_t {
        if (u >= u1)
            return -1;
        while (u >= is.last)
            few_next(p, is, UT);
        const int at = is.lo + (int)(u - is.first) * UT + warp * TB + lane;
        if (lane >= TB || at >= is.hi)
            return -1;
        const int64_t o = slot_offset<T>(p.cache, is.pages, at, is.head);
        if (o < 0)
            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
        return o;
    };
    auto copy = [&](int stage, int64_t mine) {
        uint8_t *to = ring + stage * kFewStageBytes;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const int64_t o = __shfl_sync(0xffffffffu, mine, nb * 16 + t * 8 + g);
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const int e = 32 * i + 8 * q;
                    const bool ok = o >= 0 && e < p.d;
                    tc::cp_async16(to, p.cache.k + (ok ? o + e * 2 : 0), ok);
                    to += 512;
                }
            }
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const int64_t o = __shfl_sync(0xffffffffu, mine, nb * 16 + 2 * q + (t & 1) + (t >> 1) * 8);
#pragma unroll
                for (int i = 0; i < VS; i++) {
                    const int e = 64 * i + 8 * g;
                    const bool ok = o >= 0 && e < p.d;
                    tc::cp_async16(to, p.cache.v + (ok ? o + e * 2 : 0), ok);
                    to += 512;
                }
            }
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    int64_t next = place(u0);
#pragma unroll
    for (int i = 0; i < kFewStages - 1; i++) {
        if (u0 + i < u1)
            copy(i, next);
        commit();
        next = place(u0 + i + 1);
    }

    uint32_t qa[KG][8];      // queries: rows g and g + 8, two MMA steps a group
    float o[VS][8][4], m[2], l[2];
    int lo[2], hi[2], rows = 0;
    bool fresh = true, first_item = true;
    int stage = 0;
    for (int64_t u = u0; u < u1; u++) {
        if (fresh) {
            rows = it.seq.count * p.group;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = g + 8 * h, t = r / p.group;
                m[h] = -INFINITY;
                l[h] = 0.f;
                hi[h] = r < rows ? seen_hi(it.seq, p.causal, t) : 0;
                lo[h] = seen_lo(hi[h], p.window);
                const T *src = p.q.row<T>(it.seq.first + (r < rows ? t : 0),
                                          r < rows ? it.head * p.group + r - t * p.group : 0);
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const int e = 32 * i + 8 * q;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < rows && e < p.d)
                        x = *reinterpret_cast<const uint4 *>(src + e);
                    qa[i][h] = x.x;
                    qa[i][h + 2] = x.y;
                    qa[i][h + 4] = x.z;
                    qa[i][h + 6] = x.w;
                }
            }
#pragma unroll
            for (int i = 0; i < VS * 32; i++)
                (&o[0][0][0])[i] = 0.f;
            fresh = false;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 2) : "memory");
        {
            const int into = stage == 0 ? kFewStages - 1 : stage - 1;
            if (u + kFewStages - 1 < u1)
                copy(into, next);
            commit();
            next = place(u + kFewStages);
        }
        const uint4 *chunk = reinterpret_cast<const uint4 *>(ring + stage * kFewStageBytes);
        constexpr int kChunks = 2 * KG + 4 * VS;  // of 16 tokens
        const int at = it.lo + (int)(u - it.first) * UT + warp * TB;
        float s[NB][2][4];
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int t = 0; t < 2; t++) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s[nb][t][j] = 0.f;
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const uint4 k = chunk[(nb * kChunks + t * KG + i) * 32];
                    mma16816<T>(s[nb][t], qa[i], k.x, k.y);
                    mma16816<T>(s[nb][t], qa[i] + 4, k.z, k.w);
                }
            }
        // rows g (elements 0, 1) and g + 8 (elements 2, 3), tokens 2q and 2q + 1 of each 8
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int pos = at + nb * 16 + t * 8 + 2 * q + (j & 1), h = j >> 1;
                    const float x = pos >= lo[h] && pos < hi[h] ? s[nb][t][j] * p.scale_log2 : -INFINITY;
                    s[nb][t][j] = x;
                    top[h] = fmaxf(top[h], x);
                }
        float base[2];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            top[h] = fmaxf(top[h], m[h]);
            base[h] = top[h] == -INFINITY ? 0.f : top[h];
            moved |= top[h] > m[h];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const float f = exp2_approx(m[h] - base[h]);
                l[h] *= f;
                m[h] = top[h];
#pragma unroll
                for (int i = 0; i < VS; i++)
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        o[i][j][2 * h] *= f;
                        o[i][j][2 * h + 1] *= f;
                    }
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            uint32_t pa[4];  // the weights, rounded to the type; their sum is of the unrounded ones
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float x = exp2_approx(s[nb][t][2 * h] - base[h]);
                    const float y = exp2_approx(s[nb][t][2 * h + 1] - base[h]);
                    l[h] += x + y;
                    pa[2 * t + h] = pack2<T>(x, y);
                }
#pragma unroll
            for (int i = 0; i < VS; i++) {
                uint4 v[4];
#pragma unroll
                for (int t = 0; t < 4; t++)
                    v[t] = chunk[(nb * kChunks + 2 * KG + t * VS + i) * 32];
                const uint32_t *w0 = &v[0].x, *w1 = &v[1].x, *w2 = &v[2].x, *w3 = &v[3].x;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    mma16816<T>(o[i][2 * j], pa, __byte_perm(w0[j], w1[j], 0x5410), __byte_perm(w2[j], w3[j], 0x5410));
                    mma16816<T>(o[i][2 * j + 1], pa, __byte_perm(w0[j], w1[j], 0x7632),
                                __byte_perm(w2[j], w3[j], 0x7632));
                }
            }
        }
        stage = stage + 1 == kFewStages ? 0 : stage + 1;
        if (u + 1 < it.last && u + 1 < u1)
            continue;

        // the item's (or the CTA's) last unit: join the warps
#pragma unroll
        for (int h = 0; h < 2; h++) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (q == 0) {
                s_m[warp][g + 8 * h] = m[h];
                s_l[warp][g + 8 * h] = l[h];
            }
        }
        __syncthreads();
        float lse[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float all = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kFewWarps; i++)
                all = fmaxf(all, s_m[i][g + 8 * h]);
            const float b = all == -INFINITY ? 0.f : all;
#pragma unroll
            for (int i = 0; i < kFewWarps; i++)
                sum = fmaf(s_l[i][g + 8 * h], exp2_approx(s_m[i][g + 8 * h] - b), sum);
            const float f = sum > 0.f ? exp2_approx(m[h] - b) / sum : 0.f;
            lse[h] = sum > 0.f ? all + log2f(sum) : -INFINITY;
#pragma unroll
            for (int i = 0; i < VS; i++)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    o[i][j][2 * h] *= f;
                    o[i][j][2 * h + 1] *= f;
                }
        }
        float *flat = &o[0][0][0];
        if (warp >= 2)
#pragma unroll
            for (int i = 0; i < VS * 32; i++)
                merge[((warp - 2) * VS * 32 + i) * 32 + lane] = flat[i];
        __syncthreads();
        if (warp < 2)
#pragma unroll
            for (int i = 0; i < VS * 32; i++)
                flat[i] += merge[(warp * VS * 32 + i) * 32 + lane];
        if (warp == 1)
#pragma unroll
            for (int i = 0; i < VS * 32; i++)
                merge[(VS * 32 + i) * 32 + lane] = flat[i];
        __syncthreads();
        if (warp == 0) {
            const bool whole = it.first >= u0 && it.last <= u1;
            const int heads = p.cache.heads * p.group, slot = blockIdx.x * 2 + (first_item ? 0 : 1);
#pragma unroll
            for (int i = 0; i < VS * 32; i++)
                flat[i] += merge[(VS * 32 + i) * 32 + lane];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = g + 8 * h, t = r / p.group, head = it.head * p.group + r - t * p.group;
                if (r >= rows)
                    continue;
                if (q == 0) {
                    if (!whole)
                        p.part_lse[slot * p.rows + r] = lse[h];
                    else if (p.lse)
                        p.lse[(it.seq.first + t) * heads + head] = lse[h] * kLn2;
                }
#pragma unroll
                for (int i = 0; i < VS; i++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {  // columns e .. e + 7
                        const int e = 64 * i + 16 * q + 8 * c;
                        if (e >= p.d)
                            continue;
                        float x[8];
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            x[j] = o[i][j][2 * h + c];
                        if (whole) {
                            *reinterpret_cast<uint4 *>(p.out.row<T>(it.seq.first + t, head) + e) =
                                make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]),
                                           pack2<T>(x[6], x[7]));
                        } else {
                            float4 *to = reinterpret_cast<float4 *>(p.part_o + ((int64_t)slot * p.rows + r) * p.d + e);
                            to[0] = make_float4(x[0], x[1], x[2], x[3]);
                            to[1] = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
            }
        }
        fresh = true;
        first_item = false;
        if (u + 1 < u1)
            few_next(p, it, UT);
    }
}

// Joins the items that span CTAs: a warp per row of an item.
template <typename T>
__global__ void __launch_bounds__(128)
kv_attn_few_join_kernel(const __grid_constant__ AttnParams p)
{
    const int lane = threadIdx.x & 31, heads = p.cache.heads * p.group;
    const int64_t quota = few_quota(p.prefix[p.batch.S]), most = p.max_new * p.group;
    const int64_t all = p.batch.S * p.cache.heads * most;
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); i < all; i += (int64_t)gridDim.x * 4) {
        const int64_t item = i / most, s = item / p.cache.heads;
        const int r = (int)(i - item * most), head = (int)(item - s * p.cache.heads), t = r / p.group;
        const int64_t before = p.prefix[s], units = (p.prefix[s + 1] - before) / p.cache.heads;
        const int64_t first = before + head * units, c0 = first / quota, c1 = (first + units - 1) / quota;
        const int64_t token = p.batch.offsets[s] + t;
        if (units == 0 || c0 == c1 || token >= p.batch.offsets[s + 1])
            continue;
        // the first CTA's part is its last item's unless the item begins with it
        auto row = [&](int64_t c) { return (c * 2 + (c == c0 && c0 * quota < first ? 1 : 0)) * most + r; };
        float top = -INFINITY;
        for (int64_t c = c0 + lane; c <= c1; c += 32)
            top = fmaxf(top, p.part_lse[row(c)]);
        top = warp_max(top);
        const float base = top == -INFINITY ? 0.f : top;
        float total = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int64_t c = c0; c <= c1; c++) {
            const float f = exp2_approx(p.part_lse[row(c)] - base);
            const float *o = p.part_o + row(c) * p.d;
            total += f;
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (lane + 32 * j < p.d)
                    acc[j] = fmaf(o[lane + 32 * j], f, acc[j]);
        }
        const float inv = total > 0.f ? 1.f / total : 0.f;
        const int h = head * p.group + r - t * p.group;
        T *out = p.out.row<T>(token, h);
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (lane + 32 * j < p.d)
                out[lane + 32 * j] = from_f32<T>(acc[j] * inv);
        if (p.lse && lane == 0)
            p.lse[token * heads + h] = total > 0.f ? (top + log2f(total)) * kLn2 : -INFINITY;
    }
}

// Histories longer than this are shared out over CTAs in equal runs.
constexpr int64_t kFewWhole = 1024;

bool few_splits(int64_t max_len) { return max_len > kFewWhole; }

size_t few_workspace(int64_t S, int64_t rows, int d, int64_t max_len)
{
    if (!few_splits(max_len) || rows > kFewRows)
        return 0;
    return (size_t)2 * kFewCtas * rows * (d + 1) * sizeof(float) + (size_t)(S + 2) * sizeof(int64_t);
}

template <typename T, int DP>
static int launch_few(AttnParams &p, void *workspace, cudaStream_t st)
{
    constexpr int smem = kFewWarps * kFewStages * kFewStageBytes + 2 * DP / 2 * 32 * 4;
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv_attn_few_kernel<T, DP>, smem, &done);
    if (s != DLRM_OK)
        return s;
    const bool split = few_splits(p.max_len);
    p.splits = split ? 2 : 1;
    p.prefix = static_cast<int64_t *>(workspace);
    p.part_o = reinterpret_cast<float *>(p.prefix + ((p.batch.S + 2) & ~(int64_t)1));
    p.rows = (int)(p.max_new * p.group);
    p.part_lse = p.part_o + (size_t)2 * kFewCtas * p.rows * p.d;
    const int64_t items = p.batch.S * p.cache.heads;
    if (items > 0x7fffffff)
        return DLRM_ERR_UNSUPPORTED;
    kv_attn_few_kernel<T, DP><<<(unsigned)(split ? kFewCtas : items), kFewWarps * 32, smem, st>>>(p);
    count_launch(st);
    if (split) {
        const int64_t need = (items * p.max_new * p.group + 3) / 4;
        kv_attn_few_join_kernel<T><<<(unsigned)(need < 65536 ? need : 65536), 128, 0, st>>>(p);
        count_launch(st);
    }
    return launch_status();
}

int launch_kv_attn_few(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    if (dtype == DLRM_F16)
        return p.d <= 64 ? launch_few<__half, 64>(p, workspace, st) : launch_few<__half, 128>(p, workspace, st);
    return p.d <= 64 ? launch_few<__nv_bfloat16, 64>(p, workspace, st)
                     : launch_few<__nv_bfloat16, 128>(p, workspace, st);
}

}  // namespace dlrm
