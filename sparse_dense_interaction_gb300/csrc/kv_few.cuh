// Shared by the kernels of attention by rows of 16: the items, how they are
// shared out over CTAs, the MMAs and the join of items that span CTAs.
#pragma once

#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

constexpr int kFewWarps = 4, kFewRows = 16;
constexpr int kFewSms = 152, kFewMaxCtas = 3 * kFewSms;
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

// One item -- row tile `tile` of a sequence and head -- and its units
// [first, last).  Every tile of a sequence has the same units, those of the
// positions that any of its queries sees, so that a CTA finds its share by
// division.  That is right for one tile; of a causal chunk of many tiles it is
// twice what they see, and more with a window (fp32, 4 sequences of 2048 new, 4 heads on
// 2 of 64: 397 us, with a window of 128 too, where a tile sees 135 of 2176).
struct FewItem {
    Sequence seq;
    int64_t s;
    int first, last;
    int head, tile, tiles;
    int lo, hi, lo_seen;  // positions that the sequence's queries see, lo down to a multiple of `align`
    const int32_t *pages;
};

// New tokens of a sequence that this launch takes, at most.
__host__ __device__ __forceinline__ int64_t few_new(const AttnParams &p)
{
    return p.max_new < p.most_new ? p.max_new : p.most_new;
}

// Positions that a sequence's queries see, and the units of one of its items
// (one at least where there are queries: their rows are written).
__device__ __forceinline__ int few_units(const AttnParams &p, const Sequence &q, int unit, int &lo, int &hi, int align)
{
    lo = hi = 0;
    if (q.count == 0 || !attn_takes(p, q))
        return 0;
    hi = seen_hi(q, p.causal, q.count - 1);
    lo = seen_lo(seen_hi(q, p.causal, 0), p.window);
    return hi > lo ? (hi - (lo & -align) + unit - 1) / unit : 1;
}

__device__ __forceinline__ int few_tiles(const AttnParams &p, const Sequence &q)
{
    return (int)(((int64_t)q.count * p.group + kFewRows - 1) / kFewRows);
}

// Sets the item to sequence s's first, from unit `first`; false where the
// sequence has no units.
__device__ __forceinline__ bool few_sequence(const AttnParams &p, FewItem &w, int64_t s, int first, int unit, int align)
{
    if (!read_sequence(p.batch, s, p.max_new, p.max_len, w.seq, nullptr))
        return false;
    const int units = few_units(p, w.seq, unit, w.lo_seen, w.hi, align);
    w.lo = w.lo_seen & -align;
    w.s = s;
    w.head = w.tile = 0;
    w.tiles = few_tiles(p, w.seq);
    w.first = first;
    w.last = first + units;
    w.pages = p.batch.table + s * p.batch.table_stride;
    return units > 0;
}

// Sequences of a thread when the batch's are shared out over a CTA.
__device__ __forceinline__ int few_run(const AttnParams &p)
{
    return (int)((p.batch.S + kFewWarps * 32 - 1) / (kFewWarps * 32));
}

// The first sequence after `s` that has new tokens, by a whole warp; -1: none.  Idle sequences (slots of users
// who wait) are passed over 32 at a time, then whole runs of them (busy: the first sequence with new tokens of
// each run, -1: none).  Two users with 200000 events, 12000 idle ones between them: 103 us, the search for the
// CTAs' shares; read one by one 4930.  Not inlined: it is rare, and its copies would cost registers.
static __device__ __noinline__ int few_busy_after(const AttnParams &p, int s0, const int *busy)
{
    const int lane = threadIdx.x & 31, S = (int)p.batch.S, run = few_run(p), here = s0 / run;
    const int end = min((here + 1) * run, S);
    int next = -1;
    for (int s = s0 + 1; s < end && next < 0; s += 32) {
        Sequence mine;
        const bool some = s + lane < end && read_sequence(p.batch, s + lane, p.max_new, p.max_len, mine, nullptr) &&
                          mine.count > 0 && attn_takes(p, mine);
        const uint32_t found = __ballot_sync(0xffffffffu, some);
        next = found ? s + __ffs(found) - 1 : -1;
    }
    for (int r = here + 1; r < kFewWarps * 32 && next < 0; r += 32) {
        const int mine = r + lane < kFewWarps * 32 ? busy[r + lane] : -1;
        const uint32_t found = __ballot_sync(0xffffffffu, mine >= 0);
        next = found ? __shfl_sync(0xffffffffu, mine, __ffs(found) - 1) : -1;
    }
    return next;
}

// The next item, by a whole warp.
__device__ __forceinline__ void few_next(const AttnParams &p, FewItem &w, int unit, int align, const int *busy)
{
    if (++w.tile == w.tiles) {
        w.tile = 0;
        w.head++;
    }
    if (w.head < p.cache.heads) {
        const int units = w.last - w.first;
        w.first = w.last;
        w.last += units;
        return;
    }
    const int first = w.last, next = few_busy_after(p, (int)w.s, busy);
    if (next >= 0 && few_sequence(p, w, next, first, unit, align))
        return;
    w.last = 0x7fffffff;  // not reached: a CTA's units end with the last item's
}

// Units of a CTA when `total` are shared out.
__host__ __device__ __forceinline__ int64_t few_quota(int64_t total, int ctas)
{
    const int64_t q = (total + ctas - 1) / ctas;
    return q < kFewMinUnits ? kFewMinUnits : q;
}

// The CTA's share of all units: sums every sequence's units (each thread a run
// of sequences), finds the item that holds the first unit of the share.
static __device__ bool few_share(const AttnParams &p, FewItem &w, int &units, int &quota_units, int unit, int align, int *busy)
{
    __shared__ int64_t sums[kFewWarps], found[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t run = few_run(p);
    const int64_t from = min(threadIdx.x * run, p.batch.S), to = min(from + run, p.batch.S);
    int64_t mine = 0;
    Sequence q;
    int lo, hi, first = -1;
    for (int64_t s = from; s < to; s++)
        if (read_sequence(p.batch, s, p.max_new, p.max_len, q, blockIdx.x == 0 ? p.err : nullptr)) {
            mine += (int64_t)few_units(p, q, unit, lo, hi, align) * few_tiles(p, q) * p.cache.heads;
            first = first < 0 && q.count > 0 && attn_takes(p, q) ? (int)s : first;
        }
    busy[threadIdx.x] = first;
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
    const int64_t quota = few_quota(total, gridDim.x);
    const int64_t u0 = min(blockIdx.x * quota, total);
    units = (int)(min(u0 + quota, total) - u0);
    quota_units = (int)quota;
    const bool here = units > 0 && u0 >= before && u0 < before + mine;
    for (int64_t s = from; here && s < to; s++) {
        int64_t here_units = 0;
        if (read_sequence(p.batch, s, p.max_new, p.max_len, q, nullptr))
            here_units = (int64_t)few_units(p, q, unit, lo, hi, align) * few_tiles(p, q) * p.cache.heads;
        if (u0 >= before && u0 < before + here_units) {
            found[0] = s;
            found[1] = before;
        }
        before += here_units;
    }
    __syncthreads();
    if (units == 0)
        return false;
    // the sequence's items before it may be many: their units are counted from the share's
    // first in 64 bits, the item's own fit in 32
    few_sequence(p, w, found[0], 0, unit, align);
    const int64_t each = w.last, skip = (u0 - found[1]) / each;
    w.tile = (int)(skip % w.tiles);
    w.head = (int)(skip / w.tiles);
    w.first = (int)(found[1] + skip * each - u0);
    w.last = w.first + (int)each;
    return true;
}

// The cache as bulk tensor copies see it: (element, slot, head, page).
struct FewMaps {
    CUtensorMap k, v;
    int rows;  // of a box
};

// Transposes an 8 x 8 matrix of 16-bit elements over a warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Joins the items that span CTAs: CTA x of this kernel the item that the
// main kernel's CTA x began and did not end, row blockIdx.y of it.  A warp
// sums every eighth part, 4 columns a lane (and 4 more of wide heads).
constexpr int kJoinWarps = 8;

template <typename T, int kHalves>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv_attn_few_join_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float4 sums[kJoinWarps][kHalves][32];
    __shared__ float weights[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = p.cache.heads * p.group;
    const FewJoin j = p.joins[blockIdx.x];
    if ((int)blockIdx.y >= j.rows)
        return;
    // its parts: of the first CTA the one it says, of the others their first
    const int c0 = blockIdx.x, c1 = j.last;
    auto row = [&](int c) { return (int64_t)(c == c0 ? j.first : c * 2) * p.rows + blockIdx.y; };
    float top = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32)
        top = fmaxf(top, p.part_lse[row(c)]);
    top = warp_max(top);
    const float base = top == -INFINITY ? 0.f : top;
    float weight = 0.f;
    float4 sum[kHalves];
#pragma unroll
    for (int i = 0; i < kHalves; i++)
        sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = c0 + warp; c <= c1; c += kJoinWarps) {
        const float f = exp2_approx(p.part_lse[row(c)] - base);
        weight += f;
#pragma unroll
        for (int i = 0; i < kHalves; i++)
            if (i * 128 + lane * 4 < p.d) {
                const float4 x = *reinterpret_cast<const float4 *>(p.part_o + row(c) * p.d + i * 128 + lane * 4);
                sum[i] = make_float4(fmaf(x.x, f, sum[i].x), fmaf(x.y, f, sum[i].y), fmaf(x.z, f, sum[i].z),
                                     fmaf(x.w, f, sum[i].w));
            }
    }
#pragma unroll
    for (int i = 0; i < kHalves; i++)
        sums[warp][i][lane] = sum[i];
    if (lane == 0)
        weights[warp] = weight;
    __syncthreads();
    if (warp != 0)
        return;
    weight = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; w++)
        weight += weights[w];
    const float inv = weight == 0.f ? 0.f : 1.f / weight;
    const int r = j.row + blockIdx.y, t = r / p.group, h = j.head + r - t * p.group;
    const int64_t token = j.token + t;
#pragma unroll
    for (int i = 0; i < kHalves; i++)
        if (i * 128 + lane * 4 < p.d) {
            float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kJoinWarps; w++) {
                const float4 x = sums[w][i][lane];
                all = make_float4(all.x + x.x, all.y + x.y, all.z + x.z, all.w + x.w);
            }
            T *out = p.out.row<T>(token, h) + i * 128 + lane * 4;
            out[0] = from_f32<T>(all.x * inv);
            out[1] = from_f32<T>(all.y * inv);
            out[2] = from_f32<T>(all.z * inv);
            out[3] = from_f32<T>(all.w * inv);
        }
    if (p.lse && lane == 0)
        p.lse[token * heads + h] = weight == 0.f ? -INFINITY : (top + log2f(weight)) * kLn2;
}

// Whether the positions are shared out in equal runs, or an item is a CTA's
// whole.  Runs keep every CTA busy whatever the lengths; whole items need no
// search for the CTA's share and no join, their CTAs start and end beside one
// another, and an SM that is faster takes more of them.  Against that stands
// the last CTAs' unevenness, a part of the time in which a CTA reads the
// longest item.  So short items stay whole, and longer ones where there are
// more to even them out.  bf16, whole against runs: 64 users with up to 2000
// events, 8 heads of 64: 35 and 48 us; 256 users 98 and 128; 512 users with up to
// 4000, 4 heads of 128: 326 and 352; 256 with up to 8192: 335 and 328; 64 users with
// up to 8000, 2 heads of 64: 65 and 39; one with 3000: 26 and 16.
constexpr int64_t kFewWholeBytes = 384 << 10, kFewWholeBytesPerItem = 3 << 10;

inline bool few_splits(int64_t seen, int d, int es, int64_t items, int64_t whole = kFewWholeBytes,
                       int64_t per_item = kFewWholeBytesPerItem)
{
    return seen * d * 2 * es > whole + items * per_item;
}

inline int64_t few_rows(int64_t rows) { return rows < kFewRows ? rows : kFewRows; }

}  // namespace dlrm
