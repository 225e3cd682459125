// Shared by the event-history kernels: kernel-parameter views of the host
// structs, the paged cache's addressing, the search for a token's sequence.
#pragma once

#include "common.cuh"
#include "dlrm_history.h"

namespace dlrm {

struct HeadsView {
    char *ptr;
    int64_t ts, hs;  // elements
    int heads;

    template <typename T>
    __device__ __forceinline__ T *row(int64_t token, int h) const
    {
        return reinterpret_cast<T *>(ptr) + token * ts + h * hs;
    }
};

struct RopeView {
    const float *table;  // null: no rotation
    int64_t length;
    const int64_t *positions;
    int rot;
    bool interleaved;
};

// x / d for x < 2^31: one multiplication and one shift.
struct FastDiv {
    uint32_t d, mul, shift;

    __host__ static FastDiv make(uint32_t d)
    {
        FastDiv f;
        f.d = d;
        f.shift = 0;
        while ((1ull << f.shift) < d)
            f.shift++;
        f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
        return f;
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const { return (__umulhi(x, mul) + x) >> shift; }
};

struct CacheView {
    char *k, *v;
    int64_t page_stride, slot_stride, head_stride;  // elements
    uint32_t pages;
    FastDiv page;  // divides a position by the page size
    int heads;
};

// Exponents of a cache in 8 bits, one for each block of a page's slots and head.
struct ExpView {
    uint8_t *k, *v;
    int64_t page_stride, block_stride, head_stride;
    FastDiv block;  // divides a slot by the block's size
};

struct BatchView {
    int64_t S, n;
    const int64_t *offsets, *lengths;
    const int32_t *table;
    int64_t table_stride, capacity;  // capacity: positions a table row can hold
};

// One sequence of the batch: first new token, new tokens, stored tokens.
struct Sequence {
    int64_t first;
    int count, length;

    // offsets that are not monotone lead the searches below anywhere
    __device__ __forceinline__ bool has(int64_t token) const { return token >= first && token < first + count; }
};

// Reads sequence s; false (with the flag raised) where the batch's numbers
// contradict each other or the bounds.  The flag is also raised where the first
// or the last sequence leaves tokens to nobody.
__device__ __forceinline__ bool read_sequence(const BatchView &b, int64_t s, int64_t max_new, int64_t max_len,
                                              Sequence &q, int32_t *err)
{
    const int64_t f = b.offsets[s], e = b.offsets[s + 1], len = b.lengths[s];
    if (f < 0 || e < f || e > b.n || e - f > max_new || len < 0 || len > max_len || len > b.capacity) {
        raise_flag(err, DLRM_FLAG_BAD_OFFSETS);
        return false;
    }
    if (err && ((s == 0 && f != 0) || (s == b.S - 1 && e != b.n)))
        raise_flag(err, DLRM_FLAG_BAD_OFFSETS);
    q.first = f;
    q.count = (int)(e - f);
    q.length = (int)len;
    return true;
}

// Raises the flag for this thread's share of the sequences, with and without new
// tokens, if they are to be appended (attention reads every sequence anyway).
__device__ __forceinline__ void check_sequences(const BatchView &b, int64_t thread, int64_t threads, int32_t *err)
{
    Sequence q;
    for (int64_t s = thread; err && s < b.S; s += threads)
        if (read_sequence(b, s, b.n, b.capacity, q, err) && q.count > q.length)
            raise_flag(err, DLRM_FLAG_BAD_OFFSETS);
}

// The last sequence that starts at or before token i, by one warp: 32 probes
// a step, so two steps up to 1024 sequences.  -1 where there is none.
__device__ __forceinline__ int64_t find_sequence(const BatchView &b, int64_t i)
{
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = b.S;
    while (true) {
        const int64_t step = (hi - lo + 31) >> 5;
        const int64_t at = lo + lane * step;
        const int c = __popc(__ballot_sync(0xffffffffu, at < hi && b.offsets[at] <= i));
        if (c == 0)
            return -1;
        lo += (c - 1) * step;
        if (step == 1)
            return lo;
        hi = lo + step < hi ? lo + step : hi;
    }
}

// The positions that the queries first .. last of a sequence see: [lo, hi).
__device__ __forceinline__ int seen_hi(const Sequence &q, bool causal, int i)
{
    const int hi = causal ? q.length - q.count + i + 1 : q.length;
    return hi < 0 ? 0 : hi;
}
__device__ __forceinline__ int seen_lo(int hi, int window) { return window > 0 && hi > window ? hi - window : 0; }

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// 2^x by the hardware's approximation (relative error about 2^-22).
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

constexpr float kLn2 = 0.69314718055994530942f;

// log2 of the largest weight that the 16-bit kernels keep.  A weight 2^(s - m) of
// at most 1 wastes half of fp16's range: from 2^-14 on it is subnormal and below
// 2^-25 it is gone, while the sum still counts it (40000 such weights under one
// strong key lost all that they gather).  So fp16 weights are lifted to 2^15;
// sum and output carry the same factor.  bf16 has fp32's range.  The maxima are
// rounded up and the lifted exponents down, so that no weight exceeds it.
template <typename T>
constexpr float kWeightTop = 0.f;
template <>
constexpr float kWeightTop<__half> = 15.f;

// The attention's launch: which kernel, rows (token, head of a group) of a
// tile, and how the positions are split.
enum AttnKernel { kAttnGeneral, kAttnTile };

// Rows of the tensor-core tiles: two query tiles of 128 on an SM of their own;
// with heads of 64 and at most 256 rows in all (the candidates of a user) one,
// and two CTAs on an SM, so that one starts and ends while the other computes.
// More rows keep the pair, which reads keys and values once for both tiles.  us
// with one and with two query tiles, f16, 8 heads of 64, users with up to so many events:
//   64 users    128 rows     256 rows     400 rows     800 rows
//      500      23.4  33.9   34.0  39.8   47.9  46.6   85.5  83.0
//     2000      41.2  58.8   57.2  64.1   97.1  91.2    159   146
//     8000       109   147    160   167    225   204    365   327
// 256 users of 4 heads and up to 250 events: 48.3 and 50.2, 49.2 and 56.4, 78.9 and 79.0, 127 and 122.  Only
// where the pairs already fit beside one another is one tile worse at few rows (64 users of 2 heads,
// 4 query heads each, up to 250 events, 128 rows: 15.8 and 12.5).
// Heads above 128 (a cache in 8 bits alone) leave room for one, and for one CTA on an SM.
inline int tile_rows(int64_t rows, int d) { return d > 128 || (d <= 64 && rows <= 256) ? 128 : 256; }
// CTAs that run at once
__host__ __device__ constexpr int tile_places(int rows, int d) { return rows == 128 && d <= 64 ? 2 * 152 : 152; }

struct AttnPlan {
    AttnKernel kernel;
    int rows;        // rows of a tile
    int64_t tiles;   // row tiles of a sequence, at most
    int split_len;   // positions of a split
    int splits;      // at most
};

// An item of up to 16 rows that a CTA began and the ones after it went on with.
struct FewJoin {
    int64_t token;         // the sequence's first new token
    int head, row, rows;   // its first query head, first row and rows (0: there is no such item)
    int first, last;       // the CTA's own part; the last CTA
    int unused;
};

struct AttnParams {
    HeadsView q, out;
    BatchView batch;
    CacheView cache;
    int64_t max_new, max_len;
    int from_new, most_new;  // this launch takes the sequences of so many new tokens, and leaves the others to another
    int d, group;       // group: query heads of a cache head
    float scale_log2;   // scale * log2(e)
    bool causal;
    int window;
    float *lse;         // [n][q heads] or null
    int rows, split_len, splits;
    int64_t tiles;
    float *part_o, *part_lse;  // [splits][n][q heads]([d]): partial rows, log2 of their sums
    FewJoin *joins;            // rows of 16: an item that each CTA left unfinished
    int wait_polls;            // of a wait inside a kernel, before it gives up
    int32_t *err;
    ExpView exp;               // of a cache in 8 bits
    // of a 16-bit copy of such a cache, [sequence][page][head]: exponents that a page's keys (low byte; bf16 keys are
    // as they are) and values are relative to
    const uint16_t *refs;
};

__device__ __forceinline__ bool attn_takes(const AttnParams &p, const Sequence &q)
{
    return q.count >= p.from_new && q.count <= p.most_new;
}

// What one CTA works on: rows of tile `tile` of head `head` of the sequence,
// positions [lo, hi) of split `split`; whole: the tile needs no other split.
struct AttnWork {
    Sequence seq;
    int64_t s;
    int head, split, row0, rows, lo, hi;
    bool whole;
};

// The first position of a tile's splits: the first that its first query sees,
// down to a multiple of 128.
__device__ __forceinline__ int split_base(const Sequence &q, bool causal, int window, int token)
{
    return seen_lo(seen_hi(q, causal, token), window) & ~127;
}

// The CTA's number: head fastest, then split, then tile, then sequence (or its
// rank); returns the last, sets the head and the split.
__device__ __forceinline__ int64_t attn_number(const AttnParams &p, uint32_t cta, AttnWork &w, int64_t &tile)
{
    const uint32_t hk = p.cache.heads, splits = p.splits, tiles = (uint32_t)p.tiles;
    w.head = (int)(cta % hk);
    cta /= hk;
    w.split = (int)(cta % splits);
    cta /= splits;
    tile = tiles - 1 - cta % tiles;  // the longest rows of a causal chunk first
    return cta / tiles;
}

// The rows and positions of a tile of the sequence w.seq; false where there is
// nothing to do.
__device__ __forceinline__ bool attn_rows(const AttnParams &p, int64_t tile, AttnWork &w)
{
    const int64_t row0 = tile * p.rows, all = (int64_t)w.seq.count * p.group;
    if (row0 >= all)
        return false;
    w.row0 = (int)row0;
    w.rows = (int)(all - row0 < p.rows ? all - row0 : p.rows);
    const int t0 = w.row0 / p.group, t1 = (w.row0 + w.rows - 1) / p.group;
    const int base = split_base(w.seq, p.causal, p.window, t0);
    const int hi = seen_hi(w.seq, p.causal, t1), lo = seen_lo(seen_hi(w.seq, p.causal, t0), p.window);
    w.whole = hi - base <= p.split_len;
    const int64_t from = (int64_t)base + (int64_t)w.split * p.split_len, to = from + p.split_len;
    if (w.split > 0 && from >= hi)
        return false;
    w.lo = from > lo ? (int)from : lo;
    w.hi = to < hi ? (int)to : hi;
    return true;
}

__device__ __forceinline__ bool attn_work(const AttnParams &p, uint32_t cta, AttnWork &w)
{
    int64_t tile;
    w.s = attn_number(p, cta, w, tile);
    return read_sequence(p.batch, w.s, p.max_new, p.max_len, w.seq, p.err) && attn_takes(p, w.seq) &&
           attn_rows(p, tile, w);
}

// Byte offset of a position's slot row in the cache (head's own offset
// included), or -1 for a page number outside the cache.
template <typename T>
__device__ __forceinline__ int64_t slot_offset(const CacheView &c, const int32_t *pages, int position, int head)
{
    const uint32_t page = c.page.div((uint32_t)position), slot = (uint32_t)position - page * c.page.d;
    const uint32_t id = (uint32_t)pages[page];
    if (id >= c.pages)
        return -1;
    return (id * c.page_stride + slot * c.slot_stride + head * c.head_stride) * (int64_t)sizeof(T);
}

}  // namespace dlrm
