// Attention over the paged cache for many rows: tiles of 256 (or 128) rows on
// the tensor cores.
//
// A CTA holds two query tiles of 128 packed rows and walks the positions in
// tiles of 128.  Warp roles:
//  - the warp after the softmax's copies keys and values into a ring of tiles
//    in the 128-byte swizzle, by bulk tensor copies through the page table
//    where pages are multiples of 8 slots, in boxes of the largest power of two
//    up to 128 that divides a page; the rows of a value tile that no query sees
//    may hold anything, so it overwrites them with zeros before it hands the
//    tile over.  Other page sizes: two warps copy row by row in asynchronous
//    16-byte copies and fill such rows with zeros without reading them;
//  - one thread of the last warp issues the MMAs: S = Q K^T (both operands in
//    shared memory, K-major) and O += P V (P in tensor memory, V MN-major as it
//    lies);
//  - the first 8 warps for each query tile are its softmax: a thread owns half
//    of a row's 128 scores, agrees on the row's maximum with the thread that
//    owns the other half, and writes the weights over the scores, in 16 bits
//    (one thread to a row, 8 warps in all: 3.5 % more time for long chunks).
// The two tiles take turns: while one's scores are exponentiated the other's
// MMAs run.  The running maximum a row is scaled by lags: the output (in
// tensor memory) and the sum are rescaled only when the maximum has grown by
// more than 2^8 (fp16: 2^4, which leaves more of its range to the weights), which
// rarely happens after the first tiles; a weight is then at most that much above
// 1, and sum and output carry the same factor, so nothing is lost.
// Tensor memory: scores 2 x 128 columns (the weights on top of them), output
// 2 x DP.
//
// 4 sequences of 2048 new events on 8192 (16 heads on 4, 128 bf16 elements):
// 355 us, 1350 TFLOP/s, 0.71 of a large matrix product's rate (0.79 of the rate
// that one keeps up for seconds): inside a CTA the tensor pipe is busy 80 % of
// the time, and the chip draws all the power it may.  Up to 200 candidates of
// each of 64 users with up to 2000 events (8 heads of 64 f16 elements): 53 us,
// where a CTA lives for 9 tiles of positions and its start, its end and the
// last CTAs' uneven ends count most.
#include "kv8.cuh"
#include "kv_tile.cuh"

namespace dlrm {

constexpr int kTileLag = 3;         // copied tiles that may be in flight before one is waited for

// Bulk tensor copies: keys and values as (element, slot, head, page) in boxes
// of `rows` slots; queries as (element, head, token) in boxes of one group's heads
// and 128 / group tokens, where a group divides 128 (q_rows: else row by row).
struct TileMaps {
    CUtensorMap k, v, q;
    int rows;
    bool q_rows;
};

// Copies 32 rows (this warp's) of a tile: lane t of the warp knows row t's
// byte offset from `base`, -1 for a row of zeros.
template <typename Sh>
__device__ __forceinline__ void copy_rows(uint8_t *tile, const char *base, int64_t mine, int row0, int d)
{
    constexpr int C = Sh::kChunks, kRows = 32 / C;  // rows of a step
    const int lane = threadIdx.x & 31, c = lane % C;
#pragma unroll
    for (int i = 0; i < C; i++) {
        const int r = i * kRows + lane / C;
        const int64_t o = __shfl_sync(0xffffffffu, mine, r);
        const bool ok = o >= 0 && c * 8 < d;
        tc::cp_async16(tile + (c >> 3) * Sh::kBlock + (row0 + r) * 128 + (((c & 7) ^ (r & 7)) << 4),
                       base + (ok ? o + c * 16 : 0), ok);
    }
}

// Copies the queries' rows (in groups of this call's threads: rows of zeros
// past the last; what lies in the groups after that reaches no output).
template <typename Sh, int kThreads>
__device__ __forceinline__ void copy_queries(const AttnParams &p, const AttnWork &w, uint8_t *sq)
{
    const int tid = threadIdx.x - Sh::kSoftmaxThreads, row0 = tid & ~31;
#pragma unroll 1
    for (int r0 = 0; r0 < w.rows; r0 += kThreads) {
        const int r = r0 + tid, row = w.row0 + r, token = row / p.group;
        const int64_t o = r < w.rows ? ((w.seq.first + token) * p.q.ts +
                                        (int64_t)(w.head * p.group + row - token * p.group) * p.q.hs) * 2
                                     : -1;
        copy_rows<Sh>(sq + (r0 >> 7) * Sh::kTileBytes, p.q.ptr, o, (r0 & 127) + row0, p.d);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// The copy warp, by bulk tensor copies.  A tile begins at a multiple of 128
// positions; lane i copies box i % boxes of the tile, if there are as many.
template <typename T, int DP, bool kTwo>
__device__ void tile_copy_bulk(const AttnParams &p, const AttnWork &w, const TileMaps &maps, uint8_t *sq,
                               uint8_t *ring, TileBars &b, int tiles)
{
    using Sh = TileShape<DP, kTwo>;
    constexpr int kColumns = DP / 64;
    const int lane = threadIdx.x & 31, start = w.lo & ~127, parts = kTilePos / maps.rows;
    const int32_t *pages = p.batch.table + w.s * p.batch.table_stride;
    // part i of tile j: its page number (-1: nothing of it is seen) and slot
    auto find = [&](int j, int i, int &page, int &slot) {
        const int at = start + j * kTilePos + i * maps.rows;
        page = -1;
        slot = 0;
        if (i < parts && at < w.hi && at + maps.rows > w.lo) {
            const uint32_t n = p.cache.page.div((uint32_t)at);
            slot = at - (int)(n * p.cache.page.d);
            page = __ldg(pages + n);
        }
    };
    int page, slot, next_page, next_slot;
    int patched = 0;  // value tiles mended so far
    auto left_behind = [&](int copied, int landing) {
        if (lane == 0) {
            b.copied = copied;
            b.landing = landing;
        }
    };
    find(0, lane, next_page, next_slot);
    if (maps.q_rows) {
        copy_queries<Sh, 32>(p, w, sq);
    } else if (lane == 0) {
        const int n = w.rows > 128 ? 2 : 1;
        tc::mbar_expect_tx(&b.q_full, n * Sh::kTileBytes);
        for (int t = 0; t < n; t++)
            for (int c = 0; c < kColumns; c++)
                tc::tma_load_3d(sq + t * Sh::kTileBytes + c * Sh::kBlock, &maps.q, c * 64, w.head * p.group,
                                (int)w.seq.first + (w.row0 + t * 128) / p.group, &b.q_full);
    }
    for (int j = 0; j < tiles; j++) {
        page = next_page;
        slot = next_slot;
        find(j + 1, lane, next_page, next_slot);
        const int at = start + j * kTilePos;
        const bool seen = at + lane * maps.rows < w.hi && at + (lane + 1) * maps.rows > w.lo;
        if (lane < parts && seen && (uint32_t)page >= p.cache.pages)
            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
        page = (uint32_t)page < p.cache.pages ? page : -1;  // outside the map: zeros
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            const int i = 2 * j + kv, ring_slot = i % Sh::kSlots;
            uint8_t *tile = ring + ring_slot * Sh::kTileBytes;
            if (i >= Sh::kSlots && !warp_wait(&b.empty[ring_slot], (i / Sh::kSlots - 1) & 1, &b.aborted, p.wait_polls))
                return left_behind(i, -1);
            const bool mend = kv == 1 && (at < w.lo || at + kTilePos > w.hi);
            uint64_t *bar = mend ? &b.landed : &b.full[ring_slot];
            if (lane == 0)
                tc::mbar_expect_tx(bar, Sh::kTileBytes);
            __syncwarp();
            if (lane < parts)
#pragma unroll
                for (int c = 0; c < kColumns; c++)
                    tc::tma_load_4d(tc::smem_u32(tile) + c * Sh::kBlock + lane * maps.rows * 128,
                                    kv ? &maps.v : &maps.k, c * 64, slot, w.head, page, bar);
            if (i == 0 && maps.q_rows) {
                tc::cp_async_wait_all();
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&b.q_full);
            }
            if (mend) {
                if (!warp_wait(&b.landed, patched & 1, &b.aborted, p.wait_polls))
                    return left_behind(i, patched & 1);
                patched++;
                for (int r = 0; r < kTilePos; r++)
                    if (at + r < w.lo || at + r >= w.hi)
                        for (int c = lane; c < Sh::kChunks; c += 32)
                            *reinterpret_cast<uint4 *>(tile + (c >> 3) * Sh::kBlock + r * 128 + ((c & 7) << 4)) =
                                make_uint4(0, 0, 0, 0);
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&b.full[ring_slot]);
            }
        }
    }
    left_behind(2 * tiles, -1);
}

// After a wait was given up: waits for the copies that may still be in flight,
// the queries' and those of the last tiles.  (A mended tile's have landed, and
// its barrier has been arrived at, but for the one that was waited for.)
template <int kSlots>
__device__ __noinline__ void tile_drain(TileBars &b, bool q_rows)
{
    if (!q_rows)
        tc::mbar_drain(&b.q_full, 0);
    for (int i = max(b.copied - kSlots, 0); i < b.copied; i++)
        tc::mbar_drain(&b.full[i % kSlots], (i / kSlots) & 1);
    if (b.landing >= 0)
        tc::mbar_drain(&b.landed, b.landing);
}

// The copy warps, row by row.
template <typename T, int DP, bool kTwo>
__device__ void tile_copy_rows(const AttnParams &p, const AttnWork &w, uint8_t *sq, uint8_t *ring, TileBars &b,
                               int tiles)
{
    using Sh = TileShape<DP, kTwo>;
    const int tid = threadIdx.x - Sh::kSoftmaxThreads, row0 = tid & ~31, start = w.lo & ~127;
    copy_queries<Sh, 64>(p, w, sq);
    const int32_t *pages = p.batch.table + w.s * p.batch.table_stride;
    auto place = [&](int j, int half) -> int64_t {
        const int at = start + j * kTilePos + half * 64 + tid;
        if (j >= tiles || at >= w.hi || at < w.lo)
            return -1;
        const int64_t o = slot_offset<T>(p.cache, pages, at, w.head);
        if (o < 0)
            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
        return o;
    };
    int64_t next0 = place(0, 0), next1 = place(0, 1);
    int done = 0;  // tiles handed over
    for (int j = 0; j < tiles; j++) {
        const int64_t mine0 = next0, mine1 = next1;
        next0 = place(j + 1, 0);
        next1 = place(j + 1, 1);
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            const int i = 2 * j + kv, slot = i % Sh::kSlots;
            if (i >= Sh::kSlots && !tc::mbar_wait(&b.empty[slot], (i / Sh::kSlots - 1) & 1, &b.aborted, p.wait_polls))
                return tc::cp_async_wait_all();
            copy_rows<Sh>(ring + slot * Sh::kTileBytes, kv ? p.cache.v : p.cache.k, mine0, row0, p.d);
            copy_rows<Sh>(ring + slot * Sh::kTileBytes, kv ? p.cache.v : p.cache.k, mine1, 64 + row0, p.d);
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (i == 1) {  // the queries and the first keys are wanted at once
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                tc::fence_async_smem();
                tc::mbar_arrive(&b.q_full);
                tc::mbar_arrive(&b.full[0]);
                done = 1;
            } else if (i - kTileLag >= done) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kTileLag) : "memory");
                tc::fence_async_smem();
                tc::mbar_arrive(&b.full[done++ % Sh::kSlots]);
            }
        }
    }
    tc::cp_async_wait_all();
    tc::fence_async_smem();
    while (done < 2 * tiles)
        tc::mbar_arrive(&b.full[done++ % Sh::kSlots]);
}

// kPowers: keys and values are those of a cache in 8 bits, the values (in fp16 the keys too) relative to powers of their
// page of 128 positions, which is a tile.  The keys' power is part of the tile's scale.  The output is relative to the
// largest of the values' powers so far; where a tile's is 2^-x of it, its weights are lifted by so much less (x up to 60: no
// sum loses anything).  Weights are fp16 then, whatever T.  (A tile's powers are asked for a tile ahead, at a place that
// takes one register: with a pointer, and bf16 keys relative too, 392 us instead of 378 for 4 sequences of 2048 new on
// 8192, cold, 16 heads on 4 of 128 bf16 elements.)
template <typename T, bool kPowers>
using TileWeight = typename std::conditional<kPowers, __half, T>::type;

template <typename T, int DP, bool kTwo, bool kPowers>
__device__ void tile_softmax(const AttnParams &p, const AttnWork &w, uint8_t *sq, TileBars &b, int tiles)
{
    using Sh = TileShape<DP, kTwo>;
    using W = TileWeight<T, kPowers>;
    constexpr int kHalf = kTilePos / 2, kCols = DP / 2;  // scores, output columns of a thread
    const int warp = threadIdx.x >> 5, t = warp >> 3, half = (warp >> 2) & 1;
    const int in = (warp & 3) * 32 + (threadIdx.x & 31), r = t * 128 + in, pair = 1 + t * 4 + (warp & 3);
    const uint32_t lanes = b.tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lanes + t * 128 + half * kHalf, p_at = lanes + t * 128 + half * (kHalf / 2);
    const uint32_t o_at = lanes + Sh::kScoreCols + t * DP + half * kCols;
    const int row = w.row0 + r, token = row / p.group;
    const bool mine = r < w.rows;
    // a row past the last sees everything: it needs no mask, and nothing of it is written
    const int hi = mine ? min(seen_hi(w.seq, p.causal, token), w.hi) : 0x7fffffff;
    const int lo = mine ? max(seen_lo(seen_hi(w.seq, p.causal, token), p.window), w.lo) : 0;
    float m = -INFINITY, l = 0.f;
    int ref_at = 0, next_ref = 0;  // of the next tile
    if constexpr (kPowers) {
        ref_at = (int)((w.s * p.batch.table_stride + (w.lo >> 7)) * p.cache.heads) + w.head;
        next_ref = tiles > 0 ? __ldg(p.refs + ref_at) : 0;
    }
    const ScoreScale scale_of(p.scale_log2, -kCodeLift - 127);
    int v_ref = 0;  // the exponent that the output is relative to
    for (int j = 0; j < tiles; j++) {
        float scale_log2 = p.scale_log2;
        int fall = 0, now_ref = 0;  // how far the tile's values' power lies below the output's
        if constexpr (kPowers) {
            const int ref = next_ref;
            ref_at += p.cache.heads;
            next_ref = j + 1 < tiles ? __ldg(p.refs + ref_at) : 0;
            if constexpr (std::is_same<T, __half>::value)
                scale_log2 = scale_of.times(ref & 255);
            now_ref = max(v_ref, ref >> 8);
            fall = min(now_ref - (ref >> 8), 60);
        }
        // a wait that runs out is seen at the end; the pair's barriers below want every warp
        tc::mbar_wait(&b.s_full[t], j & 1, &b.aborted, p.wait_polls);
        __syncwarp();
        tc::fence_after_sync();
        uint32_t s[kHalf];
        const int at = (w.lo & ~127) + j * kTilePos + half * kHalf;
        tc::tmem_ld32_async(s_at, s);
        tc::tmem_ld32_async(s_at + 32, s + 32);
        tc::tmem_ld_wait(s);
        tc::tmem_ld_wait(s + 32);
        if (!__all_sync(0xffffffffu, at >= lo && at + kHalf <= hi)) {
#pragma unroll
            for (int i = 0; i < kHalf; i++)
                s[i] = at + i >= lo && at + i < hi ? s[i] : 0xff800000u;
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kHalf; i += 2)
            top[i / 2 & 3] = fmaxf(top[i / 2 & 3], fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
        float now = __fmul_ru(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), scale_log2);
        b.agree[t][half][in] = now;
        tc::named_sync(pair, 64);
        now = fmaxf(now, b.agree[t][1 - half][in]);
        if (__any_sync(0xffffffffu, now - m > kTileSlack<W> || (kPowers && now_ref > v_ref))) {
            // also from -infinity; the output of the tiles before is complete: the scores' MMA came after it
            // (over codes a row goes by its own growth alone, so that its bits do not depend on the other rows')
            const float next = !kPowers || now - m > kTileSlack<W> ? fmaxf(m, now) : m;
            float f = next == -INFINITY ? 1.f : exp2_approx(m - next);
            m = next;
            l *= f;
            if constexpr (kPowers) {
                f *= __uint_as_float((uint32_t)max(127 + v_ref - now_ref, 0) << 23);
                v_ref = now_ref;
            }
            if (j > 0) {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t o[16];
                    tc::tmem_ld16(o_at + c, o);
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tc::tmem_st16(o_at + c, o);
                }
            }
        }
        const float lift = __fsub_rd(kTileLift<W> - (float)fall, m == -INFINITY ? 0.f : m);
        const float2 scale = make_float2(scale_log2, scale_log2), off = make_float2(lift, lift);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kHalf / 32; c++) {
            uint32_t packed[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int k = c * 32 + 2 * i;
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale, off);
                const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                packed[i] = pack2<W>(e.x, e.y);
            }
            tc::tmem_st16(p_at + c * 16, packed);
        }
        const float sums = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        l += kPowers ? sums * __uint_as_float((uint32_t)(127 + fall) << 23) : sums;
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            tc::mbar_arrive(&b.p_ready[t]);
    }
    tc::named_sync(pair, 64);  // the last maxima have been read
    b.agree[t][half][in] = l;
    tc::named_sync(pair, 64);
    l = b.agree[t][0][in] + b.agree[t][1][in];
    float inv = 0.f, lse = -INFINITY;
    if (l != 0.f) {  // not a number either: then neither is the row
        inv = 1.f / l;
        if constexpr (kPowers)
            inv *= exp_power((uint32_t)v_ref) * (1.f / (1 << kCodeLift));
        lse = m + (log2f(l) - kTileLift<W>);
    }
    if (tiles > 0) {
        tc::mbar_wait(&b.o_full[t], 0, &b.aborted, p.wait_polls);
        __syncwarp();
        tc::fence_after_sync();
    }
    tile_write<T, DP, kTwo>(p, w, sq, b.tmem, t, half, tiles, inv, lse);
}

template <typename T, int DP, bool kBulk, bool kTwo, bool kPowers>
__global__ void __launch_bounds__(TileShape<DP, kTwo>::threads(kBulk), kTwo ? 1 : 2)
kv_attn_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ TileMaps maps)
{
    using Sh = TileShape<DP, kTwo>;
    constexpr int kLast = Sh::threads(kBulk) / 32 - 1;
    extern __shared__ __align__(1024) uint8_t sq[];  // query tiles, the ring, then the rest: all that an SM has
    uint8_t *ring = sq + Sh::kRows / 128 * Sh::kTileBytes;
    TileBars &b = *reinterpret_cast<TileBars *>(sq + Sh::kTiles);
    const int warp = threadIdx.x >> 5;
    if (kBulk && threadIdx.x == Sh::kSoftmaxThreads) {  // on their way while the CTA finds its work
        if (!maps.q_rows)
            tc::prefetch_map(&maps.q);
        tc::prefetch_map(&maps.k);
        tc::prefetch_map(&maps.v);
    }
    AttnWork w;
    if (!tile_work(p, reinterpret_cast<int *>(sq), w))
        return;
    const int tiles = w.hi > w.lo ? (w.hi - (w.lo & ~127) + kTilePos - 1) / kTilePos : 0;  // 0: rows that see nothing
    const bool two = kTwo && w.rows > 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kSlots; i++) {
            tc::mbar_init(&b.full[i], kBulk ? 1 : copy_threads(false));
            tc::mbar_init(&b.empty[i], 1);
        }
        tc::mbar_init(&b.q_full, kBulk ? 1 : copy_threads(false));
        tc::mbar_init(&b.drained, 1);
        tc::mbar_init(&b.landed, 1);
        for (int t = 0; t < 2; t++) {
            tc::mbar_init(&b.s_full[t], 1);
            tc::mbar_init(&b.p_ready[t], 8);  // the tile's warps
            tc::mbar_init(&b.o_full[t], 1);
        }
        b.aborted = b.copied = 0;
        b.landing = -1;
        tc::mbar_init_fence();
    }
    if (warp == kLast)
        tc::tmem_alloc<Sh::kTmem>(&b.tmem);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp < Sh::kSoftmaxWarps) {
        if (warp < 8 || two)
            tile_softmax<T, DP, kTwo, kPowers>(p, w, sq, b, tiles);
    } else if (warp < kLast) {
        if (tiles > 0) {
            if constexpr (kBulk) {
                tile_copy_bulk<T, DP, kTwo>(p, w, maps, sq, ring, b, tiles);
            } else {
                tile_copy_rows<T, DP, kTwo>(p, w, sq, ring, b, tiles);
            }
        }
    } else if (tiles > 0) {
        tile_mma<T, TileWeight<T, kPowers>, DP, kTwo>(sq, ring, b, tiles, two, p.wait_polls);
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // Nobody waits any more, so all see the same.  No copy and no MMA may be in flight when the memory is given back.
    if (*reinterpret_cast<volatile int *>(&b.aborted)) {
        if (threadIdx.x == 0)
            raise_flag(p.err, DLRM_FLAG_WAIT_TIMEOUT);
        if (kBulk && warp == Sh::kSoftmaxWarps && tiles > 0)
            tile_drain<Sh::kSlots>(b, maps.q_rows);
        if (warp == kLast && tiles > 0 && tc::elect_one()) {
            tc::mma_commit(&b.drained);
            tc::mbar_drain(&b.drained, 0);
        }
        __syncthreads();
    }
    if (warp == kLast)
        tc::tmem_free<Sh::kTmem>(b.tmem);
}

// Maps of the cache; false where it cannot be described so.
static bool tile_maps(const AttnParams &p, int dtype, TileMaps &m)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc || p.cache.page.d % 8 != 0)
        return false;
    m.rows = 8;
    while (m.rows < kTilePos && p.cache.page.d % (2 * m.rows) == 0)
        m.rows *= 2;
    const CUtensorMapDataType type = dtype == DLRM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    auto encode = [&](CUtensorMap *map, int rank, void *base, const cuuint64_t *dims, const cuuint64_t *strides,
                      const cuuint32_t *box) {
        const cuuint32_t one[4] = {1, 1, 1, 1};
        return enc(map, type, rank, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, p.cache.page.d, (cuuint64_t)p.cache.heads, p.cache.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.cache.slot_stride * 2, (cuuint64_t)p.cache.head_stride * 2,
                                   (cuuint64_t)p.cache.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)m.rows, 1, 1};
    if (!encode(&m.k, 4, p.cache.k, dims, strides, box) || !encode(&m.v, 4, p.cache.v, dims, strides, box))
        return false;
    const cuuint64_t q_dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.q.heads, (cuuint64_t)p.batch.n};
    const cuuint64_t q_strides[2] = {(cuuint64_t)p.q.hs * 2, (cuuint64_t)p.q.ts * 2};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(128 / (p.group <= 128 ? p.group : 128))};
    m.q_rows = p.group > 128 || 128 % p.group != 0 || !encode(&m.q, 3, p.q.ptr, q_dims, q_strides, q_box);
    return true;
}

template <typename T, int DP, bool kBulk, bool kTwo, bool kPowers = false>
static int launch_tile(const AttnParams &p, const TileMaps &maps, int64_t ctas, cudaStream_t st)
{
    using Sh = TileShape<DP, kTwo>;
    constexpr int smem = Sh::kTiles + sizeof(TileBars);
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv_attn_tile_kernel<T, DP, kBulk, kTwo, kPowers>, smem, &done);
    if (s != DLRM_OK)
        return s;
    kv_attn_tile_kernel<T, DP, kBulk, kTwo, kPowers><<<(unsigned)ctas, Sh::threads(kBulk), smem, st>>>(p, maps);
    count_launch(st);
    return DLRM_OK;
}

template <typename T, bool kBulk>
static int launch_tile_shape(const AttnParams &p, const TileMaps &maps, int64_t ctas, cudaStream_t st)
{
    if (p.d > 64)
        return launch_tile<T, 128, kBulk, true>(p, maps, ctas, st);
    return p.rows > 128 ? launch_tile<T, 64, kBulk, true>(p, maps, ctas, st)
                        : launch_tile<T, 64, kBulk, false>(p, maps, ctas, st);
}

template <typename T>
static int launch_tile_type(const AttnParams &p, int dtype, int64_t ctas, cudaStream_t st)
{
    TileMaps maps = {};
    const bool bulk = tile_maps(p, dtype, maps);
    if (p.refs) {  // pages of 128, and more than 256 rows
        if (!bulk || p.rows != 256)
            return DLRM_ERR_UNSUPPORTED;
        return p.d > 64 ? launch_tile<T, 128, true, true, true>(p, maps, ctas, st)
                        : launch_tile<T, 64, true, true, true>(p, maps, ctas, st);
    }
    return bulk ? launch_tile_shape<T, true>(p, maps, ctas, st) : launch_tile_shape<T, false>(p, maps, ctas, st);
}

int launch_kv_attn_tile(const AttnParams &p, int dtype, int64_t ctas, cudaStream_t st)
{
    return dtype == DLRM_F16 ? launch_tile_type<__half>(p, dtype, ctas, st)
                             : launch_tile_type<__nv_bfloat16>(p, dtype, ctas, st);
}

}  // namespace dlrm
