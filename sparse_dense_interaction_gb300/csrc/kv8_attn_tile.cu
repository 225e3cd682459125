// Attention over the cache in 8 bits for many rows: tiles of 256 (or 128) rows on
// the tensor cores, in fp16 whatever the queries' 16-bit type.
//
// The tiles, their MMAs and their softmax are those of the 16-bit cache
// (tensor memory, one warp that issues, a lagging maximum).  What 8 bits change:
//  - Keys and values are converted on their way into the ring of tiles: warps of their own
//    copy 16 codes a lane from the pages, asynchronously and two tiles ahead, and
//    write them as fp16 into the swizzled tiles that the MMAs read; they take groups of rows in
//    turn.  A lane converts the chunks that it copied, so a warp waits for its own
//    copies alone, and pages of any size take this path.
//  - Every code is multiplied by its block's power relative to a power of the tile
//    (2^7 lifts it to fp16's range; the product is exact but for what lies 2^-41 below the
//    largest): for keys the tile's largest, which then is part of the tile's
//    scale, for values the largest so far, and the output is scaled down when it grows, as it
//    is when a maximum does.  So the softmax does nothing more for an element.
//  - The softmax's threads fetch the queries, which are idle until then: bf16 rows
//    are lifted by a power of two each, so that they fit fp16 exactly but for
//    what lies 2^-38 below a row's largest.
//  - Weights are rounded to fp16 once: 2^-11 of each, as much as an fp16 output's own rounding and an eighth of a bf16
//    one's (candidates, fp16: error against 64 bits 2.5 to 2.8e-4, the plain form's 2.1e-4).  A second part would be a second
//    MMA for each tile of values.
//  - The softmax reads half of a thread's scores at a time, twice: that leaves it 80 registers,
//    and 7 warps (3 where two CTAs share an SM) to convert.  (Nothing spills but bf16 heads above 128, 176 bytes.)
//
// What bounds it: the converting warps' own path (copies, conversion, hand-over).  49 users' 56 rows
// on up to 51630 (8 heads on 4 of 80) take 685 us, without the softmax 652, without converting 522, without both and
// the copies 300.  16 sequences of 256 new on up to 8192 (16 heads on 4, 128 bf16
// elements): 142 us; 64 users' 200
// candidates on up to 2000, 8 heads of 64: 68 us (16-bit cache: 55); 4 times 2048 on 4096, 8 heads
// on 2 of 256: 282 us.  Longer chunks of narrower heads convert once instead (4 of 2048 on 8192,
// 16 heads on 4 of 128, would take 461 us here in fp16, 470 in bf16).
// Slower: 15 such warps for one query tile (714 us for the 56 rows); 4 or 8 warps that load a
// tile ahead into registers (764, 613 us for those 4 of 2048, then 476); registers dealt out anew by
// role (650); bulk copies by a warp of their own (468, and 75 against 73 for the candidates,
// so neither better); two query tiles a CTA for heads of 64.
#include "kv8.cuh"
#include "kv_tile.cuh"

namespace dlrm {

template <int DP, bool kTwo>
struct Tile8Shape : TileShape<DP, kTwo, (DP == 256 ? 2 : DP == 128 || !kTwo ? 4 : 8)> {
    using Sh = TileShape<DP, kTwo, (DP == 256 ? 2 : DP == 128 || !kTwo ? 4 : 8)>;
    static constexpr int kResident = kTwo || DP == 256 ? 1 : 2;  // CTAs of an SM
    // that convert: as many as leave the others 80 registers a thread
    static constexpr int kWarps = kResident == 1 ? 7 : 3;
    static constexpr int kMmaWarp = Sh::kSoftmaxWarps + kWarps, kThreads = kMmaWarp * 32 + 32;
    static constexpr int kStepRows = 32 / (DP / 16);     // rows of which a warp's lanes take a chunk at once
    static constexpr int kGroups = kTilePos / kStepRows;  // of rows, which the warps take in turn
    static constexpr int kSteps = (kGroups + kWarps - 1) / kWarps;
    static constexpr int kOwn = (kSteps * kStepRows + 31) / 32;  // rows whose places a lane finds
    // Codes on their way: a tile of keys and one of values; with heads of 256, which leave room for one, a step's place is
    // filled again as soon as it has been read, and L2 is told of the rows a tile ahead.
    static constexpr int kRawTiles = DP == 256 ? 1 : 2, kRawBytes = kTilePos * DP;
    static constexpr int kBars = Sh::kTiles + kRawTiles * kRawBytes;
};

constexpr int kTile8Refs = 8;   // tiles whose powers are kept: more than the ring holds
constexpr int kConvertBarrier = 9;

struct Tile8Bars : TileBars {
    int k_ref[kTile8Refs], v_ref[kTile8Refs];  // of a tile: the exponents that its codes are relative to
    int warp_ref[2][8][2];
};

// The warps that convert.  A tile begins at a multiple of 128 positions.  A lane reads back the chunks of codes
// that it copied itself, so a warp waits for nobody's copies but its own.
template <int DP, bool kTwo>
__device__ void tile8_convert(const AttnParams &p, const AttnWork &w, uint8_t *ring, uint8_t *raw, Tile8Bars &b, int tiles)
{
    using Sh = Tile8Shape<DP, kTwo>;
    constexpr int kOwn = Sh::kOwn, kSteps = Sh::kSteps, kStepRows = Sh::kStepRows;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - Sh::kSoftmaxWarps;
    const int start = w.lo & ~127;
    const int32_t *pages = p.batch.table + w.s * p.batch.table_stride;
    // the lane's row and chunk of a step: 8 lanes write to every bank once
    const int step_row = DP == 256 ? (lane >> 2) & 1 : DP == 128 ? ((lane >> 2) & 1) | (lane >> 4) << 1 : lane >> 2;
    const int chunk = DP == 256 ? (lane & 3) | (lane >> 3) << 2 : DP == 128 ? (lane & 3) | ((lane >> 3) & 1) << 2 : lane & 3;
    const bool inside = chunk * 16 < p.d;
    uint8_t *mine = raw + lane * 16;
    // the rows of the warp's step i, and of its own row n: those of a group
    auto group = [&](int i) { return warp + i * Sh::kWarps; };
    auto row_of = [&](int n) { return group(n / kStepRows) * kStepRows + n % kStepRows; };

    int32_t page[kOwn], slot[kOwn];  // of a coming tile's rows lane, lane + 32; slot -1: nothing of it is seen
    int64_t off[kOwn], off_now[kOwn];  // codes of the next tile's rows, of this one's; -1: a row of zeros
    uint32_t k_next[kOwn], v_next[kOwn];  // their exponents
    auto find = [&](int j) {
#pragma unroll
        for (int i = 0; i < kOwn; i++) {
            const int row = row_of(i * 32 + lane), at = start + j * kTilePos + row;
            slot[i] = -1;
            if (j < tiles && row < kTilePos && at >= w.lo && at < w.hi) {
                const uint32_t n = p.cache.page.div((uint32_t)at);
                slot[i] = at - (int)(n * p.cache.page.d);
                page[i] = __ldg(pages + n);
            }
        }
    };
    auto place = [&]() {
#pragma unroll
        for (int i = 0; i < kOwn; i++) {
            off[i] = -1;
            k_next[i] = v_next[i] = 0;
            if (slot[i] < 0)
                continue;
            if ((uint32_t)page[i] >= p.cache.pages) {
                raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
                continue;
            }
            off[i] = page[i] * p.cache.page_stride + slot[i] * p.cache.slot_stride + w.head * p.cache.head_stride;
            const int64_t x = exp_offset(p.exp, page[i], slot[i], w.head);
            k_next[i] = p.exp.k[x];
            v_next[i] = p.exp.v[x];
            if (Sh::kRawTiles == 1) {
                for (int c = 0; c < p.d; c += 128) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.cache.k + off[i] + c));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.cache.v + off[i] + c));
                }
            }
        }
    };
    // step i of a tile of keys or values from the rows `from`
    auto copy_step = [&](const char *base, const int64_t *from, uint8_t *to, int i) {
        const int64_t o = __shfl_sync(0xffffffffu, from[i * kStepRows / 32], (i * kStepRows + step_row) & 31);
        const bool there = o >= 0 && inside;
        if (group(i) < Sh::kGroups)
            tc::cp_async16(to + group(i) * 512, base + (there ? o + chunk * 16 : 0), there);
    };
    auto copy = [&](const char *base, int kv) {
#pragma unroll
        for (int i = 0; i < kSteps; i++)
            copy_step(base, off, mine + kv * Sh::kRawBytes, i);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // `base`, `from`: of the next tile, step by step, where it has no place of its own
    auto convert = [&](uint8_t *tile, const uint32_t *factor, int kv, const char *base, const int64_t *from) {
        uint8_t *codes = mine + (Sh::kRawTiles == 1 ? 0 : kv * Sh::kRawBytes);
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
            if (group(i) >= Sh::kGroups)
                break;
            const uint32_t f = __shfl_sync(0xffffffffu, factor[i * kStepRows / 32], (i * kStepRows + step_row) & 31);
            const uint4 c = *reinterpret_cast<const uint4 *>(codes + group(i) * 512);
            const uint32_t in[4] = {c.x, c.y, c.z, c.w};
            uint32_t x[8];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                decode4(in[k], x[2 * k], x[2 * k + 1]);
                x[2 * k] = hmul2(x[2 * k], f);
                x[2 * k + 1] = hmul2(x[2 * k + 1], f);
            }
            const int r = group(i) * kStepRows + step_row, unit = 2 * (chunk & 3);
            uint8_t *to = tile + (chunk >> 2) * Sh::kBlock + r * 128;
            *reinterpret_cast<uint4 *>(to + ((unit ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4 *>(to + (((unit + 1) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
            if constexpr (Sh::kRawTiles == 1)
                copy_step(base, from, mine, i);
        }
    };
    // after a wait that ran out the warps still meet at their barrier, but hand nothing over
    bool dead = false;
    auto hand_over = [&](int i, const uint32_t *factor, const char *base, const int64_t *from) {
        if (!dead && i >= Sh::kSlots &&
            !warp_wait(&b.empty[i % Sh::kSlots], (i / Sh::kSlots - 1) & 1, &b.aborted, p.wait_polls))
            dead = true;
        asm volatile("cp.async.wait_group %0;" ::"n"(Sh::kRawTiles - 1) : "memory");
        if (!dead) {
            convert(ring + i % Sh::kSlots * Sh::kTileBytes, factor, i & 1, base, from);
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(&b.full[i % Sh::kSlots]);
        }
        if constexpr (Sh::kRawTiles == 1)
            asm volatile("cp.async.commit_group;" ::: "memory");
    };

    find(0);
    place();
    copy(p.cache.k, 0);
    if constexpr (Sh::kRawTiles == 2)
        copy(p.cache.v, 1);
    find(1);
    int v_ref = 0;
#pragma unroll 1
    for (int j = 0; j < tiles; j++) {
        // what the tile's codes are relative to
        uint32_t kf[kOwn], vf[kOwn], k_top = 0, v_top = 0;
#pragma unroll
        for (int i = 0; i < kOwn; i++) {
            kf[i] = k_next[i];
            vf[i] = v_next[i];
            k_top = max(k_top, kf[i]);
            v_top = max(v_top, vf[i]);
        }
        k_top = __reduce_max_sync(0xffffffffu, k_top);
        v_top = __reduce_max_sync(0xffffffffu, v_top);
        if (lane == 0) {
            b.warp_ref[j & 1][warp][0] = (int)k_top;
            b.warp_ref[j & 1][warp][1] = (int)v_top;
        }
        tc::named_sync(kConvertBarrier, Sh::kWarps * 32);
        int k_ref = 0;
#pragma unroll
        for (int i = 0; i < Sh::kWarps; i++) {
            k_ref = max(k_ref, b.warp_ref[j & 1][i][0]);
            v_ref = max(v_ref, b.warp_ref[j & 1][i][1]);
        }
        if (warp == 0 && lane == 0) {
            b.k_ref[j % kTile8Refs] = k_ref;
            b.v_ref[j % kTile8Refs] = v_ref;
        }
#pragma unroll
        for (int i = 0; i < kOwn; i++) {
            kf[i] = relative_power((int)kf[i] - k_ref);
            vf[i] = relative_power((int)vf[i] - v_ref);
        }
#pragma unroll
        for (int i = 0; i < kOwn; i++)
            off_now[i] = off[i];
        place();
        find(j + 2);
        hand_over(2 * j, kf, p.cache.v, off_now);
        if constexpr (Sh::kRawTiles == 2)
            copy(p.cache.k, 0);
        hand_over(2 * j + 1, vf, p.cache.k, off);
        if constexpr (Sh::kRawTiles == 2)
            copy(p.cache.v, 1);
    }
    tc::cp_async_wait_all();
}

// A softmax thread's half of its query row, as fp16 in the swizzled tile; 2 to the power of what it returns undoes the
// row's lifting.
template <typename T, int DP, bool kTwo>
__device__ __forceinline__ int tile8_query(const AttnParams &p, const AttnWork &w, uint8_t *sq, Tile8Bars &b, int t,
                                             int half, int in, int pair)
{
    using Sh = Tile8Shape<DP, kTwo>;
    constexpr int kChunks = DP / 16;  // of 8 elements, of half a row
    const int r = t * 128 + in, row = w.row0 + r, token = row / p.group;
    const bool mine = r < w.rows;
    const T *src = p.q.row<T>(mine ? w.seq.first + token : 0, mine ? w.head * p.group + row - token * p.group : 0);
    uint4 x[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
        const int e = half * (DP / 2) + c * 8;
        x[c] = mine && e < p.d ? *reinterpret_cast<const uint4 *>(src + e) : make_uint4(0, 0, 0, 0);
    }
    int back = 0;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
            const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 y = unpack2<T>(v[i]);
                top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
        }
        b.agree[t][half][in] = top;
        tc::named_sync(pair, 64);
        top = fmaxf(top, b.agree[t][1 - half][in]);
        float lift = 1.f;
        const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
        if (top > 0.f && e < 255) {
            lift = __uint_as_float((268 - e) << 23);  // 2^(127 + 14 - e)
            back = (int)e - (127 + 14);
        }
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
            uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 y = unpack2<T>(v[i]);
                v[i] = pack2<__half>(y.x * lift, y.y * lift);
            }
            x[c] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
        const int e = half * (DP / 2) + c * 8;
        *reinterpret_cast<uint4 *>(sq + t * Sh::kTileBytes + (e >> 6) * Sh::kBlock + in * 128 +
                                   ((((e >> 3) & 7) ^ (in & 7)) << 4)) = x[c];
    }
    tc::fence_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        tc::mbar_arrive(&b.q_full);
    return back;
}

template <typename T, int DP, bool kTwo>
__device__ void tile8_softmax(const AttnParams &p, const AttnWork &w, uint8_t *sq, Tile8Bars &b, int tiles)
{
    using Sh = Tile8Shape<DP, kTwo>;
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
    // Rows that see nothing want no query: the warps' outputs go through the queries' tiles, and no MMA comes between
    const int back = tiles > 0 ? tile8_query<T, DP, kTwo>(p, w, sq, b, t, half, in, pair) : 0;
    const ScoreScale scale_of(p.scale_log2, back - kCodeLift - 127);
    float m = -INFINITY, l = 0.f;
    int v_ref = 0;  // the exponent that the output is relative to
    for (int j = 0; j < tiles; j++) {
        // a wait that runs out is seen at the end; the pair's barriers below want every warp
        tc::mbar_wait(&b.s_full[t], j & 1, &b.aborted, p.wait_polls);
        __syncwarp();
        tc::fence_after_sync();
        // half of the thread's scores at a time, read twice: all of them and the rest want 96 registers, a fifth more
        uint32_t s[32];
        const int at = (w.lo & ~127) + j * kTilePos + half * kHalf;
        const bool whole = __all_sync(0xffffffffu, at >= lo && at + kHalf <= hi);
        auto scores = [&](int c) {
            tc::tmem_ld32_async(s_at + c, s);
            tc::tmem_ld_wait(s);
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 32; i++)
                    s[i] = at + c + i >= lo && at + c + i < hi ? s[i] : 0xff800000u;
            }
        };
        const int k_ref = b.k_ref[j % kTile8Refs], now_ref = b.v_ref[j % kTile8Refs];
        const float scale_log2 = scale_of.times(k_ref);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
            scores(kHalf - 32 - c);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
                top[i / 2 & 3] = fmaxf(top[i / 2 & 3], fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
        }
        float now = __fmul_ru(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), scale_log2);
        b.agree[t][half][in] = now;
        tc::named_sync(pair, 64);
        now = fmaxf(now, b.agree[t][1 - half][in]);
        if (__any_sync(0xffffffffu, now - m > kTileSlack<__half> || now_ref > v_ref)) {
            // also from -infinity; the output of the tiles before is complete: the scores' MMA came after it
            // (a row's own growth alone, so that its bits do not depend on the other rows')
            const float next = now - m > kTileSlack<__half> ? now : m, f = next == -INFINITY ? 1.f : exp2_approx(m - next);
            const float down = f * __uint_as_float((uint32_t)max(127 + v_ref - now_ref, 0) << 23);
            m = next;
            l *= f;
            v_ref = now_ref;
            if (j > 0) {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t o[16];
                    tc::tmem_ld16(o_at + c, o);
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * down);
                    tc::tmem_st16(o_at + c, o);
                }
            }
        }
        const float lift = __fsub_rd(kTileLift<__half>, m == -INFINITY ? 0.f : m);
        const float2 scale = make_float2(scale_log2, scale_log2), off = make_float2(lift, lift);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t packed[32];
#pragma unroll
        for (int c = 0; c < kHalf / 32; c++) {
            if (c > 0)
                scores(c * 32);
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int k = 2 * i;
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale, off);
                const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                packed[c * 16 + i] = pack2<__half>(e.x, e.y);
            }
        }
        tc::named_sync(pair, 64);
        tc::tmem_st16(p_at, packed);
        tc::tmem_st16(p_at + 16, packed + 16);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
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
        inv = 1.f / l * exp_power((uint32_t)v_ref) * (1.f / (1 << kCodeLift));
        lse = m + (log2f(l) - kTileLift<__half>);
    }
    if (tiles > 0) {
        tc::mbar_wait(&b.o_full[t], 0, &b.aborted, p.wait_polls);
        __syncwarp();
        tc::fence_after_sync();
    }
    tile_write<T, DP, kTwo>(p, w, sq, b.tmem, t, half, tiles, inv, lse);
}

template <typename T, int DP, bool kTwo>
__global__ void __launch_bounds__(Tile8Shape<DP, kTwo>::kThreads, Tile8Shape<DP, kTwo>::kResident)
kv8_attn_tile_kernel(const __grid_constant__ AttnParams p)
{
    using Sh = Tile8Shape<DP, kTwo>;
    constexpr int kLast = Sh::kMmaWarp;
    extern __shared__ __align__(1024) uint8_t sq[];  // query tiles, the ring, then the rest: all that an SM has
    uint8_t *ring = sq + Sh::kRows / 128 * Sh::kTileBytes;
    Tile8Bars &b = *reinterpret_cast<Tile8Bars *>(sq + Sh::kBars);
    const int warp = threadIdx.x >> 5;
    AttnWork w;
    if (!tile_work(p, reinterpret_cast<int *>(sq), w))
        return;
    const int tiles = w.hi > w.lo ? (w.hi - (w.lo & ~127) + kTilePos - 1) / kTilePos : 0;  // 0: rows that see nothing
    const bool two = kTwo && w.rows > 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kSlots; i++) {
            tc::mbar_init(&b.full[i], Sh::kWarps);
            tc::mbar_init(&b.empty[i], 1);
        }
        tc::mbar_init(&b.q_full, two ? 16 : 8);  // the softmax's warps
        tc::mbar_init(&b.drained, 1);
        for (int t = 0; t < 2; t++) {
            tc::mbar_init(&b.s_full[t], 1);
            tc::mbar_init(&b.p_ready[t], 8);  // the tile's warps
            tc::mbar_init(&b.o_full[t], 1);
        }
        b.aborted = 0;
        tc::mbar_init_fence();
    }
    if (warp == kLast)
        tc::tmem_alloc<Sh::kTmem>(&b.tmem);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp < Sh::kSoftmaxWarps) {
        if (warp < 8 || two)
            tile8_softmax<T, DP, kTwo>(p, w, sq, b, tiles);
    } else if (warp < kLast) {
        if (tiles > 0)
            tile8_convert<DP, kTwo>(p, w, ring, sq + Sh::kTiles, b, tiles);
    } else if (tiles > 0) {
        tile_mma<__half, __half, DP, kTwo, typename Sh::Sh>(sq, ring, b, tiles, two, p.wait_polls);
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // Nobody waits any more, so all see the same.  No MMA may be in flight when the memory is given back.
    if (*reinterpret_cast<volatile int *>(&b.aborted)) {
        if (threadIdx.x == 0)
            raise_flag(p.err, DLRM_FLAG_WAIT_TIMEOUT);
        if (warp == kLast && tiles > 0 && tc::elect_one()) {
            tc::mma_commit(&b.drained);
            tc::mbar_drain(&b.drained, 0);
        }
        __syncthreads();
    }
    if (warp == kLast)
        tc::tmem_free<Sh::kTmem>(b.tmem);
}

template <typename T, int DP, bool kTwo>
static int launch_tile8(const AttnParams &p, int64_t ctas, cudaStream_t st)
{
    constexpr int smem = Tile8Shape<DP, kTwo>::kBars + sizeof(Tile8Bars);
    static_assert(smem <= (Tile8Shape<DP, kTwo>::kResident == 1 ? 232448 : 115200), "an SM's shared memory");
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv8_attn_tile_kernel<T, DP, kTwo>, smem, &done);
    if (s != DLRM_OK)
        return s;
    kv8_attn_tile_kernel<T, DP, kTwo><<<(unsigned)ctas, Tile8Shape<DP, kTwo>::kThreads, smem, st>>>(p);
    count_launch(st);
    return DLRM_OK;
}

template <typename T>
static int launch_tile8_shape(const AttnParams &p, int64_t ctas, cudaStream_t st)
{
    if (p.d > 128)
        return launch_tile8<T, 256, false>(p, ctas, st);
    if (p.d > 64)
        return launch_tile8<T, 128, true>(p, ctas, st);
    return p.rows > 128 ? launch_tile8<T, 64, true>(p, ctas, st) : launch_tile8<T, 64, false>(p, ctas, st);
}

int launch_kv8_attn_tile(const AttnParams &p, int dtype, int64_t ctas, cudaStream_t st)
{
    return dtype == DLRM_F16 ? launch_tile8_shape<__half>(p, ctas, st) : launch_tile8_shape<__nv_bfloat16>(p, ctas, st);
}

}  // namespace dlrm
