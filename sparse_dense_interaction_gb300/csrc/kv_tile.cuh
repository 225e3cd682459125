// Shared by the kernels of attention by tiles of 256 (or 128) rows: the shared
// memory, the warp that issues the MMAs, the rows' output and the CTA's work.
#pragma once

#include <type_traits>

#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

constexpr int kTilePos = 128;
__host__ __device__ constexpr int copy_threads(bool bulk) { return bulk ? 32 : 64; }

// log2 of the growth of a maximum that is let pass, and of what is left of the
// range that weights may use (kWeightTop) to lift them by.
template <typename T>
constexpr float kTileSlack = 8.f;
template <>
constexpr float kTileSlack<__half> = 4.f;
template <typename T>
constexpr float kTileLift = kWeightTop<T> > 0.f ? kWeightTop<T> - kTileSlack<T> : 0.f;

// kTwo: two query tiles of a CTA that has the SM, else one, and two CTAs share the SM.
template <int DP, bool kTwo, int kRing = DP == 128 || !kTwo ? 5 : 8>
struct TileShape {
    static constexpr int kRows = kTwo ? 256 : 128;
    static constexpr int kSoftmaxThreads = 2 * kRows, kSoftmaxWarps = kSoftmaxThreads / 32;
    static constexpr int kScoreCols = kRows, kTmem = DP > 128 ? 512 : 2 * kRows;  // tensor-memory columns: scores, all
    __host__ __device__ static constexpr int threads(bool bulk) { return kSoftmaxThreads + copy_threads(bulk) + 32; }
    static constexpr int kTileBytes = kTilePos * DP * 2;  // of keys or values; a query tile too
    static constexpr int kSlots = kRing;
    static constexpr int kTiles = kRows / 128 * kTileBytes + kSlots * kTileBytes;
    static constexpr int kBlock = kTilePos * 128;         // bytes between 64-column blocks of a tile
    static constexpr int kChunks = DP / 8;                // 16-byte chunks of a row
};

// A wait by a whole warp, whose lanes go on or give up together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *aborted, int polls)
{
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, aborted, polls));
}

struct TileBars {
    uint64_t full[8], empty[8], landed, q_full, s_full[2], p_ready[2], o_full[2], drained;
    uint32_t tmem;
    int aborted;
    int copied, landing;  // what the copy warp left behind: tiles copied, parity of a wait for `landed` (-1: none)
    float agree[2][2][128];  // [query tile][half][row]: a maximum of half a row's scores; at the end its sum
};

// T: the type of queries and keys; W: of weights and values.
template <typename T, typename W, int DP, bool kTwo, typename Sh = TileShape<DP, kTwo>>
__device__ void tile_mma(uint8_t *sq, uint8_t *ring, TileBars &b, int tiles, bool two, int polls)
{
    constexpr int kType = std::is_same<T, __nv_bfloat16>::value ? 1 : 0, kTypeW = std::is_same<W, __nv_bfloat16>::value ? 1 : 0;
    constexpr uint32_t kScores = tc::f16_idesc(kType, 128, kTilePos, false), kOut = tc::f16_idesc(kTypeW, 128, DP, true);
    // all lanes run this; one issues.  Descriptors of a later place are the first plus its distance / 16.
    const uint32_t tmem = __shfl_sync(0xffffffffu, b.tmem, 0);
    tiles = __shfl_sync(0xffffffffu, tiles, 0);  // known to be the warp's: the loop's values are uniform
    two = __shfl_sync(0xffffffffu, two, 0);
    const uint64_t q_desc = tc::sw128_desc(tc::smem_u32(sq)), k_desc = tc::sw128_desc(tc::smem_u32(ring));
    const uint64_t v_desc = tc::sw128_mn_desc(tc::smem_u32(ring), Sh::kBlock);
    auto scores = [&](int t, int j) {
        const uint64_t q = q_desc + t * (Sh::kTileBytes >> 4), k = k_desc + (2 * j % Sh::kSlots) * (Sh::kTileBytes >> 4);
        if (tc::elect_one()) {
#pragma unroll
            for (int e = 0; e < DP / 16; e++) {
                const int at = ((e >> 2) * Sh::kBlock + (e & 3) * 32) >> 4;
                tc::mma_f16(tmem + t * 128, q + at, k + at, kScores, e > 0);
            }
            tc::mma_commit(&b.s_full[t]);
        }
        __syncwarp();
    };
    auto output = [&](int t, int j) {
        const uint64_t v = v_desc + ((2 * j + 1) % Sh::kSlots) * (Sh::kTileBytes >> 4);
        if (tc::elect_one()) {
#pragma unroll
            for (int e = 0; e < kTilePos / 16; e++)
                tc::mma_f16_ta(tmem + Sh::kScoreCols + t * DP, tmem + t * 128 + e * 8, v + e * (2048 >> 4), kOut,
                               j > 0 || e > 0);
        }
        __syncwarp();
    };
    auto commit = [&](uint64_t *bar) {
        if (tc::elect_one())
            tc::mma_commit(bar);
        __syncwarp();
    };
    auto ready = [&](int i) { return warp_wait(&b.full[i % Sh::kSlots], (i / Sh::kSlots) & 1, &b.aborted, polls); };
    if (!warp_wait(&b.q_full, 0, &b.aborted, polls) || !ready(0))
        return;
    tc::fence_after_sync();
    scores(0, 0);
    if (two)
        scores(1, 0);
    commit(&b.empty[0]);
    for (int j = 0; j < tiles; j++) {
        for (int t = 0; t < (two ? 2 : 1); t++) {
            if (t == 0 && !ready(2 * j + 1))
                return;
            if (!warp_wait(&b.p_ready[t], j & 1, &b.aborted, polls))
                return;
            tc::fence_after_sync();
            output(t, j);
            if (t == (two ? 1 : 0))
                commit(&b.empty[(2 * j + 1) % Sh::kSlots]);
            if (j + 1 < tiles) {
                if (t == 0 && !ready(2 * j + 2))
                    return;
                scores(t, j + 1);
                if (t == (two ? 1 : 0))
                    commit(&b.empty[(2 * j + 2) % Sh::kSlots]);
            } else {
                commit(&b.o_full[t]);
            }
        }
    }
}

// Writes a softmax thread's half row, whose output lies in tensor memory, times `inv`, and the row's log2 of its sum.
template <typename T, int DP, bool kTwo>
__device__ __forceinline__ void tile_write(const AttnParams &p, const AttnWork &w, uint8_t *sq, uint32_t tmem, int t,
                                           int half, int tiles, float inv, float lse)
{
    using Sh = TileShape<DP, kTwo>;
    constexpr int kCols = DP / 2;
    const int warp = threadIdx.x >> 5, r = t * 128 + (warp & 3) * 32 + (threadIdx.x & 31);
    const uint32_t o_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + Sh::kScoreCols + t * DP + half * kCols;
    const int row = w.row0 + r, token = row / p.group;
    const bool mine = r < w.rows;
    const int heads = p.cache.heads * p.group, h = w.head * p.group + row - token * p.group;
    const int64_t part = ((int64_t)w.split * p.batch.n + w.seq.first + token) * heads + h;
    if (mine && half == 0) {
        if (!w.whole)
            p.part_lse[part] = lse;
        else if (p.lse)
            p.lse[(w.seq.first + token) * heads + h] = lse * kLn2;
    }
    // Through the queries' tiles (their MMAs are done), so that a row's lines are
    // written whole: a warp's 32 half rows, chunks of a row turned by its number
    // against bank conflicts.  Partial rows are fp32 and take two passes.  (Written
    // from the registers, a thread a row: 93 us instead of 88 for up to 300 new
    // tokens of each of 64 sequences on up to 1000, 16 heads on 4 of 128.)
    constexpr int kRowBytes = kCols * 2, kRowChunks = kRowBytes / 16;
    uint8_t *room = sq + warp * 32 * kRowBytes;
    const int lane = threadIdx.x & 31;
    auto at = [&](int r, int c) {
        return reinterpret_cast<uint4 *>(room + r * kRowBytes + ((c ^ (kRowChunks == 8 ? r & 7 : r >> 1 & 3)) << 4));
    };
    char *to = nullptr;
    if (mine)
        to = w.whole ? reinterpret_cast<char *>(p.out.row<T>(w.seq.first + token, h))
                     : reinterpret_cast<char *>(p.part_o + part * p.d);
    auto write = [&](auto whole) {
        constexpr int es = decltype(whole)::value ? 2 : 4, cols = kRowBytes / es;
#pragma unroll 1
        for (int c0 = 0; c0 < kCols; c0 += cols) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < cols; c += 16) {
                uint32_t x[16];
                float o[16];
                if (tiles > 0)
                    tc::tmem_ld16(o_at + c0 + c, x);
#pragma unroll
                for (int i = 0; i < 16; i++)
                    o[i] = inv != 0.f ? __uint_as_float(x[i]) * inv : 0.f;
                if constexpr (es == 2)
#pragma unroll
                    for (int i = 0; i < 16; i += 8)
                        *at(lane, (c + i) / 8) = make_uint4(pack2<T>(o[i], o[i + 1]), pack2<T>(o[i + 2], o[i + 3]),
                                                            pack2<T>(o[i + 4], o[i + 5]), pack2<T>(o[i + 6], o[i + 7]));
                else
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *at(lane, (c + i) / 4) = make_uint4(__float_as_uint(o[i]), __float_as_uint(o[i + 1]),
                                                            __float_as_uint(o[i + 2]), __float_as_uint(o[i + 3]));
            }
            __syncwarp();
            const int e = half * kCols + c0, c = lane % kRowChunks;
#pragma unroll
            for (int i = 0; i < kRowChunks; i++) {
                const int r = (i * 32 + lane) / kRowChunks;
                char *row_to = reinterpret_cast<char *>(__shfl_sync(0xffffffffu, reinterpret_cast<int64_t>(to), r));
                if (row_to && e + c * (16 / es) < p.d)
                    *reinterpret_cast<uint4 *>(row_to + e * es + c * 16) = *at(r, c);
            }
        }
    };
    if (w.whole)
        write(std::true_type{});
    else
        write(std::false_type{});
}

// The CTA's work.  In batches of up to kRanked sequences the longest come
// first, so that the last to start are the shortest: every CTA ranks the
// lengths (64 users with up to 200 candidates: 63 us in the batch's order, 55
// ranked).  More CTAs even out by themselves and would pay for the ranking (77
// users' own up to 439 events, 64 heads on 8 of 64: 300 us against 353).
// `room`: shared memory for kRanked lengths and one sequence.
constexpr int kRanked = 256;

static __device__ bool tile_work(const AttnParams &p, int *room, AttnWork &w)
{
    if (p.batch.S > kRanked || gridDim.x > 5 * tile_places(p.rows, p.d))
        return attn_work(p, blockIdx.x, w);
    int64_t tile;
    const int64_t rank = attn_number(p, blockIdx.x, w, tile);
    const int t = threadIdx.x, S = (int)p.batch.S, padded = (S + 3) & ~3;
    int *found = room + kRanked;  // sequence, first new token, new tokens, stored tokens
    Sequence seq = {0, 0, 0};
    int key = -1;  // of a sequence without work, and past the last
    if (t < S && read_sequence(p.batch, t, p.max_new, p.max_len, seq, blockIdx.x == 0 ? p.err : nullptr) &&
        seq.count > 0 && attn_takes(p, seq))
        key = seq.length;
    if (t < padded)
        room[t] = key;
    if (t == 0)
        found[2] = 0;
    __syncthreads();
    if (key >= 0) {
        int before = 0;
        for (int i = 0; i < padded; i += 4) {
            const int4 other = *reinterpret_cast<const int4 *>(room + i);
            before += (other.x > key || (other.x == key && i < t)) + (other.y > key || (other.y == key && i + 1 < t)) +
                      (other.z > key || (other.z == key && i + 2 < t)) + (other.w > key || (other.w == key && i + 3 < t));
        }
        if (before == rank) {
            found[0] = t;
            found[1] = (int)seq.first;
            found[2] = seq.count;
            found[3] = seq.length;
        }
    }
    __syncthreads();
    w.s = found[0];
    w.seq.first = found[1];
    w.seq.count = found[2];
    w.seq.length = found[3];
    tc::fence_async_smem();  // the room is overwritten by bulk copies, after the barrier that follows
    return w.seq.count > 0 && attn_rows(p, tile, w);
}

}  // namespace dlrm
