// Attention over the cache in 8 bits by rows of 16: single tokens and short
// chunks, and chunks of every length in fp32 or with heads above 128.
//
// Memory bounds it, with half the bytes of the 16-bit cache, and the design is
// that of its rows of 16: items laid end to end in units, equal runs of them to
// the CTAs, a ring of stages for each warp that bulk tensor copies fill through
// the page table, the warp's own MMAs with the tokens as their 16 rows.  What 8
// bits change:
//  - E4M3's values are fp16 values, so codes become fp16 two at a time by one
//    conversion each and every product runs in fp16, whatever the queries' type.
//    bf16 and fp32 queries are lifted by a power of two that takes a row's largest element to 2^14
//    (exact but for what lies 2^-38 below that element); fp32 ones in two parts,
//    22 bits, as are their weights.
//  - A lane's 16-byte chunk of a key row serves four MMA steps, 16 columns of a
//    value row are a lane's; the codes of two tokens are interleaved by byte
//    permutes before they are converted, which puts them where the MMA wants pairs.
//  - The keys' powers multiply the scores, the values' powers the weights, in
//    fp32: a factor for a token and all rows, so 2 products for a score.  The keys' are relative to
//    the largest that the warp has seen so far, which is part of the scale, so that a lifted sum stays finite.
//    A weight is held relative to the largest power that the warp has seen so far
//    and rises with it (the output is scaled down when that grows, as it is when a maximum
//    does), so fp16's range is the row's: what a token gathers is off by at most
//    2^-36 of the largest weight times the largest power.
//  - A lane asks for the exponents of one token of the block (of two where it has 64) beside
//    the copies, a ring's length ahead; shuffles hand them out.  One lane issues a block's copies.
//  - A block is 8 KB where the registers allow: 64 tokens of heads of up to 64, 32 of
//    up to 128.  What a block costs beside its bytes (the wait, the maximum, the issue of its
//    copies) is the same for half as many.
//
// What bounds it: memory, and nearly as much the warps themselves.  Of 8 KB a warp
// takes 560 instructions, 128 of them conversions, which take two cycles of a
// quarter of an SM each.  One event each of 256 users with up to 8192 events (16 heads
// on 4, 128 bf16 elements): 174 us, 5.9 TB/s, 0.87 of a plain copy; the copies alone take
// 155, the arithmetic alone 135.  With heads of 64 fp16 elements: 111 us, 4.6 TB/s (140
// with blocks of 32 tokens); there a token's arithmetic, not its bytes, bounds it.  One
// history of 262143: 59 us, of which the join, the launches and the first loads take 12.
// 12 rows of 8 heads on 2 of 256 of 96 users with up to 3000: 65 us, 2.1 TB/s; their
// outputs' registers leave 8 warps an SM, each bound by its own latencies (75 us with the queries in
// registers too).  Slower: exponents by copies of 4 bytes (193 us for the 256 users), keys and values handed back one by one
// (188), blocks of 16 tokens with 4 CTAs an SM (247), scores by MMAs of E4M3 with
// queries in parts (205: the chip composes them of fp16 ones).
#include <type_traits>

#include "kv8.cuh"
#include "kv_few.cuh"

namespace dlrm {

// log2 of the growth of a maximum that is let pass before the output is scaled down, and of what weights are
// lifted by: at most 2^15 in all, fp16's range.  (A tile of 16 rows sees some maximum grow in almost every block of
// a short history.)
constexpr float kFew8Slack = 4.f, kFew8Lift = kWeightTop<__half> - kFew8Slack;

template <typename T, int DP, int kGroups>
struct Few8Shape {
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int MG = 16;                        // tokens of an MMA group
    static constexpr int TB = DP == 64 && !kWide ? 64 : DP <= 128 ? 32 : 16, NB = TB / MG, UT = kFewWarps * TB;
    static constexpr int kSets = TB > 32 ? 2 : 1;        // tokens of a block that a lane looks after
    static constexpr int KG = DP / 64;                   // a lane's chunks of 16 codes of a key row
    static constexpr int VB = DP >= 128 ? 16 : 8, VS = DP / (8 * VB);  // codes of its chunks of a value row, and their number
    static constexpr int kStageBytes = TB * 2 * DP;
    static constexpr int kStats = 2 * kGroups;           // rows whose statistics a lane holds
    // Two parts of a weight where fp16's 11 bits are not enough: fp32, and fp16 outputs of narrow tiles
    static constexpr bool kTwoParts = kWide || (std::is_same<T, __half>::value && kGroups == 1);
    static constexpr int kOutMmas = VB / 2;              // of a set of output columns
    static constexpr int kOut = kGroups * VS * kOutMmas * 4;
    static constexpr int kResident = !kWide && kGroups == 1 && DP <= 128 ? 3 : 2;
    static constexpr int kStages = kResident == 3 ? 2 : kStageBytes < 8192 ? 4 : 3;
    static constexpr int kCtas = kResident * kFewSms;
    static constexpr int kMerge = kOut < 32 ? kOut : 32;
    // Beside 128 registers of outputs the queries' 64 are too many: they lie in shared memory, where the warps' outputs
    // are joined later.  (fp32 heads of 128 on 16 rows, 64 users with up to 4000: 85 us so, 84 in registers.)
    static constexpr bool kQueryShared = DP == 256 && kGroups == 2;
    static constexpr int kSmem = 1024 + kFewWarps * kStages * kStageBytes + 2 * kMerge * 32 * 4;
    // a stage: columns of kWidth bytes of the block's keys, then of its values, each TB rows, swizzled over its width
    static constexpr int kWidth = DP >= 128 ? 128 : 64, kColumns = DP / kWidth, kColumnBytes = TB * kWidth;
    static_assert(2 * kColumns * kColumnBytes == kStageBytes && kCtas <= kFewMaxCtas, "a stage holds a block");

    // place of 16-byte unit u of row r in a column
    __device__ __forceinline__ static int at(int r, int u)
    {
        return r * kWidth + ((u ^ (kWidth == 128 ? r & 7 : r >> 1 & 3)) << 4);
    }
    // the 16 elements that a lane of quarter q takes of chunk i of a row: its column, and unit in it.  (Which are
    // summed together is free; so 8 lanes of a read meet no bank twice.)
    __device__ __forceinline__ static constexpr int column(int i) { return kWidth == 128 ? i >> 1 : 0; }
    __device__ __forceinline__ static constexpr int unit(int i, int q) { return kWidth == 128 ? 2 * q + (i & 1) : q; }

    // the row of a lane's statistic i, and the statistic of its output register o
    __device__ __forceinline__ static int row(int i, int q) { return 2 * q + (i & 1) + 8 * (i >> 1); }
    __device__ __forceinline__ static constexpr int stat(int o) { return (o & 1) + 2 * (o / (VS * kOutMmas * 4)); }
};

// 8 query elements as they lie.
template <typename T>
struct Few8Query {
    uint4 x[sizeof(T) / 2];

    __device__ __forceinline__ void load(const T *src, bool there)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++)
            x[i] = there ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ float2 pair(int i) const  // elements 2i, 2i + 1
    {
        if constexpr (sizeof(T) == 4) {
            const uint32_t *w = &x[i / 2].x + 2 * (i & 1);
            return make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        } else {
            return unpack2<T>((&x[0].x)[i]);
        }
    }
};

template <typename T, int DP, int kGroups>
__global__ void __launch_bounds__(kFewWarps * 32, Few8Shape<T, DP, kGroups>::kResident)
kv8_attn_few_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FewMaps maps)
{
    using Sh = Few8Shape<T, DP, kGroups>;
    constexpr int KG = Sh::KG, VS = Sh::VS, VB = Sh::VB, NB = Sh::NB, TB = Sh::TB, UT = Sh::UT, kStages = Sh::kStages;
    constexpr int kParts = Sh::kWide ? 2 : 1;  // of a query
    extern __shared__ uint8_t raw[];
    __shared__ float s_m[kFewWarps][kFewRows], s_l[kFewWarps][kFewRows];
    __shared__ uint64_t bars[kFewWarps][kStages];
    __shared__ int busy[kFewWarps * 32];
    __shared__ int aborted, died_at[kFewWarps];  // died_at: the unit whose wait ran out
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    uint8_t *smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    uint8_t *ring = smem + warp * kStages * Sh::kStageBytes;
    float *merge = reinterpret_cast<float *>(smem + kFewWarps * kStages * Sh::kStageBytes);  // [2][kMerge][32]

    FewItem it;  // of the unit being computed; `is`: of the unit whose addresses come next
    int units, quota = 0;  // of this CTA; the items' are counted from its first
    if (p.splits > 1) {
        const bool any = few_share(p, it, units, quota, UT, TB, busy);
        if (threadIdx.x == 0)
            p.joins[blockIdx.x].rows = 0;  // until an item is left unfinished
        if (!any)
            return;
    } else {
        const int64_t most = (few_new(p) * p.group + kFewRows - 1) / kFewRows, of = blockIdx.x / most;
        const int64_t s = of / p.cache.heads;
        if (!read_sequence(p.batch, s, p.max_new, p.max_len, it.seq, p.err) || !few_sequence(p, it, s, 0, UT, TB))
            return;
        it.head = (int)(of - s * p.cache.heads);
        it.tile = (int)(blockIdx.x - of * most);
        if (it.tile >= it.tiles)
            return;
        units = it.last;
    }
    FewItem is = it;

    // A lane finds the page and slot of one token of the warp's block, of two of 64 (their exponents are the lane's to
    // fetch), and one copies the boxes, whose places the lanes of their first tokens know; a box that no query sees anything of is
    // outside the map: zeros.
    const int parts = TB / maps.rows;
    constexpr int kSets = Sh::kSets;
    int page_id[kSets], page_slot[kSets];  // of the lane's tokens: lane, lane + 32
    bool token_seen[kSets];
    auto find = [&](int u) {
#pragma unroll
        for (int i = 0; i < kSets; i++) {
            page_id[i] = -1;
            page_slot[i] = 0;
            token_seen[i] = false;
        }
        if (u >= units)
            return;
        while (u >= is.last)
            few_next(p, is, UT, TB, busy);
#pragma unroll
        for (int i = 0; i < kSets; i++) {
            const int at = is.lo + (u - is.first) * UT + warp * TB + i * 32 + (lane & (TB - 1)), box = at & -maps.rows;
            if (box < is.hi && box + maps.rows > is.lo_seen) {
                const uint32_t page = p.cache.page.div((uint32_t)at);
                page_slot[i] = at - (int)(page * p.cache.page.d);
                page_id[i] = __ldg(is.pages + page);
                token_seen[i] = at >= is.lo_seen && at < is.hi;
            }
        }
    };
    const uint32_t ring_at = tc::smem_u32(ring);
    uint32_t k_exp[kStages][kSets], v_exp[kStages][kSets];  // of the lane's tokens of the next units
    bool dead = false;  // a wait ran out: nothing more is copied, the results are invalid
    // copies of unit u, whose page numbers were asked for a unit before, into a stage; then asks for the next
    auto copy = [&](int u, int stage, uint32_t *ke, uint32_t *ve) {
        if (u < units && !dead) {
            int known[kSets];
#pragma unroll
            for (int i = 0; i < kSets; i++) {
                const bool sound = (uint32_t)page_id[i] < p.cache.pages;
                if (token_seen[i] && !sound)
                    raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
                known[i] = sound ? page_id[i] : -1;
            }
            uint64_t *bar = &bars[warp][stage];
            // One lane issues them all: a copy's operands are the warp's, and lanes that each issue one take turns.
#pragma unroll 1
            for (int i = 0; i < parts; i++) {
                const int first = i * maps.rows;  // token
                const bool second = kSets > 1 && first >= 32;
                const int page = __shfl_sync(0xffffffffu, second ? known[kSets - 1] : known[0], first & 31);
                const int slot = __shfl_sync(0xffffffffu, second ? page_slot[kSets - 1] : page_slot[0], first & 31);
                if (tc::elect_one()) {
                    if (i == 0)
                        tc::mbar_expect_tx(bar, Sh::kStageBytes);
                    const uint32_t to = ring_at + stage * Sh::kStageBytes + first * Sh::kWidth;
#pragma unroll
                    for (int c = 0; c < Sh::kColumns; c++) {
                        tc::tma_load_4d(to + c * Sh::kColumnBytes, &maps.k, c * Sh::kWidth, slot, is.head, page, bar);
                        tc::tma_load_4d(to + (Sh::kColumns + c) * Sh::kColumnBytes, &maps.v, c * Sh::kWidth, slot, is.head,
                                        page, bar);
                    }
                }
                __syncwarp();
            }
        }
#pragma unroll
        for (int i = 0; i < kSets; i++) {
            ke[i] = ve[i] = 0;
            if (u < units && !dead && token_seen[i] && (uint32_t)page_id[i] < p.cache.pages) {
                const int64_t x = exp_offset(p.exp, page_id[i], page_slot[i], is.head);
                ke[i] = p.exp.k[x];
                ve[i] = p.exp.v[x];
            }
        }
        find(u + 1);
    };
    if (lane == 0)
        for (int i = 0; i < kStages; i++)
            tc::mbar_init(&bars[warp][i], 1);
    if (threadIdx.x == 0)
        aborted = 0;
    tc::mbar_init_fence();
    __syncthreads();
    find(0);
#pragma unroll
    for (int i = 0; i < kStages; i++)
        copy(i, i, k_exp[i], v_exp[i]);

    // the queries' chunks of rows g, g + 8 as fp16 (fp32: and the rest)
    uint32_t qa[Sh::kQueryShared ? 1 : kGroups][KG][kParts][8];
    uint4 *shared_q = reinterpret_cast<uint4 *>(merge) + lane;  // [group][chunk][part][2][32]
    float o[Sh::kOut], m[Sh::kStats], l[Sh::kStats], scale[Sh::kStats];
    int lo[Sh::kStats], hi[Sh::kStats], rows = 0;  // rows: of the sequence
    int all_lo = 0, all_hi = 0;  // positions that every row of the tile sees
    int key_exp = 0, top_exp = 0;  // the largest exponents of keys and values so far: scores and weights are relative to them
    int back[kGroups];             // of rows g, g + 8: 2^back undoes their queries' lifting
    auto set_scale = [&]() {
        const ScoreScale all(p.scale_log2, key_exp - 127);
#pragma unroll
        for (int i = 0; i < Sh::kStats; i++)
            scale[i] = all.times(std::is_same<T, __half>::value
                                     ? 0
                                     : __shfl_sync(0xffffffffu, back[i >> 1], (2 * q + (i & 1)) * 4));
    };
    bool fresh = true, first_item = true;
    int stage = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (int u = 0; u < units; u++) {
        if (fresh) {
            const int row0 = it.tile * kFewRows;
            rows = it.seq.count * p.group;
            all_hi = seen_hi(it.seq, p.causal, row0 / p.group);
            all_lo = seen_lo(seen_hi(it.seq, p.causal, (min(rows, row0 + kFewRows) - 1) / p.group), p.window);
            if constexpr (Sh::kQueryShared)
                __syncthreads();  // the item before has been joined
#pragma unroll
            for (int h = 0; h < kGroups; h++) {
                const int r = row0 + g + 8 * h, t = r / p.group;
                const T *src = p.q.row<T>(it.seq.first + (r < rows ? t : 0),
                                          r < rows ? it.head * p.group + r - t * p.group : 0);
                Few8Query<T> x[KG][2];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < KG; i++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const int e = Sh::column(i) * Sh::kWidth + Sh::unit(i, q) * 16 + 8 * j;
                        x[i][j].load(src + e, r < rows && e < p.d);
                        if constexpr (!std::is_same<T, __half>::value)
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const float2 y = x[i][j].pair(k);
                                top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
                            }
                    }
                float lift = 1.f;
                back[h] = 0;
                if constexpr (!std::is_same<T, __half>::value) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
                    if (top > 0.f && e < 255) {
                        lift = __uint_as_float((268 - e) << 23);  // 2^(127 + 14 - e)
                        back[h] = (int)e - (127 + 14);
                    }
                }
#pragma unroll
                for (int i = 0; i < KG; i++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            uint32_t &w = qa[Sh::kQueryShared ? 0 : h][i][0][4 * j + k];
                            if constexpr (std::is_same<T, __half>::value) {
                                w = (&x[i][j].x[0].x)[k];
                            } else {
                                float2 y = x[i][j].pair(k);
                                y = make_float2(y.x * lift, y.y * lift);
                                w = pack2<__half>(y.x, y.y);
                                if constexpr (Sh::kWide) {
                                    const float2 z = unpack2<__half>(w);
                                    qa[Sh::kQueryShared ? 0 : h][i][1][4 * j + k] = pack2<__half>(y.x - z.x, y.y - z.y);
                                }
                            }
                        }
                if constexpr (Sh::kQueryShared)
#pragma unroll
                    for (int i = 0; i < KG * kParts; i++) {
                        const uint32_t *w = qa[0][i / kParts][i % kParts];
                        uint4 *to = shared_q + (h * KG * kParts + i) * 64;
                        if (i % kFewWarps == warp) {
                            to[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            to[32] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
            }
            if constexpr (Sh::kQueryShared)
                __syncthreads();
#pragma unroll
            for (int i = 0; i < Sh::kStats; i++) {
                const int r = row0 + Sh::row(i, q);
                m[i] = -INFINITY;
                l[i] = 0.f;
                hi[i] = r < rows ? seen_hi(it.seq, p.causal, r / p.group) : 0;
                lo[i] = seen_lo(hi[i], p.window);
            }
            key_exp = 0;
            set_scale();
#pragma unroll
            for (int i = 0; i < Sh::kOut; i++)
                o[i] = 0.f;
            top_exp = 0;
            fresh = false;
        }
        if (!dead && !tc::mbar_wait(&bars[warp][stage], phase, &aborted, p.wait_polls)) {
            dead = true;
            died_at[warp] = u;
        }
        dead = __any_sync(0xffffffffu, dead);
        const uint8_t *block = ring + stage * Sh::kStageBytes;
        const int at = it.lo + (u - it.first) * UT + warp * TB;

        // scores: s[nb][x][j] is of token nb * 16 + g + 8 * (j >> 1) and statistic 2 * x + (j & 1)
        float s[NB][kGroups][4], weight[NB][2];  // weight: the power of a token's values
        auto stat_of = [](int x, int j) { return 2 * x + (j & 1); };
        int exps[kSets], new_key = 0, new_exp = 0;
#pragma unroll
        for (int i = 0; i < kSets; i++) {
            exps[i] = (int)(k_exp[0][i] | v_exp[0][i] << 8);
            new_key = max(new_key, (int)k_exp[0][i]);
            new_exp = max(new_exp, (int)v_exp[0][i]);
        }
        new_key = __reduce_max_sync(0xffffffffu, new_key);
        new_exp = max(top_exp, __reduce_max_sync(0xffffffffu, new_exp));
        if (new_key > key_exp) {
            key_exp = new_key;
            set_scale();
        }
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            float other[kGroups][4];  // every second MMA's sum: two chains, half as long
#pragma unroll
            for (int x = 0; x < kGroups; x++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s[nb][x][j] = other[x][j] = 0.f;
#pragma unroll
            for (int i = 0; i < KG; i++) {
                uint32_t a[4][4];  // of the chunk's four steps
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const uint4 k = *reinterpret_cast<const uint4 *>(
                        block + Sh::column(i) * Sh::kColumnBytes + Sh::at(nb * Sh::MG + t * 8 + g, Sh::unit(i, q)));
                    const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        decode4(w[e], a[e][t], a[e][t + 2]);
                }
#pragma unroll
                for (int n = 0; n < kGroups; n++) {
                    uint32_t b[kParts][8];
#pragma unroll
                    for (int part = 0; part < kParts; part++) {
                        if constexpr (Sh::kQueryShared) {
                            const uint4 *from = shared_q + ((n * KG + i) * kParts + part) * 64;
                            const uint4 x = from[0], y = from[32];
                            b[part][0] = x.x, b[part][1] = x.y, b[part][2] = x.z, b[part][3] = x.w;
                            b[part][4] = y.x, b[part][5] = y.y, b[part][6] = y.z, b[part][7] = y.w;
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; k++)
                                b[part][k] = qa[n][i][part][k];
                        }
                    }
                    if constexpr (Sh::kWide) {
                        // The MMA's own sums are cut off, not rounded: two steps, small terms first, then fp32
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int part = 1; part >= 0; part--)
#pragma unroll
                                for (int f = e; f < e + 2; f++)
                                    mma16816<__half>(t, a[f], b[part][2 * f], b[part][2 * f + 1]);
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                s[nb][n][j] += t[j];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            mma16816<__half>(e & 1 ? other[n] : s[nb][n], a[e], b[0][2 * e], b[0][2 * e + 1]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t mine = (uint32_t)__shfl_sync(0xffffffffu, exps[nb / 2 % kSets], (nb & 1) * Sh::MG + g + 8 * h);
                const float power = exp_power((uint32_t)max((int)(mine & 255) - key_exp + 127, 0));
                weight[nb][h] = __uint_as_float((uint32_t)max((int)(mine >> 8) - new_exp + 127, 0) << 23);
#pragma unroll
                for (int x = 0; x < kGroups; x++)
#pragma unroll
                    for (int j = 2 * h; j < 2 * h + 2; j++)
                        s[nb][x][j] = (s[nb][x][j] + other[x][j]) * power;
            }
        }
        const bool edge = at < all_lo || at + TB > all_hi;
        if (edge) {
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int x = 0; x < kGroups; x++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int pos = at + nb * Sh::MG + g + 8 * (j >> 1), i = stat_of(x, j);
                        s[nb][x][j] = pos >= lo[i] && pos < hi[i] ? s[nb][x][j] : -INFINITY;
                    }
            // values that no query sees may be anything: a zero weight would not do
            uint8_t *values = ring + stage * Sh::kStageBytes + Sh::kColumns * Sh::kColumnBytes;
            for (int r = lane; r < TB; r += 32)
                if (at + r < it.lo_seen || at + r >= it.hi)
                    for (int c = 0; c < 2 * DP / 32; c++)
                        *reinterpret_cast<uint4 *>(values + c * 16 / Sh::kWidth * Sh::kColumnBytes + r * Sh::kWidth +
                                                   c * 16 % Sh::kWidth) = make_uint4(0, 0, 0, 0);
            tc::fence_async_smem();  // the next copies come after
            __syncwarp();
        }
        float top[Sh::kStats], off[Sh::kStats];
        bool moved = new_exp > top_exp;
#pragma unroll
        for (int i = 0; i < Sh::kStats; i++) {
            top[i] = -INFINITY;
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int x = 0; x < kGroups; x++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (stat_of(x, j) == i)
                            top[i] = fmaxf(top[i], s[nb][x][j]);
#pragma unroll
            for (int step = 4; step < 32; step *= 2)
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], step));
            top[i] = __fmul_ru(top[i], scale[i]);
            moved |= top[i] > m[i] + kFew8Slack;
        }
        if (__any_sync(0xffffffffu, moved)) {
            const float down = __uint_as_float((uint32_t)max(127 + top_exp - new_exp, 0) << 23);
            float f[Sh::kStats];
#pragma unroll
            for (int i = 0; i < Sh::kStats; i++) {
                // a row's own growth alone, so that its bits do not depend on the other rows'
                const float next = top[i] > m[i] + kFew8Slack ? top[i] : m[i];
                f[i] = exp2_approx(m[i] - (next == -INFINITY ? 0.f : next));
                l[i] *= f[i];
                f[i] *= down;
                m[i] = next;
            }
#pragma unroll
            for (int i = 0; i < Sh::kOut; i++)
                o[i] *= f[Sh::stat(i)];
            top_exp = new_exp;
        }
#pragma unroll
        for (int i = 0; i < Sh::kStats; i++)
            off[i] = __fsub_rd(kFew8Lift, m[i] == -INFINITY ? 0.f : m[i]);
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
#pragma unroll
            for (int x = 0; x < kGroups; x++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int i = stat_of(x, j);
                    const float e = exp2_approx(fmaf(s[nb][x][j], scale[i], off[i]));
                    l[i] += e;
                    s[nb][x][j] = e * weight[nb][j >> 1];
                }
            // the weights, rounded to fp16, and in two parts what that leaves of them, rows to columns
            uint32_t b[kGroups][2], rest[kGroups][2];
#pragma unroll
            for (int n = 0; n < kGroups; n++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float x = s[nb][n][2 * h], y = s[nb][n][2 * h + 1];
                    const uint32_t w = pack2<__half>(x, y);
                    b[n][h] = transpose8x8(w);
                    if (Sh::kTwoParts) {
                        const float2 r = unpack2<__half>(w);
                        rest[n][h] = transpose8x8(pack2<__half>(x - r.x, y - r.y));
                    }
                }
#pragma unroll
            for (int i = 0; i < VS; i++) {
                uint32_t v[4][VB / 4];  // the lane's columns of tokens 2q, 2q + 1 and of those + 8
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    const int row = nb * Sh::MG + 2 * q + (t & 1) + 8 * (t >> 1);
                    const uint8_t *from = block + (Sh::kColumns + i) * Sh::kColumnBytes;
                    if constexpr (VB == 16) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(from + Sh::at(row, g));
                        v[t][0] = x.x, v[t][1] = x.y, v[t][2] = x.z, v[t][3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(from + Sh::at(row, g >> 1) + (g & 1) * 8);
                        v[t][0] = x.x, v[t][1] = x.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < VB / 4; j++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {  // columns 4j + 2c and the next of the lane's
                        const uint32_t x = __byte_perm(v[0][j], v[1][j], c ? 0x7362 : 0x5140);
                        const uint32_t y = __byte_perm(v[2][j], v[3][j], c ? 0x7362 : 0x5140);
                        uint32_t a[4];
                        decode4(x, a[0], a[1]);
                        decode4(y, a[2], a[3]);
#pragma unroll
                        for (int n = 0; n < kGroups; n++) {
                            float *sum = o + ((n * VS + i) * Sh::kOutMmas + 2 * j + c) * 4;
                            if constexpr (Sh::kWide) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816<__half>(t, a, rest[n][0], rest[n][1]);
                                mma16816<__half>(t, a, b[n][0], b[n][1]);
#pragma unroll
                                for (int k = 0; k < 4; k++)
                                    sum[k] += t[k];
                            } else {
                                if (Sh::kTwoParts)
                                    mma16816<__half>(sum, a, rest[n][0], rest[n][1]);
                                mma16816<__half>(sum, a, b[n][0], b[n][1]);
                            }
                        }
                    }
            }
        }
        __syncwarp();  // every lane has read the stage that is filled next
#pragma unroll
        for (int i = 0; i + 1 < kStages; i++) {
#pragma unroll
            for (int j = 0; j < kSets; j++) {
                k_exp[i][j] = k_exp[i + 1][j];
                v_exp[i][j] = v_exp[i + 1][j];
            }
        }
        copy(u + kStages, stage, k_exp[kStages - 1], v_exp[kStages - 1]);
        stage++;
        if (stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
        if (u + 1 < it.last && u + 1 < units)
            continue;

        // the item's (or the CTA's) last unit: join the warps
#pragma unroll
        for (int i = 0; i < Sh::kStats; i++) {
#pragma unroll
            for (int step = 4; step < 32; step *= 2)
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], step);
            if (g == 0) {
                s_m[warp][Sh::row(i, q)] = m[i];
                s_l[warp][Sh::row(i, q)] = l[i];
            }
        }
        __syncthreads();
        float lse[Sh::kStats], f[Sh::kStats];
        const float power = exp_power((uint32_t)top_exp);
#pragma unroll
        for (int i = 0; i < Sh::kStats; i++) {
            const int r = Sh::row(i, q);
            float all = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kFewWarps; w++)
                all = fmaxf(all, s_m[w][r]);
            const float b = all == -INFINITY ? 0.f : all;
#pragma unroll
            for (int w = 0; w < kFewWarps; w++)
                sum = fmaf(s_l[w][r], exp2_approx(s_m[w][r] - b), sum);
            // no weight at all: nothing is seen; a sum that is not a number stays one
            f[i] = sum == 0.f ? 0.f : exp2_approx(m[i] - b) / sum * power;
            lse[i] = sum == 0.f ? -INFINITY : all + (log2f(sum) - kFew8Lift);
        }
#pragma unroll
        for (int i = 0; i < Sh::kOut; i++)
            o[i] *= f[Sh::stat(i)];
#pragma unroll
        for (int r = 0; r < Sh::kOut; r += Sh::kMerge) {
            if (r > 0)
                __syncthreads();
            if (warp >= 2)
#pragma unroll
                for (int i = 0; i < Sh::kMerge; i++)
                    merge[((warp - 2) * Sh::kMerge + i) * 32 + lane] = o[r + i];
            __syncthreads();
            if (warp < 2)
#pragma unroll
                for (int i = 0; i < Sh::kMerge; i++)
                    o[r + i] += merge[(warp * Sh::kMerge + i) * 32 + lane];
            if (warp == 1)
#pragma unroll
                for (int i = 0; i < Sh::kMerge; i++)
                    merge[(Sh::kMerge + i) * 32 + lane] = o[r + i];
            __syncthreads();
            if (warp == 0)
#pragma unroll
                for (int i = 0; i < Sh::kMerge; i++)
                    o[r + i] += merge[(Sh::kMerge + i) * 32 + lane];
        }
        if (warp == 0) {
            const bool whole = it.first >= 0 && it.last <= units;
            const int heads = p.cache.heads * p.group, slot = blockIdx.x * 2 + (first_item ? 0 : 1);
#pragma unroll
            for (int i = 0; i < Sh::kStats; i++) {
                const int in = Sh::row(i, q), r = it.tile * kFewRows + in, t = r / p.group;
                const int head = it.head * p.group + r - t * p.group;
                if (r >= rows)
                    continue;
                if (g == 0) {
                    if (!whole)
                        p.part_lse[slot * p.rows + in] = lse[i];
                    else if (p.lse)
                        p.lse[(it.seq.first + t) * heads + head] = lse[i] * kLn2;
                }
                // the lane's runs of VB columns of this row, 8 at a time
#pragma unroll
                for (int c = 0; c < VS * VB / 8; c++) {
                    const int set = c / (VB / 8), in_set = c % (VB / 8), e = (8 * set + g) * VB + in_set * 8;
                    if (e >= p.d)
                        continue;
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        x[j] = o[(((i >> 1) * VS + set) * Sh::kOutMmas + in_set * 4 + (j >> 1)) * 4 + 2 * (j & 1) + (i & 1)];
                    T *out = p.out.row<T>(it.seq.first + t, head) + e;
                    float4 *wide = Sh::kWide && whole ? reinterpret_cast<float4 *>(out)
                                                      : reinterpret_cast<float4 *>(p.part_o + ((int64_t)slot * p.rows + in) * p.d + e);
                    if (!whole || Sh::kWide) {
                        wide[0] = make_float4(x[0], x[1], x[2], x[3]);
                        wide[1] = make_float4(x[4], x[5], x[6], x[7]);
                    } else if constexpr (!Sh::kWide) {
                        *reinterpret_cast<uint4 *>(out) = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]),
                                                                     pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
                    }
                }
            }
        }
        if (threadIdx.x == 0 && it.first >= 0 && it.last > units) {  // the CTAs after this one go on with it
            const int row0 = it.tile * kFewRows;
            FewJoin j;
            j.token = it.seq.first;
            j.head = it.head * p.group;
            j.row = row0;
            j.rows = min(rows - row0, kFewRows);
            j.first = blockIdx.x * 2 + (first_item ? 0 : 1);
            j.last = blockIdx.x + (it.last - 1) / quota;
            p.joins[blockIdx.x] = j;
        }
        fresh = true;
        first_item = false;
        if (u + 1 < units)
            few_next(p, it, UT, TB, busy);
    }
    if (dead) {
        // that unit and those copied ahead of it may still be in flight: none may be when the memory is given back
        __syncwarp();
        const int first = died_at[warp];
        for (int i = first; i < min(first + kStages, units); i++)
            tc::mbar_drain(&bars[warp][i % kStages], (i / kStages) & 1);
        if (lane == 0)
            raise_flag(p.err, DLRM_FLAG_WAIT_TIMEOUT);
    }
}

// Maps of the codes with boxes of `rows` slots; false where they cannot be described so.
static bool few8_maps(const AttnParams &p, int rows, FewMaps &m)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, p.cache.page.d, (cuuint64_t)p.cache.heads, p.cache.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.cache.slot_stride, (cuuint64_t)p.cache.head_stride,
                                   (cuuint64_t)p.cache.page_stride};
    const cuuint32_t box[4] = {p.d > 64 ? 128u : 64u, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = p.d > 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    // lines of 256 bytes where a head's rows fill them; else they would be its neighbours'
    const CUtensorMapL2promotion lines = p.cache.slot_stride == p.d ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                                                    : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    m.rows = rows;
    auto encode = [&](CUtensorMap *map, void *codes) {
        return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, codes, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, lines, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return encode(&m.k, p.cache.k) && encode(&m.v, p.cache.v);
}

// Bytes of an item up to which it stays whole.  Whole against runs, us (bf16): 256 users with up to 8192, 4 heads of 128,
// 187 and 178; 64 with up to 2000 28 and 36; 16 with up to 2000 22 and 25; one with 3000 20 and 18; 96 with 1500, 12
// rows of 2 heads of 256, 51 and 59.
constexpr int64_t kFew8WholeBytes = 480 << 10, kFew8WholeBytesPerItem = 1536;

template <typename T, int DP, int kGroups>
static int launch_few8(AttnParams &p, const FewMaps &maps, void *workspace, cudaStream_t st)
{
    using Sh = Few8Shape<T, DP, kGroups>;
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv8_attn_few_kernel<T, DP, kGroups>, Sh::kSmem, &done);
    if (s != DLRM_OK)
        return s;
    // a window bounds what an item's rows see, whatever the history's length
    const int64_t seen = p.window > 0 ? p.window + (p.causal ? few_new(p) : 0) : p.max_len;
    // items, idle sequences' among them; the batch cannot have more busy sequences than tokens
    const int64_t each = p.cache.heads * ((few_new(p) * p.group + kFewRows - 1) / kFewRows), items = p.batch.S * each;
    const int64_t busy = (p.batch.S < p.batch.n ? p.batch.S : p.batch.n) * each;
    const bool split = few_splits(seen < p.max_len ? seen : p.max_len, p.d, 1, busy, kFew8WholeBytes, kFew8WholeBytesPerItem);
    p.splits = split ? 2 : 1;
    p.joins = static_cast<FewJoin *>(workspace);
    p.part_o = reinterpret_cast<float *>(p.joins + kFewMaxCtas);
    p.rows = (int)few_rows(few_new(p) * p.group);
    p.part_lse = p.part_o + (size_t)2 * kFewMaxCtas * p.rows * p.d;
    if (items > 0x7fffffff)
        return DLRM_ERR_UNSUPPORTED;
    kv8_attn_few_kernel<T, DP, kGroups>
        <<<(unsigned)(split ? Sh::kCtas : items), kFewWarps * 32, Sh::kSmem, st>>>(p, maps);
    count_launch(st);
    if (split) {
        const dim3 grid(Sh::kCtas - 1, (unsigned)p.rows);
        kv_attn_few_join_kernel<T, (DP > 128 ? 2 : 1)><<<grid, kJoinWarps * 32, 0, st>>>(p);
        count_launch(st);
    }
    return launch_status();
}

template <typename T>
static int launch_few8_width(AttnParams &p, const FewMaps &maps, void *workspace, cudaStream_t st)
{
    const bool narrow = few_new(p) * p.group <= 8;
    if (p.d <= 64)
        return narrow ? launch_few8<T, 64, 1>(p, maps, workspace, st) : launch_few8<T, 64, 2>(p, maps, workspace, st);
    if constexpr (sizeof(T) == 2)
        if (p.d > 128)
            return narrow ? launch_few8<T, 256, 1>(p, maps, workspace, st)
                          : launch_few8<T, 256, 2>(p, maps, workspace, st);
    return narrow ? launch_few8<T, 128, 1>(p, maps, workspace, st) : launch_few8<T, 128, 2>(p, maps, workspace, st);
}

// False where the codes cannot be copied so (pages that are no multiple of 8 slots, strides or addresses that are
// none of 16 bytes); else launched, with `status`.
bool launch_kv8_attn_few(AttnParams &p, int dtype, void *workspace, cudaStream_t st, int &status)
{
    FewMaps maps = {};
    // of a box: a block's, where it does not cross a page
    int rows = p.d > 128 ? 16 : p.d > 64 || dtype == DLRM_F32 ? 32 : 64;
    while (rows > 8 && p.cache.page.d % rows != 0)
        rows /= 2;
    if (p.cache.page.d % rows != 0 || !few8_maps(p, rows, maps))
        return false;
    status = dtype == DLRM_F32   ? launch_few8_width<float>(p, maps, workspace, st)
             : dtype == DLRM_F16 ? launch_few8_width<__half>(p, maps, workspace, st)
                                 : launch_few8_width<__nv_bfloat16>(p, maps, workspace, st);
    return true;
}

}  // namespace dlrm
