// Attention over the paged cache by rows of 16: single tokens and short chunks,
// and chunks of every length in fp32 or with 16-bit heads above 128.
//
// Such a call reads every key and value once and does little with each, so
// memory bounds it, and the design keeps loads in flight.  An item is a tile of
// 16 packed rows of one sequence and cache head; the positions of all items are
// laid end to end in units of four warp blocks, a CTA takes an equal run of
// units, whatever the lengths, and its warps stream their blocks through rings
// that do not stop between items.  Pages of a multiple of 8 slots are copied by
// bulk tensor copies through the page table, in boxes of 8 or 16 rows: keys in
// columns of 64 bytes, values in columns of 128 bytes swizzled, so that the
// reads below meet no bank twice.  Other page sizes take asynchronous 16-byte
// copies, row by row, where every lane reads back exactly the chunks it copied
// itself; they share the load/store pipe with the reads (256 users of up to
// 8192 events: 444 us against 328).
//  - scores: MMAs of 16 tokens x 8 rows (m16n8k16; fp32: m16n8k8).  The order
//    of the summed elements is free, so a lane's 16-byte chunk of a key serves
//    two MMA steps as it is, with the query's chunks in the same order.
//  - output: MMAs of 16 columns x 8 rows, 16 tokens deep (fp32: 8).  Which
//    columns form an MMA's 16 is free too: a lane's chunks of the same columns
//    of four tokens, interleaved by byte permutes, are the operands of 4 MMAs
//    (fp32: of two tokens, 2 MMAs, as they are).  The weights, whose tokens are
//    in the lanes that hold rows next, are transposed by movmatrix (fp32: each
//    half of their bits).
// These are the warp's own MMAs, not those of tensor memory: 16 rows would fill
// an eighth of such a tile, and the tensor pipe is 15 % busy as it is.
// fp32 runs on TF32 MMAs: an operand is itself rounded to TF32 plus the rest (of
// which the MMA reads 11 bits), and the three products of the split that matter
// carry each product of two elements to about 2^-22 of its magnitude.  An MMA
// starts from zero and its sum is added in fp32: the MMA's own additions are
// cut off, which leaves 1e-5 of the output after 20000 events where a chain of
// MMAs runs on (4e-7 so).
// A warp keeps its own running maximum, sum and output; the four are joined in
// shared memory at an item's end.  An item that spans CTAs leaves normalised
// partial rows and log2 of their sums, which a second kernel joins.
//
// One event each of 256 users with up to 8192 events (16 heads on 4, 128 bf16
// elements): 322 us, 6.3 TB/s, 0.93 of a plain copy.  One history of 262143:
// 100 us, 5.4 TB/s, of which the join and its launch take 10.  fp32, 128 users who see
// 512 events (4 heads on 2 of 64): 21 us, 2.5 TB/s; there a CTA has 9 units, and its
// start, its end and the uneven spread of 256 items over 304 places count.
#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

constexpr int kFewWarps = 4, kFewRows = 16;
constexpr int kFewSms = 152, kFewMaxCtas = 3 * kFewSms;
constexpr int kFewStageBytes = 8192;  // of a warp: keys and values of a block (16 tokens of 128 16-bit elements)
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

// The same in fp32, 8 deep, as three TF32 MMAs: x = x rounded to TF32 + lo.
__device__ __forceinline__ void mma1688(float *c, const float *a, float b0, float b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
struct Split {
    float hi, lo;

    __device__ __forceinline__ Split() {}
    __device__ __forceinline__ Split(float x) : hi(tc::tf32_round(x)), lo(x - hi) {}
};
// Two steps.  The MMA's own sums are cut off, not rounded: it adds up 16
// products, small terms first, and the rest is added in fp32.
__device__ __forceinline__ void mma_fp32(float *c, const Split *a, const Split *b)
{
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int pass = 0; pass < 3; pass++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const Split *x = a + 4 * k, *y = b + 2 * k;
            float ax[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                ax[i] = pass == 0 ? x[i].lo : x[i].hi;
            mma1688(t, ax, pass == 1 ? y[0].lo : y[0].hi, pass == 1 ? y[1].lo : y[1].hi);
        }
#pragma unroll
    for (int i = 0; i < 4; i++)
        c[i] += t[i];
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
    int lo, hi, lo_seen;  // positions that the sequence's queries see, lo down to a multiple of 16
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
    return hi > lo ? (hi - (lo & ~15) + unit - 1) / unit : 1;
}

__device__ __forceinline__ int few_tiles(const AttnParams &p, const Sequence &q)
{
    return (int)(((int64_t)q.count * p.group + kFewRows - 1) / kFewRows);
}

// Sets the item to sequence s's first, from unit `first`; false where the
// sequence has no units.
__device__ __forceinline__ bool few_sequence(const AttnParams &p, FewItem &w, int64_t s, int first, int unit)
{
    if (!read_sequence(p.batch, s, p.max_new, p.max_len, w.seq, nullptr))
        return false;
    const int units = few_units(p, w.seq, unit, w.lo_seen, w.hi);
    w.lo = w.lo_seen & ~15;
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
__device__ __noinline__ int few_busy_after(const AttnParams &p, int s0, const int *busy)
{
    const int lane = threadIdx.x & 31, S = (int)p.batch.S, run = few_run(p), here = s0 / run;
    const int end = min((here + 1) * run, S);
    int next = -1;
    for (int s = s0 + 1; s < end && next < 0; s += 32) {
        Sequence mine;
        const bool some = s + lane < end && read_sequence(p.batch, s + lane, p.max_new, p.max_len, mine, nullptr) &&
                          mine.count > 0;
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
__device__ __forceinline__ void few_next(const AttnParams &p, FewItem &w, int unit, const int *busy)
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
    if (next >= 0 && few_sequence(p, w, next, first, unit))
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
__device__ bool few_share(const AttnParams &p, FewItem &w, int &units, int &quota_units, int unit, int *busy)
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
            mine += (int64_t)few_units(p, q, unit, lo, hi) * few_tiles(p, q) * p.cache.heads;
            first = first < 0 && q.count > 0 ? (int)s : first;
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
            here_units = (int64_t)few_units(p, q, unit, lo, hi) * few_tiles(p, q) * p.cache.heads;
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
    few_sequence(p, w, found[0], 0, unit);
    const int64_t each = w.last, skip = (u0 - found[1]) / each;
    w.tile = (int)(skip % w.tiles);
    w.head = (int)(skip / w.tiles);
    w.first = (int)(found[1] + skip * each - u0);
    w.last = w.first + (int)each;
    return true;
}

// Rows of a lane's softmax statistics and the layout of its output registers.
// The tokens are the MMAs' 16 rows and the query rows their 8 columns, kGroups
// of 8 (narrow tiles do half the work).
template <typename T, int DP, int kGroups, bool kBulk>
struct FewShape {
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int E = 16 / sizeof(T);                     // elements of a chunk
    static constexpr int MG = 16;                                // tokens of an MMA group
    static constexpr int KT = MG / 8, VT = MG / 4;               // a lane's key and value rows of a group
    static constexpr int KG = DP / (4 * E), VS = DP / (8 * E);   // its chunks of a key row, of a value row
    static constexpr int kTokenBytes = 2 * DP * (int)sizeof(T);  // keys and values
    // A group that fills two stages has its keys in one and its values in the next.
    static constexpr int kParts = MG * kTokenBytes / kFewStageBytes > 1 ? 2 : 1;
    static constexpr int TB = kParts * kFewStageBytes / kTokenBytes, NB = TB / MG, UT = kFewWarps * TB;
    static constexpr int kChunks = kParts > 1 ? 0 : KT * KG + VT * VS;  // from a group to the next
    static constexpr int kStats = 2 * kGroups;                   // rows whose statistics a lane holds
    // Up to 8 rows a 16-bit weight is carried in two parts, so that the output is rounded once: of 256 users
    // with up to 8192 events 323 -> 325 us, one of 262143 100.5 -> 100.8.  With 16 rows the
    // second MMA costs more than one rounding is worth (64 users 44 -> 47 us; 64 new of 256-wide heads 290 -> 319).
    static constexpr bool kTwoParts = !kWide && kGroups == 1;
    static constexpr int kOutMmas = E / 2;                       // of a set of output columns
    static constexpr int kOut = kGroups * VS * kOutMmas * 4;     // output registers
    // registers joined at a time: with all 64 of them two CTAs would not fit on an SM
    // CTAs of an SM and stages of a warp's ring: where 3 CTAs have the registers,
    // two stages each keep as many bytes in flight as three of 2, and an item's
    // start and end hide behind two others (with weights in one part: 256 users of up to 8192
    // events 320 us, 329 with 2; 512 users of up to 1000, 8 heads of 64: 94 and 117)
    static constexpr int kResident = kBulk && !kWide && kGroups == 1 && DP <= 128 ? 3 : 2, kStages = kResident == 3 ? 2 : 3;
    static constexpr int kCtas = kResident * kFewSms;
    static constexpr int kMerge = kOut < 32 ? kOut : 32;
    static constexpr int kSmem = 1024 + kFewWarps * kStages * kFewStageBytes + 2 * kMerge * 32 * 4;
    static constexpr int kKeyBox = MG * 64, kValueBox = MG * 128;  // bytes of a column of a group's keys, values
    static constexpr int kKeyBytes = kParts > 1 ? 0 : KG * kKeyBox;  // before a group's values
    static constexpr int kKeyChunks = kParts > 1 ? 0 : KT * KG;
    static constexpr int kGroupBytes = KG * kKeyBox + VS * kValueBox;
    static_assert(NB * MG == TB && (kParts == 1 || NB == 1), "a stage holds whole groups");

    // the row of a lane's statistic i, and the statistic of its output register o
    __device__ __forceinline__ static int row(int i, int q) { return 2 * q + (i & 1) + 8 * (i >> 1); }
    __device__ __forceinline__ static constexpr int stat(int o) { return (o & 1) + 2 * (o / (VS * kOutMmas * 4)); }
};

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

template <typename T, int DP, int kGroups, bool kBulk>
__global__ void __launch_bounds__(kFewWarps * 32, FewShape<T, DP, kGroups, kBulk>::kResident)
kv_attn_few_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FewMaps maps)
{
    using Sh = FewShape<T, DP, kGroups, kBulk>;
    constexpr int E = Sh::E, KT = Sh::KT, VT = Sh::VT, KG = Sh::KG, VS = Sh::VS, NB = Sh::NB, UT = Sh::UT;
    constexpr int kParts = Sh::kParts, kFewStages = Sh::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ float s_m[kFewWarps][kFewRows], s_l[kFewWarps][kFewRows];
    __shared__ uint64_t bars[kFewWarps][kFewStages];
    __shared__ int busy[kFewWarps * 32];
    __shared__ int aborted, died_at[kFewWarps];  // died_at: the part whose wait ran out
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    uint8_t *smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    uint8_t *ring = smem + warp * kFewStages * kFewStageBytes;
    float *merge = reinterpret_cast<float *>(smem + kFewWarps * kFewStages * kFewStageBytes);  // [2][kMerge][32]

    FewItem it;  // of the unit being computed; `is`: of the unit whose addresses come next
    int units, quota = 0;  // of this CTA; the items' are counted from its first
    if (p.splits > 1) {
        const bool any = few_share(p, it, units, quota, UT, busy);
        if (threadIdx.x == 0)
            p.joins[blockIdx.x].rows = 0;  // until an item is left unfinished
        if (!any)
            return;
    } else {
        const int64_t most = (p.max_new * p.group + kFewRows - 1) / kFewRows, of = blockIdx.x / most;
        const int64_t s = of / p.cache.heads;
        if (!read_sequence(p.batch, s, p.max_new, p.max_len, it.seq, p.err) || !few_sequence(p, it, s, 0, UT))
            return;
        it.head = (int)(of - s * p.cache.heads);
        it.tile = (int)(blockIdx.x - of * most);
        if (it.tile >= it.tiles)
            return;
        units = it.last;
    }
    FewItem is = it;

    // What this lane copies of the warp's block of unit u -- a box of its own, or
    // the row of token `lane` -- as a page number and slot; no slot where no
    // query sees it.
    const int boxes = Sh::MG / maps.rows * (KG + VS);  // of a group: its keys' columns, then its values'
    const int my_group = kBulk ? lane / boxes : lane / Sh::MG, my_box = kBulk ? lane - my_group * boxes : 0;
    const int my_part = kBulk ? my_box % (Sh::MG / maps.rows) : 0, my_column = kBulk ? my_box / (Sh::MG / maps.rows) : 0;
    const int my_token = kBulk ? my_group * Sh::MG + my_part * maps.rows : lane;
    const bool copies = my_group < NB;
    int page_id = 0, page_slot = -1;
    auto find = [&](int u) {
        page_slot = -1;
        if (u >= units)
            return;
        while (u >= is.last)
            few_next(p, is, UT, busy);
        const int at = is.lo + (u - is.first) * UT + warp * Sh::TB + my_token;
        if (copies && at < is.hi && at + (kBulk ? maps.rows : 1) > is.lo_seen) {
            const uint32_t page = p.cache.page.div((uint32_t)at);
            page_slot = at - (int)(page * p.cache.page.d);
            page_id = __ldg(is.pages + page);
        }
    };
    const uint32_t ring_at = tc::smem_u32(ring);
    auto copy_boxes = [&](int stage, int part) {
        if (lane == 0)
            tc::mbar_expect_tx(&bars[warp][stage], kFewStageBytes);
        __syncwarp();
        if (!copies || (kParts > 1 && (my_column >= KG) != part))
            return;
        if (page_slot >= 0 && (uint32_t)page_id >= p.cache.pages)
            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
        // a page number outside the cache, and -1 for what no query sees, is outside the map: zeros
        const int page = page_slot >= 0 && (uint32_t)page_id < p.cache.pages ? page_id : -1, slot = max(page_slot, 0);
        const uint32_t to = ring_at + stage * kFewStageBytes + my_group * Sh::kGroupBytes;
        if (my_column < KG)
            tc::tma_load_4d(to + my_column * Sh::kKeyBox + my_part * maps.rows * 64, &maps.k, my_column * 4 * E, slot,
                            is.head, page, &bars[warp][stage]);
        else
            tc::tma_load_4d(to + Sh::kKeyBytes + (my_column - KG) * Sh::kValueBox + my_part * maps.rows * 128,
                            &maps.v, (my_column - KG) * 8 * E, slot, is.head, page, &bars[warp][stage]);
    };
    // the lane's row: its place in the cache, -1 where there is none
    auto place = [&]() -> int64_t {
        if (page_slot < 0)
            return -1;
        if ((uint32_t)page_id >= p.cache.pages) {
            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
            return -1;
        }
        return (page_id * p.cache.page_stride + page_slot * p.cache.slot_stride + is.head * p.cache.head_stride) *
               (int64_t)sizeof(T);
    };
    auto copy_rows = [&](int stage, int part, int64_t mine) {
        uint32_t to = ring_at + stage * kFewStageBytes + lane * 16;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
#pragma unroll
            for (int t = 0; t < KT + VT; t++) {
                const bool key = t < KT;
                if (kParts > 1 && key == part)
                    continue;
                const int v = t - KT, token = key ? t * 8 + g : 2 * q + (v & 1) + (v >> 1) * 8;
                const int64_t at = __shfl_sync(0xffffffffu, mine, nb * Sh::MG + token);
                const char *from = (key ? p.cache.k + q * 16 : p.cache.v + g * 16) + (at >= 0 ? at : 0);
#pragma unroll
                for (int i = 0; i < (key ? KG : VS); i++) {
                    const bool there = at >= 0 && (key ? 4 * i + q : 8 * i + g) * E < p.d;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                                 "l"(there ? from + i * (key ? 64 : 128) : p.cache.k), "r"(there ? 16 : 0)
                                 : "memory");
                    to += 512;
                }
            }
        }
    };
    // copies of unit u (of its keys or values), whose page numbers were asked for a unit before, into a stage; then
    // asks for the next
    bool dead = false;  // a wait ran out: nothing more is copied, the results are invalid
    auto copy = [&](int u, int part, int stage) {
        if constexpr (kBulk) {
            if (u < units && !dead)
                copy_boxes(stage, part);
            if (part == kParts - 1)
                find(u + 1);
        } else {
            const int64_t row = place();
            if (part == kParts - 1)
                find(u + 1);
            if (u < units)
                copy_rows(stage, part, row);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    if constexpr (kBulk) {
        if (lane == 0)
            for (int i = 0; i < kFewStages; i++)
                tc::mbar_init(&bars[warp][i], 1);
        if (threadIdx.x == 0)
            aborted = 0;
        tc::mbar_init_fence();
        __syncthreads();
    }
    find(0);
#pragma unroll
    for (int i = 0; i < kFewStages - (kBulk ? 0 : 1); i++)
        copy(i / kParts, i % kParts, i);

    uint4 qa[Sh::kWide ? 1 : KG][kGroups];     // the queries' chunks of rows g, g + 8
    Split qs[Sh::kWide ? KG : 1][kGroups][4];  // fp32: split
    float o[Sh::kOut], m[Sh::kStats], l[Sh::kStats];
    int lo[Sh::kStats], hi[Sh::kStats], rows = 0;  // rows: of the sequence
    int all_lo = 0, all_hi = 0;  // positions that every row of the tile sees
    bool fresh = true, first_item = true;
    int stage = 0;
    uint32_t phase = 0;
    // waits for a part of unit u; goes on to the next stage when it has been read
    auto arrived = [&](int u, int part) {
        if constexpr (kBulk) {
            if (!dead && !tc::mbar_wait(&bars[warp][stage], phase, &aborted, p.wait_polls)) {
                dead = true;
                died_at[warp] = u * kParts + part;
            }
            dead = __any_sync(0xffffffffu, dead);
        } else {
            const int next = part + kFewStages - 1;
            copy(u + next / kParts, next % kParts, stage == 0 ? kFewStages - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 1) : "memory");
        }
    };
    auto read = [&](int u, int part) {
        if constexpr (kBulk) {
            __syncwarp();  // every lane has read the stage that is filled next
            const int next = part + kFewStages;
            copy(u + next / kParts, next % kParts, stage);
        }
        stage++;
        if (stage == kFewStages) {
            stage = 0;
            phase ^= 1;
        }
    };
#pragma unroll 1
    for (int u = 0; u < units; u++) {
        if (fresh) {
            const int row0 = it.tile * kFewRows;
            rows = it.seq.count * p.group;
            all_hi = seen_hi(it.seq, p.causal, row0 / p.group);
            all_lo = seen_lo(seen_hi(it.seq, p.causal, (min(rows, row0 + kFewRows) - 1) / p.group), p.window);
#pragma unroll
            for (int i = 0; i < Sh::kStats; i++) {
                const int r = row0 + Sh::row(i, q);
                m[i] = -INFINITY;
                l[i] = 0.f;
                hi[i] = r < rows ? seen_hi(it.seq, p.causal, r / p.group) : 0;
                lo[i] = seen_lo(hi[i], p.window);
            }
#pragma unroll
            for (int h = 0; h < kGroups; h++) {
                const int r = row0 + g + 8 * h, t = r / p.group;
                const T *src = p.q.row<T>(it.seq.first + (r < rows ? t : 0),
                                          r < rows ? it.head * p.group + r - t * p.group : 0);
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const int e = (4 * i + q) * E;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (r < rows && e < p.d)
                        x = *reinterpret_cast<const uint4 *>(src + e);
                    if constexpr (Sh::kWide) {
                        qs[i][h][0] = Split(__uint_as_float(x.x));
                        qs[i][h][1] = Split(__uint_as_float(x.y));
                        qs[i][h][2] = Split(__uint_as_float(x.z));
                        qs[i][h][3] = Split(__uint_as_float(x.w));
                    } else {
                        qa[i][h] = x;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < Sh::kOut; i++)
                o[i] = 0.f;
            fresh = false;
        }
        arrived(u, 0);
        const uint8_t *block = ring + stage * kFewStageBytes;
        // chunk i of a group's key row t * 8 + g, and of its value row 2q + (t & 1) + 8 (t >> 1)
        auto key_chunk = [&](int nb, int t, int i) {
            return *reinterpret_cast<const uint4 *>(
                kBulk ? block + nb * Sh::kGroupBytes + i * Sh::kKeyBox + (t * 8 + g) * 64 + q * 16
                      : block + (nb * Sh::kChunks + t * KG + i) * 512 + lane * 16);
        };
        auto value_chunk = [&](int nb, int t, int i) {
            const int row = 2 * q + (t & 1);
            return *reinterpret_cast<const uint4 *>(
                kBulk ? block + nb * Sh::kGroupBytes + Sh::kKeyBytes + i * Sh::kValueBox + (t >> 1) * 1024 +
                            row * 128 + ((g ^ row) << 4)
                      : block + (nb * Sh::kChunks + Sh::kKeyChunks + t * VS + i) * 512 + lane * 16);
        };
        const int at = it.lo + (u - it.first) * UT + warp * Sh::TB;

        // scores: s[nb][x][j] is of token token_of(nb, x, j) and statistic stat_of(x, j)
        float s[NB][kGroups][4];
        auto token_of = [&](int nb, int j) { return nb * Sh::MG + g + 8 * (j >> 1); };
        auto stat_of = [](int x, int j) { return 2 * x + (j & 1); };
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
                const uint4 k = key_chunk(nb, 0, i), k8 = key_chunk(nb, 1, i);
                if constexpr (Sh::kWide) {
                    const Split x[8] = {__uint_as_float(k.x), __uint_as_float(k8.x), __uint_as_float(k.y),
                                        __uint_as_float(k8.y), __uint_as_float(k.z), __uint_as_float(k8.z),
                                        __uint_as_float(k.w), __uint_as_float(k8.w)};
#pragma unroll
                    for (int n = 0; n < kGroups; n++)
                        mma_fp32(i & 1 ? other[n] : s[nb][n], x, qs[i][n]);
                } else {
                    const uint32_t x[4] = {k.x, k8.x, k.y, k8.y}, y[4] = {k.z, k8.z, k.w, k8.w};
#pragma unroll
                    for (int n = 0; n < kGroups; n++) {
                        mma16816<T>(s[nb][n], x, qa[i][n].x, qa[i][n].y);
                        mma16816<T>(other[n], y, qa[i][n].z, qa[i][n].w);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < kGroups; x++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s[nb][x][j] += other[x][j];
        }
        if constexpr (kParts > 1) {
            read(u, 0);
            arrived(u, 1);
            block = ring + stage * kFewStageBytes;
        }
        const bool edge = at < all_lo || at + Sh::TB > all_hi;
        if (edge) {
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int x = 0; x < kGroups; x++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int pos = at + token_of(nb, j), i = stat_of(x, j);
                        s[nb][x][j] = pos >= lo[i] && pos < hi[i] ? s[nb][x][j] : -INFINITY;
                    }
        }
        float top[Sh::kStats], base[Sh::kStats], off[Sh::kStats];
        bool moved = false;
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
            top[i] = fmaxf(__fmul_ru(top[i], p.scale_log2), m[i]);
            base[i] = top[i] == -INFINITY ? 0.f : top[i];
            off[i] = __fsub_rd(kWeightTop<T>, base[i]);
            moved |= top[i] > m[i];
        }
        if (__any_sync(0xffffffffu, moved)) {
            float f[Sh::kStats];
#pragma unroll
            for (int i = 0; i < Sh::kStats; i++) {
                f[i] = exp2_approx(m[i] - base[i]);
                l[i] *= f[i];
                m[i] = top[i];
            }
#pragma unroll
            for (int i = 0; i < Sh::kOut; i++)
                o[i] *= f[Sh::stat(i)];
        }
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
#pragma unroll
            for (int x = 0; x < kGroups; x++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int i = stat_of(x, j);
                    s[nb][x][j] = exp2_approx(fmaf(s[nb][x][j], p.scale_log2, off[i]));
                    l[i] += s[nb][x][j];
                }
            // a box's rows that no query sees may hold anything: a zero weight would not do
            auto value = [&](int t, int i) {
                uint4 v = value_chunk(nb, t, i);
                if (kBulk && edge) {
                    const int pos = at + nb * Sh::MG + 2 * q + (t & 1) + 8 * (t >> 1);
                    if (pos < it.lo_seen || pos >= it.hi)
                        v = make_uint4(0, 0, 0, 0);
                }
                return v;
            };
            if constexpr (Sh::kWide) {
                // the weights, rows to columns: b[n] of tokens 2q, 2q + 1 and of those + 8
                Split b[kGroups][4];
#pragma unroll
                for (int n = 0; n < kGroups; n++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t w0 = __float_as_uint(s[nb][n][2 * h]), w1 = __float_as_uint(s[nb][n][2 * h + 1]);
                        const uint32_t lower = transpose8x8(__byte_perm(w0, w1, 0x5410));
                        const uint32_t upper = transpose8x8(__byte_perm(w0, w1, 0x7632));
                        b[n][2 * h] = __uint_as_float(__byte_perm(lower, upper, 0x5410));
                        b[n][2 * h + 1] = __uint_as_float(__byte_perm(lower, upper, 0x7632));
                    }
#pragma unroll
                for (int i = 0; i < VS; i++) {
                    uint4 v[VT];
#pragma unroll
                    for (int t = 0; t < VT; t++)
                        v[t] = value(t, i);
#pragma unroll
                    for (int j = 0; j < 2; j++) {  // columns 2j and 2j + 1 of each lane's four
                        Split a[8];
#pragma unroll
                        for (int t = 0; t < VT; t++) {
                            a[(t >> 1) * 4 + 2 * (t & 1)] = __uint_as_float(j ? v[t].z : v[t].x);
                            a[(t >> 1) * 4 + 2 * (t & 1) + 1] = __uint_as_float(j ? v[t].w : v[t].y);
                        }
#pragma unroll
                        for (int n = 0; n < kGroups; n++)
                            mma_fp32(o + ((n * VS + i) * 2 + j) * 4, a, b[n]);
                    }
                }
            } else {
                // the weights, rounded to the type, and in narrow tiles what that leaves of them, rows to columns
                uint32_t b[kGroups][2], rest[kGroups][2];
#pragma unroll
                for (int n = 0; n < kGroups; n++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const float x = s[nb][n][2 * h], y = s[nb][n][2 * h + 1];
                        const uint32_t w = pack2<T>(x, y);
                        const float2 r = unpack2<T>(w);
                        b[n][h] = transpose8x8(w);
                        if (Sh::kTwoParts)
                            rest[n][h] = transpose8x8(pack2<T>(x - r.x, y - r.y));
                    }
#pragma unroll
                for (int i = 0; i < VS; i++) {
                    uint4 v[VT];
#pragma unroll
                    for (int t = 0; t < VT; t++)
                        v[t] = value(t, i);
                    const uint32_t *w0 = &v[0].x, *w1 = &v[1].x, *w2 = &v[2].x, *w3 = &v[3].x;
#pragma unroll
                    for (int j = 0; j < 4; j++) {  // columns 2j and 2j + 1 of each lane's eight
                        const uint32_t a[4] = {__byte_perm(w0[j], w1[j], 0x5410), __byte_perm(w0[j], w1[j], 0x7632),
                                               __byte_perm(w2[j], w3[j], 0x5410), __byte_perm(w2[j], w3[j], 0x7632)};
#pragma unroll
                        for (int n = 0; n < kGroups; n++) {
                            float *sum = o + ((n * VS + i) * 4 + j) * 4;
                            if (Sh::kTwoParts)
                                mma16816<T>(sum, a, rest[n][0], rest[n][1]);
                            mma16816<T>(sum, a, b[n][0], b[n][1]);
                        }
                    }
                }
            }
        }
        read(u, kParts - 1);
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
            f[i] = sum == 0.f ? 0.f : exp2_approx(m[i] - b) / sum;
            lse[i] = sum == 0.f ? -INFINITY : all + (log2f(sum) - kWeightTop<T>);
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
                // the lane's runs of E columns of this row: one of each set
#pragma unroll
                for (int c = 0; c < VS; c++) {
                    const int e = (8 * c + g) * E;
                    if (e >= p.d)
                        continue;
                    float x[E];
#pragma unroll
                    for (int j = 0; j < E; j++)
                        x[j] = o[(((i >> 1) * VS + c) * Sh::kOutMmas + (j >> 1)) * 4 + 2 * (j & 1) + (i & 1)];
                    T *out = p.out.row<T>(it.seq.first + t, head) + e;
                    float4 *part = reinterpret_cast<float4 *>(p.part_o + ((int64_t)slot * p.rows + in) * p.d + e);
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < E; j += 4)
                            part[j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                    } else if constexpr (Sh::kWide) {
                        *reinterpret_cast<float4 *>(out) = make_float4(x[0], x[1], x[2], x[3]);
                    } else {
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
            few_next(p, it, UT, busy);
    }
    if (kBulk && dead) {
        // that part and those copied ahead of it may still be in flight: none may be when the memory is given back
        __syncwarp();
        const int first = died_at[warp];
        for (int i = first; i < min(first + kFewStages, units * kParts); i++)
            tc::mbar_drain(&bars[warp][i % kFewStages], (i / kFewStages) & 1);
        if (lane == 0)
            raise_flag(p.err, DLRM_FLAG_WAIT_TIMEOUT);
    }
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

static bool few_splits(int64_t seen, int d, int es, int64_t items)
{
    return seen * d * 2 * es > kFewWholeBytes + items * kFewWholeBytesPerItem;
}

static int64_t few_rows(int64_t rows) { return rows < kFewRows ? rows : kFewRows; }

size_t few_workspace(int64_t rows, int d, int64_t max_len)
{
    if (!few_splits(max_len, d, 4, 0))
        return 0;
    return (size_t)2 * kFewMaxCtas * few_rows(rows) * (d + 1) * sizeof(float) + kFewMaxCtas * sizeof(FewJoin);
}

// Maps of the cache with boxes of `rows` slots; false where it cannot be
// described so.
static bool few_maps(const AttnParams &p, int dtype, int rows, FewMaps &m)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    const int es = dtype == DLRM_F32 ? 4 : 2;
    const CUtensorMapDataType type = dtype == DLRM_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == DLRM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, p.cache.page.d, (cuuint64_t)p.cache.heads, p.cache.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.cache.slot_stride * es, (cuuint64_t)p.cache.head_stride * es,
                                   (cuuint64_t)p.cache.page_stride * es};
    const cuuint32_t k_box[4] = {(cuuint32_t)(64 / es), (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
    const cuuint32_t v_box[4] = {(cuuint32_t)(128 / es), (cuuint32_t)rows, 1, 1};
    // lines of 256 bytes where a head's rows fill them; else they would be its neighbours' (8
    // interleaved heads of 64 16-bit elements: 146 us, 126 with 128)
    const CUtensorMapL2promotion lines = p.d * es >= 256 || p.cache.slot_stride == p.d ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                                                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    m.rows = rows;
    return enc(&m.k, type, 4, p.cache.k, dims, strides, k_box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, lines, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
               CUDA_SUCCESS &&
           enc(&m.v, type, 4, p.cache.v, dims, strides, v_box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, lines, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
               CUDA_SUCCESS;
}

template <typename T, int DP, int kGroups, bool kBulk>
static int launch_few(AttnParams &p, const FewMaps &maps, void *workspace, cudaStream_t st)
{
    constexpr int smem = FewShape<T, DP, kGroups, kBulk>::kSmem;
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv_attn_few_kernel<T, DP, kGroups, kBulk>, smem, &done);
    if (s != DLRM_OK)
        return s;
    // a window bounds what an item's rows see, whatever the history's length
    const int64_t seen = p.window > 0 ? p.window + (p.causal ? p.max_new : 0) : p.max_len;
    // items, idle sequences' among them; the batch cannot have more busy sequences than tokens
    const int64_t each = p.cache.heads * ((p.max_new * p.group + kFewRows - 1) / kFewRows), items = p.batch.S * each;
    const int64_t busy = (p.batch.S < p.batch.n ? p.batch.S : p.batch.n) * each;
    const bool split = few_splits(seen < p.max_len ? seen : p.max_len, p.d, sizeof(T), busy);
    p.splits = split ? 2 : 1;
    p.joins = static_cast<FewJoin *>(workspace);
    p.part_o = reinterpret_cast<float *>(p.joins + kFewMaxCtas);
    p.rows = (int)few_rows(p.max_new * p.group);
    p.part_lse = p.part_o + (size_t)2 * kFewMaxCtas * p.rows * p.d;
    if (items > 0x7fffffff)
        return DLRM_ERR_UNSUPPORTED;
    kv_attn_few_kernel<T, DP, kGroups, kBulk>
        <<<(unsigned)(split ? FewShape<T, DP, kGroups, kBulk>::kCtas : items), kFewWarps * 32, smem, st>>>(p, maps);
    count_launch(st);
    if (split) {
        const dim3 grid(FewShape<T, DP, kGroups, kBulk>::kCtas - 1, (unsigned)p.rows);
        kv_attn_few_join_kernel<T, (DP > 128 ? 2 : 1)><<<grid, kJoinWarps * 32, 0, st>>>(p);
        count_launch(st);
    }
    return launch_status();
}

template <typename T, int kGroups>
static int launch_few_width(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    FewMaps maps = {};
    maps.rows = p.cache.page.d % 16 == 0 ? 16 : 8;
    const bool bulk = p.cache.page.d % 8 == 0 && few_maps(p, dtype, maps.rows, maps);
    if (p.d <= 64)
        return bulk ? launch_few<T, 64, kGroups, true>(p, maps, workspace, st)
                    : launch_few<T, 64, kGroups, false>(p, maps, workspace, st);
    if constexpr (sizeof(T) == 2)
        if (p.d > 128)
            return bulk ? launch_few<T, 256, kGroups, true>(p, maps, workspace, st)
                        : launch_few<T, 256, kGroups, false>(p, maps, workspace, st);
    return bulk ? launch_few<T, 128, kGroups, true>(p, maps, workspace, st)
                : launch_few<T, 128, kGroups, false>(p, maps, workspace, st);
}

int launch_kv_attn_few(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    const bool narrow = p.max_new * p.group <= 8;
    if (dtype == DLRM_F32)
        return narrow ? launch_few_width<float, 1>(p, dtype, workspace, st)
                      : launch_few_width<float, 2>(p, dtype, workspace, st);
    if (dtype == DLRM_F16)
        return narrow ? launch_few_width<__half, 1>(p, dtype, workspace, st)
                      : launch_few_width<__half, 2>(p, dtype, workspace, st);
    return narrow ? launch_few_width<__nv_bfloat16, 1>(p, dtype, workspace, st)
                  : launch_few_width<__nv_bfloat16, 2>(p, dtype, workspace, st);
}

}  // namespace dlrm
