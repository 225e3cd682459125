// Attention over the paged cache by rows of 16: single tokens and short chunks,
// and fp32 tensors of every length.
//
// Such a call reads every key and value once and does little with each, so
// memory bounds it, and the design keeps loads in flight.  An item is a
// tile of 16 packed rows of one sequence and cache head; the positions of all
// items are laid end to end in units of four warp blocks, a CTA takes an equal
// run of units, whatever the lengths, and its warps stream their blocks through
// rings of asynchronous 16-byte copies that do not stop between items.  Every
// lane reads back exactly the chunks it copied itself, so the rings need no barrier:
//  - scores: MMAs of 16 rows x 8 tokens (m16n8k16; fp32: m16n8k8).  The order of
//    the summed elements is free, so a lane's 16-byte chunk of a key serves two
//    MMA steps as it is, with the query's chunks in the same order.
//  - output: MMAs of 16 rows x 8 columns, 16 (fp32: 8) tokens deep.  Which columns
//    form an MMA's 8 is free too: a lane's chunks of the same columns of two tokens,
//    interleaved by byte permutes, are the operands of 8 MMAs (fp32: 4, as they
//    are); and the order of the tokens is the one that the scores come out in.
// fp32 runs on TF32 MMAs: an operand is its upper 19 bits, which are what the MMA reads, plus the rest,
// exactly, and the three products of the split that matter carry each product of
// two elements to about 2^-20 of its magnitude; sums are fp32.
// A warp keeps its own running maximum, sum and output; the four are joined
// in shared memory at an item's end.  An item that spans CTAs leaves
// normalised partial rows and log2 of their sums, which a second kernel joins.
#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

constexpr int kFewWarps = 4, kFewRows = 16, kFewStages = 3;
constexpr int kFewCtas = 304;      // two for each of 152 SMs
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

// The same in fp32, 8 deep, as three TF32 MMAs: x = its upper bits + lo.
__device__ __forceinline__ void mma1688(float *c, const float *a, float b0, float b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
__device__ __forceinline__ float low_part(float x) { return x - tc::tf32_trunc(x); }
__device__ __forceinline__ void mma_fp32(float *c, const float *a, const float *a_lo, float b0, float b1)
{
    mma1688(c, a_lo, b0, b1);
    mma1688(c, a, low_part(b0), low_part(b1));
    mma1688(c, a, b0, b1);
}

// One item -- row tile `tile` of a sequence and head -- and its units
// [first, last).
struct FewItem {
    Sequence seq;
    int64_t s, first, last;
    int head, tile, tiles;
    int lo, hi;  // positions that the sequence's queries see
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

__device__ __forceinline__ int few_tiles(const AttnParams &p, const Sequence &q)
{
    return (int)(((int64_t)q.count * p.group + kFewRows - 1) / kFewRows);
}

// Sets the item to sequence s's first, from unit `first`; false where the
// sequence has no units.
__device__ __forceinline__ bool few_sequence(const AttnParams &p, FewItem &w, int64_t s, int64_t first, int unit)
{
    if (!read_sequence(p.batch, s, p.max_new, p.max_len, w.seq, nullptr))
        return false;
    const int units = few_units(p, w.seq, unit, w.lo, w.hi);
    w.s = s;
    w.head = w.tile = 0;
    w.tiles = few_tiles(p, w.seq);
    w.first = first;
    w.last = first + units;
    w.pages = p.batch.table + s * p.batch.table_stride;
    return units > 0;
}

__device__ __forceinline__ void few_next(const AttnParams &p, FewItem &w, int unit)
{
    if (++w.tile == w.tiles) {
        w.tile = 0;
        w.head++;
    }
    if (w.head < p.cache.heads) {
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
            mine += (int64_t)few_units(p, q, unit, lo, hi) * few_tiles(p, q) * p.cache.heads;
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
                units = (int64_t)few_units(p, q, unit, lo, hi) * few_tiles(p, q) * p.cache.heads;
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
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int E = 16 / sizeof(T);                    // elements of a chunk
    constexpr int MG = kWide ? 8 : 16, KT = MG / 8, VT = MG / 4;  // tokens of an MMA group; a lane's key and value rows
    constexpr int KG = DP / (4 * E), VS = DP / (8 * E);  // a lane's chunks of a key row, of a value row
    constexpr int TB = kFewStageBytes / (2 * DP * (int)sizeof(T)), NB = TB / MG, UT = kFewWarps * TB;
    constexpr int kChunks = KT * KG + VT * VS, kOut = VS * E * 4;  // chunks of a group; output registers
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_m[kFewWarps][kFewRows], s_l[kFewWarps][kFewRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    uint8_t *ring = smem + warp * kFewStages * kFewStageBytes + lane * 16;
    float *merge = reinterpret_cast<float *>(smem + kFewWarps * kFewStages * kFewStageBytes);  // [2][kOut][32]

    FewItem it;  // of the unit being computed; `is`: of the unit whose addresses come next
    int64_t u0 = 0, u1;
    bool split = p.splits > 1;
    if (split) {
        if (!few_share(p, it, u0, u1, UT))
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
        u1 = it.last;
    }
    FewItem is = it;

    // this lane's token of the warp's block of unit u: its page number and slot,
    // no slot for a position that no query sees; and its place in the cache, -1
    // there and in an invalid page
    int page_id = 0, page_slot = -1;
    auto find = [&](int64_t u) {
        page_slot = -1;
        if (u >= u1)
            return;
        while (u >= is.last)
            few_next(p, is, UT);
        const int at = is.lo + (int)(u - is.first) * UT + warp * TB + lane;
        if (lane < TB && at < is.hi) {
            const uint32_t page = p.cache.page.div((uint32_t)at);
            page_slot = at - (int)(page * p.cache.page.d);
            page_id = __ldg(is.pages + page);
        }
    };
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
    auto copy = [&](int stage, int64_t mine) {
        uint8_t *to = ring + stage * kFewStageBytes;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
#pragma unroll
            for (int t = 0; t < KT; t++) {
                const int64_t o = __shfl_sync(0xffffffffu, mine, nb * MG + t * 8 + g);
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const int e = (4 * i + q) * E;
                    const bool ok = o >= 0 && e < p.d;
                    tc::cp_async16(to, p.cache.k + (ok ? o + e * (int)sizeof(T) : 0), ok);
                    to += 512;
                }
            }
#pragma unroll
            for (int t = 0; t < VT; t++) {
                const int64_t o = __shfl_sync(0xffffffffu, mine, nb * MG + 2 * q + (t & 1) + (t >> 1) * 8);
#pragma unroll
                for (int i = 0; i < VS; i++) {
                    const int e = (8 * i + g) * E;
                    const bool ok = o >= 0 && e < p.d;
                    tc::cp_async16(to, p.cache.v + (ok ? o + e * (int)sizeof(T) : 0), ok);
                    to += 512;
                }
            }
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    find(u0);
#pragma unroll
    for (int i = 0; i < kFewStages - 1; i++) {
        const int64_t mine = place();
        find(u0 + i + 1);
        if (u0 + i < u1)
            copy(i, mine);
        commit();
    }

    uint4 qa[KG][2];         // the queries' chunks: rows g and g + 8
    float qlo[kWide ? KG : 1][2][4];  // fp32: their low parts
    float o[VS][E][4], m[2], l[2];
    int lo[2], hi[2], rows = 0;  // rows: of the sequence
    bool fresh = true, first_item = true;
    int stage = 0;
    for (int64_t u = u0; u < u1; u++) {
        if (fresh) {
            rows = it.seq.count * p.group;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = it.tile * kFewRows + g + 8 * h, t = r / p.group;
                m[h] = -INFINITY;
                l[h] = 0.f;
                hi[h] = r < rows ? seen_hi(it.seq, p.causal, t) : 0;
                lo[h] = seen_lo(hi[h], p.window);
                const T *src = p.q.row<T>(it.seq.first + (r < rows ? t : 0),
                                          r < rows ? it.head * p.group + r - t * p.group : 0);
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const int e = (4 * i + q) * E;
                    qa[i][h] = make_uint4(0, 0, 0, 0);
                    if (r < rows && e < p.d)
                        qa[i][h] = *reinterpret_cast<const uint4 *>(src + e);
                    if (kWide) {
                        qlo[i][h][0] = low_part(__uint_as_float(qa[i][h].x));
                        qlo[i][h][1] = low_part(__uint_as_float(qa[i][h].y));
                        qlo[i][h][2] = low_part(__uint_as_float(qa[i][h].z));
                        qlo[i][h][3] = low_part(__uint_as_float(qa[i][h].w));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kOut; i++)
                (&o[0][0][0])[i] = 0.f;
            fresh = false;
        }
        {
            const int into = stage == 0 ? kFewStages - 1 : stage - 1;
            const int64_t mine = place();  // of unit u + kFewStages - 1, whose page numbers were asked for a unit ago
            find(u + kFewStages);
            if (u + kFewStages - 1 < u1)
                copy(into, mine);
            commit();
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 1) : "memory");
        const uint4 *chunk = reinterpret_cast<const uint4 *>(ring + stage * kFewStageBytes);
        const int at = it.lo + (int)(u - it.first) * UT + warp * TB;
        float s[NB][KT][4];
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int t = 0; t < KT; t++) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    s[nb][t][j] = 0.f;
#pragma unroll
                for (int i = 0; i < KG; i++) {
                    const uint4 k = chunk[(nb * kChunks + t * KG + i) * 32];
                    const uint4 &a = qa[i][0], &b = qa[i][1];
                    if constexpr (kWide) {
                        const float x[4] = {__uint_as_float(a.x), __uint_as_float(b.x), __uint_as_float(a.y), __uint_as_float(b.y)};
                        const float y[4] = {__uint_as_float(a.z), __uint_as_float(b.z), __uint_as_float(a.w), __uint_as_float(b.w)};
                        const float xl[4] = {qlo[i][0][0], qlo[i][1][0], qlo[i][0][1], qlo[i][1][1]};
                        const float yl[4] = {qlo[i][0][2], qlo[i][1][2], qlo[i][0][3], qlo[i][1][3]};
                        mma_fp32(s[nb][t], x, xl, __uint_as_float(k.x), __uint_as_float(k.y));
                        mma_fp32(s[nb][t], y, yl, __uint_as_float(k.z), __uint_as_float(k.w));
                    } else {
                        const uint32_t x[4] = {a.x, b.x, a.y, b.y}, y[4] = {a.z, b.z, a.w, b.w};
                        mma16816<T>(s[nb][t], x, k.x, k.y);
                        mma16816<T>(s[nb][t], y, k.z, k.w);
                    }
                }
            }
        // rows g (elements 0, 1) and g + 8 (elements 2, 3), tokens 2q and 2q + 1 of each 8
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int t = 0; t < KT; t++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int pos = at + nb * MG + t * 8 + 2 * q + (j & 1), h = j >> 1;
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
                    for (int j = 0; j < E; j++) {
                        o[i][j][2 * h] *= f;
                        o[i][j][2 * h + 1] *= f;
                    }
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
#pragma unroll
            for (int t = 0; t < KT; t++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    s[nb][t][j] = exp2_approx(s[nb][t][j] - base[j >> 1]);
                    l[j >> 1] += s[nb][t][j];
                }
            const uint4 *values = chunk + (nb * kChunks + KT * KG) * 32;
            if constexpr (kWide) {
                const float *w = s[nb][0];
                const float pa[4] = {w[0], w[2], w[1], w[3]};
                const float pl[4] = {low_part(w[0]), low_part(w[2]), low_part(w[1]), low_part(w[3])};
#pragma unroll
                for (int i = 0; i < VS; i++) {
                    const uint4 v0 = values[i * 32], v1 = values[(VS + i) * 32];
                    mma_fp32(o[i][0], pa, pl, __uint_as_float(v0.x), __uint_as_float(v1.x));
                    mma_fp32(o[i][1], pa, pl, __uint_as_float(v0.y), __uint_as_float(v1.y));
                    mma_fp32(o[i][2], pa, pl, __uint_as_float(v0.z), __uint_as_float(v1.z));
                    mma_fp32(o[i][3], pa, pl, __uint_as_float(v0.w), __uint_as_float(v1.w));
                }
            } else {
                uint32_t pa[4];  // the weights, rounded to the type; their sum is of the unrounded ones
#pragma unroll
                for (int t = 0; t < KT; t++) {
                    pa[2 * t] = pack2<T>(s[nb][t][0], s[nb][t][1]);
                    pa[2 * t + 1] = pack2<T>(s[nb][t][2], s[nb][t][3]);
                }
#pragma unroll
                for (int i = 0; i < VS; i++) {
                    uint4 v[VT];
#pragma unroll
                    for (int t = 0; t < VT; t++)
                        v[t] = values[(t * VS + i) * 32];
                    const uint32_t *w0 = &v[0].x, *w1 = &v[1].x, *w2 = &v[2].x, *w3 = &v[3].x;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        mma16816<T>(o[i][2 * j], pa, __byte_perm(w0[j], w1[j], 0x5410),
                                    __byte_perm(w2[j], w3[j], 0x5410));
                        mma16816<T>(o[i][2 * j + 1], pa, __byte_perm(w0[j], w1[j], 0x7632),
                                    __byte_perm(w2[j], w3[j], 0x7632));
                    }
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
                for (int j = 0; j < E; j++) {
                    o[i][j][2 * h] *= f;
                    o[i][j][2 * h + 1] *= f;
                }
        }
        float *flat = &o[0][0][0];
        if (warp >= 2)
#pragma unroll
            for (int i = 0; i < kOut; i++)
                merge[((warp - 2) * kOut + i) * 32 + lane] = flat[i];
        __syncthreads();
        if (warp < 2)
#pragma unroll
            for (int i = 0; i < kOut; i++)
                flat[i] += merge[(warp * kOut + i) * 32 + lane];
        if (warp == 1)
#pragma unroll
            for (int i = 0; i < kOut; i++)
                merge[(kOut + i) * 32 + lane] = flat[i];
        __syncthreads();
        if (warp == 0) {
            const bool whole = it.first >= u0 && it.last <= u1;
            const int heads = p.cache.heads * p.group, slot = blockIdx.x * 2 + (first_item ? 0 : 1);
#pragma unroll
            for (int i = 0; i < kOut; i++)
                flat[i] += merge[(kOut + i) * 32 + lane];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int in = g + 8 * h, r = it.tile * kFewRows + in, t = r / p.group;
                const int head = it.head * p.group + r - t * p.group;
                if (r >= rows)
                    continue;
                if (q == 0) {
                    if (!whole)
                        p.part_lse[slot * p.rows + in] = lse[h];
                    else if (p.lse)
                        p.lse[(it.seq.first + t) * heads + head] = lse[h] * kLn2;
                }
#pragma unroll
                for (int i = 0; i < VS; i++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {  // columns e .. e + E - 1
                        const int e = (8 * i + 2 * q + c) * E;
                        if (e >= p.d)
                            continue;
                        float x[E];
#pragma unroll
                        for (int j = 0; j < E; j++)
                            x[j] = o[i][j][2 * h + c];
                        T *out = p.out.row<T>(it.seq.first + t, head) + e;
                        float4 *part = reinterpret_cast<float4 *>(p.part_o + ((int64_t)slot * p.rows + in) * p.d + e);
                        if (!whole) {
#pragma unroll
                            for (int j = 0; j < E; j += 4)
                                part[j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                        } else if constexpr (kWide) {
                            *reinterpret_cast<float4 *>(out) = make_float4(x[0], x[1], x[2], x[3]);
                        } else {
                            *reinterpret_cast<uint4 *>(out) = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]),
                                                                         pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
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
        const int64_t of = i / most, s = of / p.cache.heads;
        const int r = (int)(i - of * most), head = (int)(of - s * p.cache.heads), t = r / p.group;
        const int64_t before = p.prefix[s], all_units = p.prefix[s + 1] - before;
        const int64_t from = p.batch.offsets[s], token = from + t;
        if (all_units == 0 || token >= p.batch.offsets[s + 1])
            continue;
        const int64_t tiles = ((p.batch.offsets[s + 1] - from) * p.group + kFewRows - 1) / kFewRows;
        const int64_t units = all_units / (p.cache.heads * tiles);
        const int64_t first = before + (head * tiles + r / kFewRows) * units;
        const int64_t c0 = first / quota, c1 = (first + units - 1) / quota;
        if (c0 == c1)
            continue;
        // the first CTA's part is its last item's unless the item begins with it
        auto row = [&](int64_t c) {
            return (c * 2 + (c == c0 && c0 * quota < first ? 1 : 0)) * p.rows + r % kFewRows;
        };
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

static int64_t few_rows(int64_t rows) { return rows < kFewRows ? rows : kFewRows; }

size_t few_workspace(int64_t S, int64_t rows, int d, int64_t max_len)
{
    if (!few_splits(max_len))
        return 0;
    return (size_t)2 * kFewCtas * few_rows(rows) * (d + 1) * sizeof(float) + (size_t)(S + 2) * sizeof(int64_t);
}

template <typename T, int DP>
static int launch_few(AttnParams &p, void *workspace, cudaStream_t st)
{
    constexpr int smem = kFewWarps * kFewStages * kFewStageBytes + DP * 32 * 4;
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv_attn_few_kernel<T, DP>, smem, &done);
    if (s != DLRM_OK)
        return s;
    const bool split = few_splits(p.max_len);
    p.splits = split ? 2 : 1;
    p.prefix = static_cast<int64_t *>(workspace);
    p.part_o = reinterpret_cast<float *>(p.prefix + ((p.batch.S + 2) & ~(int64_t)1));
    p.rows = (int)few_rows(p.max_new * p.group);
    p.part_lse = p.part_o + (size_t)2 * kFewCtas * p.rows * p.d;
    const int64_t items = p.batch.S * p.cache.heads * ((p.max_new * p.group + kFewRows - 1) / kFewRows);
    if (items > 0x7fffffff)
        return DLRM_ERR_UNSUPPORTED;
    kv_attn_few_kernel<T, DP><<<(unsigned)(split ? kFewCtas : items), kFewWarps * 32, smem, st>>>(p);
    count_launch(st);
    if (split) {
        const int64_t need = (p.batch.S * p.cache.heads * p.max_new * p.group + 3) / 4;
        kv_attn_few_join_kernel<T><<<(unsigned)(need < 65536 ? need : 65536), 128, 0, st>>>(p);
        count_launch(st);
    }
    return launch_status();
}

int launch_kv_attn_few(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    if (dtype == DLRM_F32)
        return p.d <= 64 ? launch_few<float, 64>(p, workspace, st) : launch_few<float, 128>(p, workspace, st);
    if (dtype == DLRM_F16)
        return p.d <= 64 ? launch_few<__half, 64>(p, workspace, st) : launch_few<__half, 128>(p, workspace, st);
    return p.d <= 64 ? launch_few<__nv_bfloat16, 64>(p, workspace, st)
                     : launch_few<__nv_bfloat16, 128>(p, workspace, st);
}

}  // namespace dlrm
