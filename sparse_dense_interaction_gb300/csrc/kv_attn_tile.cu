// Attention over the paged cache for many rows: tiles of 256 rows on the
// tensor cores.
//
// A CTA holds two query tiles of 128 packed rows and walks the positions in
// tiles of 128.  Warp roles:
//  - warps 8 and 9 copy: a thread resolves one position's slot through the page
//    table, and the warp copies rows with asynchronous 16-byte copies
//    into a ring of key and value tiles in the 128-byte swizzle -- any page
//    size and layout, and rows that no query sees are filled with zeros
//    without being read, so nothing stale meets a zero weight;
//  - one thread of warp 10 issues the MMAs: S = Q K^T (both operands in
//    shared memory, K-major) and O += P V (P in tensor memory, V MN-major as it lies);
//  - warps 0-3 and 4-7 are the softmax of one query tile each: a thread owns a
//    row, reads its 128 scores, and writes the weights over them, in 16 bits.
// The two tiles take turns: while one's scores are exponentiated the other's
// MMAs run.  The running maximum a row is scaled by lags: the output (in
// tensor memory) and the sum are rescaled only when the maximum has grown by more than
// 2^8, which rarely happens after the first tiles; a weight is then at most 2^8,
// and sum and output carry the same factor, so nothing is lost.
// Tensor memory: scores 2 x 128 columns (the weights on top of them), output 2 x DP.
#include <type_traits>

#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

// Eleven warps leave a thread 184 registers: a softmax row's 128 scores stay in them.
constexpr int kTileThreads = 352, kTilePos = 128, kCopyThreads = 64;
constexpr int kTileLag = 3;         // copied tiles that may be in flight before one is waited for
constexpr float kTileSlack = 8.f;   // log2 of the growth of a maximum that is let pass

template <int DP>
struct TileShape {
    static constexpr int kTileBytes = kTilePos * DP * 2;  // of keys or values; a query tile too
    static constexpr int kSlots = DP == 128 ? 5 : 8;
    static constexpr int kSmem = 1024 + 2 * kTileBytes + kSlots * kTileBytes;
    static constexpr int kBlock = kTilePos * 128;         // bytes between 64-column blocks of a tile
    static constexpr int kChunks = DP / 8;                // 16-byte chunks of a row
};

struct TileBars {
    uint64_t full[8], empty[8], q_full, s_full[2], p_ready[2], o_full[2], drained;
    uint32_t tmem;
    int aborted;
};

// Copies 32 rows (this warp's) of a tile: lane t of the warp knows row t's
// byte offset from `base`, -1 for a row of zeros.
template <int DP>
__device__ __forceinline__ void copy_rows(uint8_t *tile, const char *base, int64_t mine, int row0, int d)
{
    constexpr int C = TileShape<DP>::kChunks, kRows = 32 / C;  // rows of a step
    const int lane = threadIdx.x & 31, c = lane % C;
#pragma unroll
    for (int i = 0; i < C; i++) {
        const int r = i * kRows + lane / C;
        const int64_t o = __shfl_sync(0xffffffffu, mine, r);
        const bool ok = o >= 0 && c * 8 < d;
        tc::cp_async16(tile + (c >> 3) * TileShape<DP>::kBlock + (row0 + r) * 128 + (((c & 7) ^ (r & 7)) << 4),
                       base + (ok ? o + c * 16 : 0), ok);
    }
}

template <typename T, int DP>
__device__ void tile_copy(const AttnParams &p, const AttnWork &w, uint8_t *sq, uint8_t *ring, TileBars &b, int tiles)
{
    using Sh = TileShape<DP>;
    const int tid = threadIdx.x - 256, row0 = tid & ~31;
#pragma unroll
    for (int t = 0; t < 4; t++) {
        const int r = t * 64 + tid, row = w.row0 + r, token = row / p.group;
        const int64_t o = r < w.rows ? ((w.seq.first + token) * p.q.ts +
                                        (int64_t)(w.head * p.group + row - token * p.group) * p.q.hs) * 2
                                     : -1;
        copy_rows<DP>(sq + (t >> 1) * Sh::kTileBytes, p.q.ptr, o, (t & 1) * 64 + row0, p.d);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int32_t *pages = p.batch.table + w.s * p.batch.table_stride;
    auto place = [&](int j, int half) -> int64_t {
        const int at = w.lo + j * kTilePos + half * 64 + tid;
        if (j >= tiles || at >= w.hi)
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
            if (i >= Sh::kSlots && !tc::mbar_wait(&b.empty[slot], (i / Sh::kSlots - 1) & 1, &b.aborted))
                return tc::cp_async_wait_all();
            copy_rows<DP>(ring + slot * Sh::kTileBytes, kv ? p.cache.v : p.cache.k, mine0, row0, p.d);
            copy_rows<DP>(ring + slot * Sh::kTileBytes, kv ? p.cache.v : p.cache.k, mine1, 64 + row0, p.d);
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

template <typename T, int DP>
__device__ void tile_mma(uint8_t *sq, uint8_t *ring, TileBars &b, int tiles, bool two)
{
    using Sh = TileShape<DP>;
    constexpr int kType = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    constexpr uint32_t kScores = tc::f16_idesc(kType, 128, kTilePos, false), kOut = tc::f16_idesc(kType, 128, DP, true);
    const uint32_t q = tc::smem_u32(sq), kv = tc::smem_u32(ring);
    auto scores = [&](int t, int j) {
        const uint32_t k = kv + (2 * j % Sh::kSlots) * Sh::kTileBytes;
#pragma unroll
        for (int e = 0; e < DP / 16; e++) {
            const uint32_t at = (e >> 2) * Sh::kBlock + (e & 3) * 32;
            tc::mma_f16(b.tmem + t * 128, tc::sw128_desc(q + t * Sh::kTileBytes + at), tc::sw128_desc(k + at), kScores,
                        e > 0);
        }
        tc::mma_commit(&b.s_full[t]);
    };
    auto output = [&](int t, int j) {
        const uint32_t v = kv + ((2 * j + 1) % Sh::kSlots) * Sh::kTileBytes;
#pragma unroll
        for (int e = 0; e < kTilePos / 16; e++)
            tc::mma_f16_ta(b.tmem + 256 + t * DP, b.tmem + t * 128 + e * 8, tc::sw128_mn_desc(v + e * 2048, Sh::kBlock),
                           kOut, j > 0 || e > 0);
    };
    auto ready = [&](int i) { return tc::mbar_wait(&b.full[i % Sh::kSlots], (i / Sh::kSlots) & 1, &b.aborted); };
    if (!tc::mbar_wait(&b.q_full, 0, &b.aborted) || !ready(0))
        return;
    tc::fence_after_sync();
    scores(0, 0);
    if (two)
        scores(1, 0);
    tc::mma_commit(&b.empty[0]);
    for (int j = 0; j < tiles; j++) {
        for (int t = 0; t < (two ? 2 : 1); t++) {
            if (t == 0 && !ready(2 * j + 1))
                return;
            if (!tc::mbar_wait(&b.p_ready[t], j & 1, &b.aborted))
                return;
            tc::fence_after_sync();
            output(t, j);
            if (t == (two ? 1 : 0))
                tc::mma_commit(&b.empty[(2 * j + 1) % Sh::kSlots]);
            if (j + 1 < tiles) {
                if (t == 0 && !ready(2 * j + 2))
                    return;
                scores(t, j + 1);
                if (t == (two ? 1 : 0))
                    tc::mma_commit(&b.empty[(2 * j + 2) % Sh::kSlots]);
            } else {
                tc::mma_commit(&b.o_full[t]);
            }
        }
    }
}

template <typename T, int DP>
__device__ void tile_softmax(const AttnParams &p, const AttnWork &w, TileBars &b, int tiles)
{
    const int t = threadIdx.x >> 7, tid = threadIdx.x & 127, r = t * 128 + tid;
    const uint32_t lanes = b.tmem + ((uint32_t)(tid & ~31) << 16);
    const uint32_t s_at = lanes + t * 128, o_at = lanes + 256 + t * DP;
    const int row = w.row0 + r, token = row / p.group;
    const bool mine = r < w.rows;
    // a row past the last sees everything: it needs no mask, and nothing of it is written
    const int hi = mine ? min(seen_hi(w.seq, p.causal, token), w.hi) : 0x7fffffff;
    const int lo = mine ? seen_lo(seen_hi(w.seq, p.causal, token), p.window) : 0;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < tiles; j++) {
        if (!tc::mbar_wait(&b.s_full[t], j & 1, &b.aborted))
            return;
        tc::fence_after_sync();
        uint32_t s[128];
        const int at = w.lo + j * kTilePos;
        const bool plain = __all_sync(0xffffffffu, at >= lo && at + kTilePos <= hi);
        auto load = [&] {
#pragma unroll
            for (int c = 0; c < 4; c++)
                tc::tmem_ld32_async(s_at + c * 32, s + c * 32);
#pragma unroll
            for (int c = 0; c < 4; c++)
                tc::tmem_ld_wait(s + c * 32);
            if (!plain) {
#pragma unroll
                for (int i = 0; i < kTilePos; i++)
                    s[i] = at + i >= lo && at + i < hi ? s[i] : 0xff800000u;
            }
        };
        load();
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kTilePos; i++)
            top[i & 3] = fmaxf(top[i & 3], __uint_as_float(s[i]));
        const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2;
        if (__any_sync(0xffffffffu, now > m + kTileSlack)) {
            // also from -infinity; the output of the tiles before is complete: the scores' MMA came after it
            const float next = fmaxf(m, now), f = next == -INFINITY ? 1.f : exp2_approx(m - next);
            m = next;
            l *= f;
            if (j > 0) {
#pragma unroll
                for (int c = 0; c < DP; c += 32) {
                    float o[32];
                    tc::tmem_ld32(o_at + c, o);
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        o[i] *= f;
                    tc::tmem_st32(o_at + c, o);
                }
                load();  // the scores' registers held the output
            }
        }
        const float base = m == -INFINITY ? 0.f : m;
        const float2 scale = make_float2(p.scale_log2, p.scale_log2), off = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; c++) {
            float packed[32];
#pragma unroll
            for (int i = 0; i < 32; i++) {
                const int k = c * 64 + 2 * i;
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale, off);
                const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                packed[i] = __uint_as_float(pack2<T>(e.x, e.y));
            }
            tc::tmem_st32(s_at + c * 32, packed);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        tc::mbar_arrive(&b.p_ready[t]);
    }
    float inv = 0.f, lse = -INFINITY;
    if (l > 0.f) {
        inv = 1.f / l;
        lse = m + log2f(l);
    }
    if (tiles > 0) {
        if (!tc::mbar_wait(&b.o_full[t], 0, &b.aborted))
            return;
        tc::fence_after_sync();
    }
    const int heads = p.cache.heads * p.group, h = w.head * p.group + row - token * p.group;
    const int64_t part = ((int64_t)w.split * p.batch.n + w.seq.first + token) * heads + h;
    if (mine) {
        if (!w.whole)
            p.part_lse[part] = lse;
        else if (p.lse)
            p.lse[(w.seq.first + token) * heads + h] = lse * kLn2;
    }
#pragma unroll
    for (int c = 0; c < DP; c += 32) {
        float o[32];
        __syncwarp();
        if (tiles > 0)
            tc::tmem_ld32(o_at + c, o);
#pragma unroll
        for (int i = 0; i < 32; i++)
            o[i] = inv > 0.f ? o[i] * inv : 0.f;
        if (mine && w.whole) {
            T *out = p.out.row<T>(w.seq.first + token, h) + c;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
                if (c + i < p.d)
                    *reinterpret_cast<uint4 *>(out + i) =
                        make_uint4(pack2<T>(o[i], o[i + 1]), pack2<T>(o[i + 2], o[i + 3]), pack2<T>(o[i + 4], o[i + 5]),
                                   pack2<T>(o[i + 6], o[i + 7]));
        } else if (mine) {
            float *out = p.part_o + part * p.d + c;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                if (c + i < p.d)
                    *reinterpret_cast<float4 *>(out + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
    }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kTileThreads, 1)
kv_attn_tile_kernel(const __grid_constant__ AttnParams p)
{
    using Sh = TileShape<DP>;
    extern __shared__ uint8_t raw[];
    __shared__ TileBars b;
    uint8_t *sq = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023), *ring = sq + 2 * Sh::kTileBytes;
    const int warp = threadIdx.x >> 5;
    AttnWork w;
    if (!attn_work(p, blockIdx.x, w))
        return;
    const int tiles = (w.hi - w.lo + kTilePos - 1) / kTilePos;  // 0: rows that see nothing
    const bool two = w.rows > 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kSlots; i++) {
            tc::mbar_init(&b.full[i], kCopyThreads);
            tc::mbar_init(&b.empty[i], 1);
        }
        tc::mbar_init(&b.q_full, kCopyThreads);
        tc::mbar_init(&b.drained, 1);
        for (int t = 0; t < 2; t++) {
            tc::mbar_init(&b.s_full[t], 1);
            tc::mbar_init(&b.p_ready[t], 128);
            tc::mbar_init(&b.o_full[t], 1);
        }
        b.aborted = 0;
        tc::mbar_init_fence();
    }
    if (warp == 10)
        tc::tmem_alloc<512>(&b.tmem);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp < 8) {
        if (warp < 4 || two)
            tile_softmax<T, DP>(p, w, b, tiles);
    } else if (warp < 10) {
        if (tiles > 0)
            tile_copy<T, DP>(p, w, sq, ring, b, tiles);
    } else if ((threadIdx.x & 31) == 0 && tiles > 0) {
        tile_mma<T, DP>(sq, ring, b, tiles, two);
        if (b.aborted) {  // no MMA may be in flight when the memory is given back
            int never = 0;
            tc::mma_commit(&b.drained);
            tc::mbar_wait(&b.drained, 0, &never);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (threadIdx.x == 0 && *reinterpret_cast<volatile int *>(&b.aborted))
        raise_flag(p.err, DLRM_FLAG_WAIT_TIMEOUT);
    if (warp == 10)
        tc::tmem_free<512>(b.tmem);
}

template <typename T, int DP>
static int launch_tile(const AttnParams &p, int64_t ctas, cudaStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)kv_attn_tile_kernel<T, DP>, TileShape<DP>::kSmem, &done);
    if (s != DLRM_OK)
        return s;
    kv_attn_tile_kernel<T, DP><<<(unsigned)ctas, kTileThreads, TileShape<DP>::kSmem, st>>>(p);
    count_launch(st);
    return DLRM_OK;
}

int launch_kv_attn_tile(const AttnParams &p, int dtype, int64_t ctas, cudaStream_t st)
{
    if (dtype == DLRM_F16)
        return p.d <= 64 ? launch_tile<__half, 64>(p, ctas, st) : launch_tile<__half, 128>(p, ctas, st);
    return p.d <= 64 ? launch_tile<__nv_bfloat16, 64>(p, ctas, st) : launch_tile<__nv_bfloat16, 128>(p, ctas, st);
}

}  // namespace dlrm
