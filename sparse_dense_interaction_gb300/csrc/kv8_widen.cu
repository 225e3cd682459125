// The part of a cache in 8 bits that a batch sees, as a 16-bit cache in the workspace.
//
// Long chunks read every key and value again for each tile of their rows, and
// converting them each time costs the tiles a third of their time.  So for such batches they are
// converted once, and the 16-bit cache's tiles do the rest.  Values become fp16 relative to the largest power of
// their page of the copy, which the tiles apply to their weights; fp16 weights have as many bits as everywhere else over
// this cache.  Keys are of the queries' type: so in fp16, which the tiles apply to their scores; in bf16, which holds
// every code times its power, as they are.  (Values in bf16 would make the weights bf16: 369 us for the sequences below,
// but 1.35 times the error against 64 bits.)  Memory bounds the conversion (a byte read, two written, which mostly stay
// in L2).  With a cold L2 4 sequences of 2048 new on 8192, 16 heads on 4 of 128, take 384 us in bf16 and 392 in fp16,
// on a 16-bit cache 345 and 349.
#include <type_traits>

#include "kv8.cuh"

namespace dlrm {

constexpr int kWidenThreads = 256, kWidenPage = 128;

struct WidenParams {
    AttnParams p;
    char *k, *v;      // [sequence * pages + page][head][kWidenPage][d]; keys bf16 or fp16, values fp16
    int32_t *table;   // [sequence][pages]
    uint16_t *refs;   // [sequence][pages][heads]
    int pages;        // of a sequence
    FastDiv chunks, heads;  // 8 codes of a row; heads
};

// 8 codes, times 2^(e - 127), or for fp16 2^(e - ref + 7).  (16 a lane, in two stores that each write half sectors: 366
// us for the 4 sequences above instead of 363.)
template <typename T>
__device__ __forceinline__ void widen8(const char *from, uint32_t e, int ref, char *to)
{
    const uint2 c = *reinterpret_cast<const uint2 *>(from);
    const uint32_t in[2] = {c.x, c.y};
    const float power = exp_power(e);
    const uint32_t relative = relative_power((int)e - ref);
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint32_t h[2];
        decode4(in[i], h[0], h[1]);
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if constexpr (std::is_same<T, __half>::value) {
                x[2 * i + k] = hmul2(h[k], relative);
            } else {
                const float2 y = unpack2<__half>(h[k]);
                x[2 * i + k] = pack2<T>(y.x * power, y.y * power);
            }
        }
    }
    *reinterpret_cast<uint4 *>(to) = make_uint4(x[0], x[1], x[2], x[3]);
}

// A CTA per sequence, page of the copy and head.
template <typename T>
__global__ void __launch_bounds__(kWidenThreads)
kv8_widen_kernel(const __grid_constant__ WidenParams w)
{
    const AttnParams &p = w.p;
    __shared__ int64_t row_codes[kWidenPage];  // -1: a row of zeros
    __shared__ uint8_t row_exps[2][kWidenPage];
    __shared__ uint32_t warp_refs[kWidenThreads / 32];
    const uint32_t number = w.heads.div(blockIdx.x);  // of the page
    const int head = (int)(blockIdx.x - number * w.heads.d), page = (int)(number % (uint32_t)w.pages);
    const int64_t s = number / (uint32_t)w.pages;
    if (threadIdx.x == 0 && head == 0)
        w.table[number] = (int32_t)number;
    Sequence q;
    if (!read_sequence(p.batch, s, p.max_new, p.max_len, q, nullptr) || q.count == 0 || !attn_takes(p, q))
        return;
    const int start = page * kWidenPage, hi = min(seen_hi(q, p.causal, q.count - 1), start + kWidenPage);
    const int lo = max(seen_lo(seen_hi(q, p.causal, 0), p.window), start);
    if (lo >= hi)
        return;
    const int r = threadIdx.x;
    uint32_t k_exp = 0, v_exp = 0;
    if (r < hi - lo) {
        const uint32_t at = lo + r, n = p.cache.page.div(at), slot = at - n * p.cache.page.d;
        const uint32_t id = (uint32_t)p.batch.table[s * p.batch.table_stride + n];
        row_codes[r] = -1;
        if (id < p.cache.pages) {
            row_codes[r] = id * p.cache.page_stride + slot * p.cache.slot_stride + head * p.cache.head_stride;
            const int64_t x = exp_offset(p.exp, id, slot, head);
            row_exps[0][r] = k_exp = p.exp.k[x];
            row_exps[1][r] = v_exp = p.exp.v[x];
        } else {
            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
        }
    }
    k_exp = __reduce_max_sync(0xffffffffu, k_exp);
    v_exp = __reduce_max_sync(0xffffffffu, v_exp);
    if ((r & 31) == 0)
        warp_refs[r / 32] = k_exp | v_exp << 16;
    __syncthreads();
    int k_ref = 0, v_ref = 0;
#pragma unroll
    for (int i = 0; i < kWidenPage / 32; i++) {
        k_ref = max(k_ref, (int)(warp_refs[i] & 0xffff));
        v_ref = max(v_ref, (int)(warp_refs[i] >> 16));
    }
    if (r == 0)
        w.refs[blockIdx.x] = (uint16_t)(k_ref | v_ref << 8);
    const int per_row = p.d / 8, all = (hi - lo) * per_row;
    const int64_t base = ((int64_t)blockIdx.x * kWidenPage + lo - start) * p.d * 2;
#pragma unroll 4
    for (int i = threadIdx.x; i < all; i += kWidenThreads) {
        const int x = (int)w.chunks.div((uint32_t)i), c = i - x * per_row;
        const int64_t from = row_codes[x] + c * 8, to = base + i * 16;
        if (row_codes[x] >= 0) {
            widen8<T>(p.cache.k + from, row_exps[0][x], k_ref, w.k + to);
            widen8<__half>(p.cache.v + from, row_exps[1][x], v_ref, w.v + to);
        } else {
            *reinterpret_cast<uint4 *>(w.k + to) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(w.v + to) = make_uint4(0, 0, 0, 0);
        }
    }
}

// Bytes of the copy, 0 where there is none.  It pays where tiles of rows read a key and value often, from 6 tiles of
// 256 rows on with heads above 64 and from 8 on below.  Converted once and by every tile, us, cold L2, 16 heads on 4 of
// 128, bf16 and fp16: 4 sequences of 2048 new on 8192 each 382 and 470, 394 and 461; on up to 8192 201 and 236, 205 and
// 232; 16 of 512 on up to 4000 109 and 113, 110 and 109; of 400 91 and 89, 93 and 85, on 4000 each 220 and 230, 224 and
// 225; 16 of 600 on up to 4000, heads of 64, 113 and 113, 115 and 113.  (Fewer rows, warm: 16 of 256 on up to 8192 154 and
// 142; 64 of 500 on up to 2000, 8 heads of 64, 131 and 113.)  It takes four times the bytes of the codes up to max_len,
// which may be far above the lengths: at most kWidenMost.
constexpr int64_t kWidenMost = (int64_t)2 << 30;

size_t widen_workspace(int64_t S, int heads, int group, int d, int64_t max_new, int64_t max_len)
{
    const int64_t pages = (max_len + kWidenPage - 1) / kWidenPage;
    if (max_new * group < (d > 64 ? 1536 : 2048) || d > 128 || d % 16 != 0 || pages == 0 || S == 0 ||
        pages > kWidenMost / (4 * kWidenPage * S * heads * d))
        return 0;
    return (size_t)(4 * kWidenPage * S * pages * heads * d + (S * pages * (4 + 2 * heads) + 255) / 256 * 256);
}

// Converts, and turns the parameters to the copy; the workspace begins with it.
int launch_widen(AttnParams &p, int dtype, void *workspace, cudaStream_t st)
{
    WidenParams w;
    const int64_t pages = (p.max_len + kWidenPage - 1) / kWidenPage, all = p.batch.S * pages;
    const int64_t bytes = 2 * all * kWidenPage * p.cache.heads * p.d;
    w.p = p;
    w.k = static_cast<char *>(workspace);
    w.v = w.k + bytes;
    w.table = reinterpret_cast<int32_t *>(w.v + bytes);
    w.refs = reinterpret_cast<uint16_t *>(w.table + all);
    w.pages = (int)pages;
    w.chunks = FastDiv::make((uint32_t)p.d / 8);
    w.heads = FastDiv::make((uint32_t)p.cache.heads);
    const unsigned ctas = (unsigned)(all * p.cache.heads);
    if (dtype == DLRM_F16)
        kv8_widen_kernel<__half><<<ctas, kWidenThreads, 0, st>>>(w);
    else
        kv8_widen_kernel<__nv_bfloat16><<<ctas, kWidenThreads, 0, st>>>(w);
    count_launch(st);
    const int64_t row = p.d, head = kWidenPage * row;
    p.cache = CacheView{w.k, w.v, head * p.cache.heads, row, head, (uint32_t)all, FastDiv::make(kWidenPage), p.cache.heads};
    p.batch.table = w.table;
    p.batch.table_stride = pages;
    p.batch.capacity = p.batch.capacity < pages * kWidenPage ? p.batch.capacity : pages * kWidenPage;
    p.exp = ExpView{};
    p.refs = w.refs;
    return launch_status();
}

}  // namespace dlrm
