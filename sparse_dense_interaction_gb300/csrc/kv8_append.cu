// Appends a step's keys and values to the cache in 8 bits.
//
// A block (some consecutive slots of a page, one head, keys or values) has one
// exponent, so what enters it is encoded together: its largest magnitude first,
// then the codes.  An item is such a block; it belongs to the first new token
// that enters it, and a warp takes it.  Where the block already holds older
// tokens its exponent only grows, and only then are their codes read and
// rounded again; most steps touch no older code.
//
// Memory bounds long prompts: rows are read once into registers, a chunk of
// 8 elements each, as they lie, and written as a byte an element.  98000 new tokens of 48
// users (8 heads of 128 bf16 elements): 98 us, 554 MB, 5.6 TB/s, 0.84 of a plain copy.
// That is with blocks of 16 rows, all that a warp's registers hold (fp32: 8 rows); of larger ones it reads the rest
// twice.  With a cold L2, blocks of 8, 16, 32, 64 and 128: 130, 101, 148, 193 and 253 us; 24 of these users in
// fp32 (490 MB) 91, 121, 148, 183 and 185.  Rows off the vector path (heads of 68) 224.
// One event of each of 2048 users moves 1.6 MB: 12 us from call to call, 9.7 in a graph: a
// chain of dependent reads (offsets, table, exponent, codes) in each of 1024 CTAs, of which 608 run at once.
#include "kv8.cuh"

namespace dlrm {

constexpr int kApWarps = 8, kApMaxSlice = 32;

struct Append8Params {
    HeadsView k, v;
    BatchView batch;
    CacheView cache;
    ExpView exp;
    int d;
    int slice;       // tokens whose blocks a CTA looks after
    FastDiv chunks;  // divides by the chunks of a row
    int32_t *err;
};

// A block's first new token, and what of the block is new and older.
struct Append8Item {
    int64_t token;
    int32_t page;
    int32_t slot;   // of the token in its page
    int32_t fresh;  // new tokens in the block
    int32_t older;  // slots before the token's in the block, all filled
};

// 8 elements as they lie; read once.
template <typename T>
struct Append8Chunk {
    static constexpr int kWords = sizeof(T) * 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; i++)
            w[i] = 0;
    }
    __device__ __forceinline__ void load(const T *src)
    {
#pragma unroll
        for (int i = 0; i < kWords / 4; i++) {
            const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
    __device__ __forceinline__ float2 pair(int i) const  // elements 2i, 2i + 1
    {
        if constexpr (sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else
            return unpack2<T>(w[i]);
    }
    // The largest magnitude's bits, as an unsigned number of T's width, in each half or whole of the result and
    // `top`: magnitudes are ordered like their bits.
    __device__ __forceinline__ uint32_t largest(uint32_t top) const
    {
#pragma unroll
        for (int i = 0; i < kWords; i++)
            top = sizeof(T) == 4 ? max(top, w[i] & 0x7fffffffu) : __vmaxu2(top, w[i] & 0x7fff7fffu);
        return top;
    }
};

// The warp's largest magnitude, of what largest() left in every lane; infinity or NaN if any is.
template <typename T>
__device__ __forceinline__ float largest_of_warp(uint32_t top)
{
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
    else
        return unpack2<T>(__reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16))).x;
}

// |x| where x is finite, else 0: what is not finite does not count for the exponent.
__device__ __forceinline__ float finite_size(float x)
{
    const float a = fabsf(x);
    return a <= 3.4028234663852886e38f ? a : 0.f;
}

// The blocks that the tokens first .. first + slice of the batch begin to fill, by one warp; returns how many.
__device__ __forceinline__ int append8_items(const Append8Params &p, int64_t i0, Append8Item *items, int32_t *owner)
{
    const int lane = threadIdx.x & 31;
    const int64_t i1 = min(i0 + p.slice, p.batch.n);
    owner[lane] = -1;
    __syncwarp();
    // the slice's sequences, 32 at a time, each marks its tokens
    int64_t s = find_sequence(p.batch, i0);
    for (bool more = s >= 0; more; s += 32) {
        const bool there = s + lane < p.batch.S;
        const int64_t from = there ? p.batch.offsets[s + lane] : i1, to = there ? p.batch.offsets[s + lane + 1] : i1;
        for (int64_t t = max(from, i0); t < min(to, i1); t++)
            owner[t - i0] = (int)(s + lane);
        more = __all_sync(0xffffffffu, there && from < i1);
    }
    __syncwarp();
    const int64_t token = i0 + lane;
    const int mine = lane < i1 - i0 ? owner[lane] : -1;
    Append8Item it = {};
    bool first = false;
    Sequence q;
    if (mine >= 0 && read_sequence(p.batch, mine, p.batch.n, p.batch.capacity, q, p.err) && q.has(token) &&
        q.count <= q.length) {
        const int at = q.length - q.count + (int)(token - q.first), block = (int)p.exp.block.d;
        const uint32_t number = p.cache.page.div((uint32_t)at);
        it.token = token;
        it.slot = at - (int)(number * p.cache.page.d);
        it.older = it.slot - (int)p.exp.block.div((uint32_t)it.slot) * block;
        it.fresh = min(block - it.older, (int)(q.first + q.count - token));
        first = token == q.first || it.older == 0;
        if (first) {
            it.page = p.batch.table[mine * p.batch.table_stride + number];
            if ((uint32_t)it.page >= p.cache.pages) {
                raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
                first = false;
            }
        }
    }
    const uint32_t all = __ballot_sync(0xffffffffu, first);
    if (first)
        items[__popc(all & ((1u << lane) - 1))] = it;
    return __popc(all);
}

// One block of one head, by a warp.  kVec: chunks of 8 elements that lie on
// 16 bytes (fp32 too) and whose codes lie on 8; else element by element.
template <typename T, bool kVec>
__device__ __forceinline__ void append8_block(const Append8Params &p, const Append8Item &it, int head, bool value)
{
    constexpr int kHold = kVec ? (sizeof(T) == 4 ? 4 : 8) : 0;  // chunks of a lane that stay in registers
    const int lane = threadIdx.x & 31;
    const HeadsView &in = value ? p.v : p.k;
    uint8_t *exps = (value ? p.exp.v : p.exp.k) + exp_offset(p.exp, it.page, it.slot, head);
    char *codes = (value ? p.cache.v : p.cache.k) + it.page * p.cache.page_stride + head * p.cache.head_stride;
    const int before = it.older > 0 ? *exps : 0;
    const int per_row = kVec ? p.d / 8 : p.d, all = it.fresh * per_row;
    const T *rows = in.row<T>(it.token, head);
    // where chunk (or element) c lies, and its codes
    auto source = [&](int c) {
        const int r = (int)p.chunks.div((uint32_t)c);
        return rows + r * in.ts + (c - r * per_row) * (kVec ? 8 : 1);
    };
    auto target = [&](int c) {
        const int r = (int)p.chunks.div((uint32_t)c);
        return codes + (it.slot + r) * p.cache.slot_stride + (c - r * per_row) * (kVec ? 8 : 1);
    };
    auto size_of = [&](int c) {  // the slow way, past what is not finite
        float top = 0.f;
        if constexpr (kVec) {
            Append8Chunk<T> x;
            x.load(source(c));
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 y = x.pair(i);
                top = fmaxf(top, fmaxf(finite_size(y.x), finite_size(y.y)));
            }
        } else {
            top = finite_size(to_f32(*source(c)));
        }
        return top;
    };
    Append8Chunk<T> held[kHold > 0 ? kHold : 1];
    float top = 0.f;
    if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < kHold; i++) {
            held[i].clear();
            if (i * 32 + lane < all)
                held[i].load(source(i * 32 + lane));
        }
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < kHold; i++)
            bits = held[i].largest(bits);
        for (int c = kHold * 32 + lane; c < all; c += 32) {
            Append8Chunk<T> x;
            x.load(source(c));
            bits = x.largest(bits);
        }
        top = largest_of_warp<T>(bits);
    }
    if (!kVec || !(top <= 3.4028234663852886e38f)) {
        top = 0.f;
        for (int c = lane; c < all; c += 32)
            top = fmaxf(top, size_of(c));
        top = warp_max(top);
    }
    const int fresh = exponent_of(top), now = fresh > before ? fresh : before;
    const float scale = encode_power(now);
    auto write8 = [&](int c, const Append8Chunk<T> &x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 y = x.pair(i);
            w[i] = encode2(y.x * scale, y.y * scale);
        }
        *reinterpret_cast<uint2 *>(target(c)) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    };
#pragma unroll
    for (int i = 0; i < kHold; i++)
        if (i * 32 + lane < all)
            write8(i * 32 + lane, held[i]);
    for (int c = kHold * 32 + lane; c < all; c += 32) {
        if constexpr (kVec) {
            Append8Chunk<T> x;
            x.load(source(c));
            write8(c, x);
        } else {
            *target(c) = (char)encode2(to_f32(*source(c)) * scale, 0.f);
        }
    }
    if (it.older > 0 && now > before) {  // older codes under the larger power; below 2^-120 all of them are zeros
        const float down = __uint_as_float((uint32_t)(127 + max(before - now, -120)) << 23);
        for (int c = lane; c < it.older * p.d; c += 32) {
            const int r = c / p.d;
            char *at = codes + (it.slot - it.older + r) * p.cache.slot_stride + (c - r * p.d);
            *at = (char)encode2(decode2_f32((uint8_t)*at).x * down, 0.f);
        }
    }
    __syncwarp();  // every lane has read the exponent
    if (lane == 0)
        *exps = (uint8_t)now;
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kApWarps * 32, 4)
kv8_append_kernel(const __grid_constant__ Append8Params p)
{
    __shared__ Append8Item items[kApMaxSlice];
    __shared__ int32_t owner[32];
    __shared__ int found;
    const int warp = threadIdx.x >> 5;
    check_sequences(p.batch, (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x, p.err);
    const int64_t slices = (p.batch.n + p.slice - 1) / p.slice;
    for (int64_t i = blockIdx.x; i < slices; i += gridDim.x) {
        __syncthreads();
        if (warp == 0) {
            const int n = append8_items(p, i * p.slice, items, owner);
            if (threadIdx.x == 0)
                found = n;
        }
        __syncthreads();
        const int heads = p.cache.heads, all = found * heads * 2;
        for (int x = warp; x < all; x += kApWarps) {
            const int which = x / (2 * heads), part = x - which * 2 * heads;
            append8_block<T, kVec>(p, items[which], part >> 1, part & 1);
        }
    }
}

template <typename T>
static int launch_append8(Append8Params &p, cudaStream_t st)
{
    auto even = [](const HeadsView &h) {
        return reinterpret_cast<uintptr_t>(h.ptr) % 16 == 0 && h.ts * sizeof(T) % 16 == 0 && h.hs * sizeof(T) % 16 == 0;
    };
    const CacheView &c = p.cache;
    const bool vec = p.d % 8 == 0 && even(p.k) && even(p.v) && reinterpret_cast<uintptr_t>(c.k) % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(c.v) % 8 == 0 && c.page_stride % 8 == 0 && c.slot_stride % 8 == 0 &&
                     c.head_stride % 8 == 0;
    p.chunks = FastDiv::make((uint32_t)(vec ? p.d / 8 : p.d));
    const int64_t places = 4 * 152;
    p.slice = kApMaxSlice;
    while (p.slice > 1 && (p.batch.n + p.slice - 1) / p.slice < places)
        p.slice /= 2;
    const int64_t slices = (p.batch.n + p.slice - 1) / p.slice;
    const unsigned grid = (unsigned)(slices < 0x7fffffff ? slices : 0x7fffffff);
    if (vec)
        kv8_append_kernel<T, true><<<grid, kApWarps * 32, 0, st>>>(p);
    else
        kv8_append_kernel<T, false><<<grid, kApWarps * 32, 0, st>>>(p);
    count_launch(st);
    return launch_status();
}

int launch_kv8_append(const HeadsView &k, const HeadsView &v, const BatchView &batch, const CacheView &cache,
                      const ExpView &exp, int d, int dtype, int32_t *err, cudaStream_t st)
{
    Append8Params p = {k, v, batch, cache, exp, d, 0, {}, err};
    if (dtype == DLRM_F32)
        return launch_append8<float>(p, st);
    if (dtype == DLRM_F16)
        return launch_append8<__half>(p, st);
    return launch_append8<__nv_bfloat16>(p, st);
}

}  // namespace dlrm
