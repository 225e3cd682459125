// Shared by the kernels over rows of heads: the scalar helpers and the vector
// path's row layout.
//
// Vector path: GL lanes (4, 8, 16 or 32) hold a row of up to 8 GL elements, 8
// a lane in two pieces of 4, chosen so that the elements that turn together are
// one lane's.  A warp takes a chunk of the heads of `run` tokens (32 at most), a
// row for each lane group at a time, of one token or, where a token has at most
// half as many heads as there are groups, of 2, 4 or 8; such slots stream through a
// ring in shared memory by asynchronous copies, several ahead of the one that is
// computed: a lane reads back what it copied itself.  What a token needs beside
// its rows (its angles' row, where its rows go) one lane finds out for each
// token before the first.
#pragma once

#include "history.cuh"
#include "tc.cuh"

namespace dlrm {

constexpr int kWarps = 8;      // of a CTA

constexpr int kSlots = 4;  // of a chunk of a token's heads: a row for each lane group
constexpr int kMaxRun = 32;

// The ring of a warp: slots of kIn rows for each lane group, and the angles of
// their tokens (`fold` to a slot).
template <typename T, int GL, int kIn>
struct Ring {
    static constexpr int kPiece = 4 * sizeof(T), kSlot = kIn * 2 * 32 * kPiece, kAngles = GL * 32;
    static constexpr int kDepth = kSlot <= 512 ? 6 : (kSlot <= 1024 ? 5 : 3);  // deeper rings measured no faster
    __host__ __device__ static constexpr int bytes(int fold) { return kDepth * (kSlot + kAngles * fold); }
};

// The rope row of a position, or null with the flag raised where it is
// outside the table.
__device__ __forceinline__ const float *rope_row(const RopeView &rope, int64_t position, int32_t *err)
{
    if (position < 0 || position >= rope.length) {
        raise_flag(err, DLRM_FLAG_INDEX_OOB);
        return nullptr;
    }
    return rope.table + position * rope.rot;
}

// Four elements as they lie, and as two pairs of floats.
template <typename T>
struct Piece {
    using Raw = uint2;
    __device__ __forceinline__ static void widen(const Raw &r, float2 *v)
    {
        v[0] = pair(r.x);
        v[1] = pair(r.y);
    }
    __device__ __forceinline__ static Raw narrow(const float2 *v)
    {
        return make_uint2(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y));
    }
    __device__ __forceinline__ static float2 pair(uint32_t w);
};
template <>
__device__ __forceinline__ float2 Piece<__half>::pair(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
template <>
__device__ __forceinline__ float2 Piece<__nv_bfloat16>::pair(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
struct Piece<float> {
    using Raw = float4;
    __device__ __forceinline__ static void widen(const Raw &r, float2 *v)
    {
        v[0] = make_float2(r.x, r.y);
        v[1] = make_float2(r.z, r.w);
    }
    __device__ __forceinline__ static Raw narrow(const float2 *v) { return make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
};

// What a lane holds of every row.
template <int GL>
struct RowLane {
    int e0, e1;         // first elements of its two pieces
    int group;          // its lane group's number in the warp
    bool active;        // it holds elements at all
    int angle;          // column of its first angle, -1: its elements are not turned
    static constexpr int kGroups = 32 / GL;

    __device__ __forceinline__ RowLane(int d, const RopeView &rope)
    {
        const int lane = threadIdx.x & 31, l = lane % GL;
        group = lane / GL;
        active = 8 * l < d;
        angle = rope.table && 8 * l < rope.rot ? 4 * l : -1;
        const bool apart = angle >= 0 && !rope.interleaved;
        e0 = apart ? 4 * l : 8 * l;
        e1 = apart ? (rope.rot >> 1) + 4 * l : 8 * l + 4;
    }
};

// A lane's 8 elements of a row: the first and second elements of its four
// pairs, two pairs in a float2 (the arithmetic is two floats wide).
template <typename T, bool kInterleaved>
__device__ __forceinline__ void widen_row(const typename Piece<T>::Raw *r, float2 *a, float2 *b)
{
    float2 x[2], y[2];
    Piece<T>::widen(r[0], x);
    Piece<T>::widen(r[1], y);
    a[0] = kInterleaved ? make_float2(x[0].x, x[1].x) : x[0];
    a[1] = kInterleaved ? make_float2(y[0].x, y[1].x) : x[1];
    b[0] = kInterleaved ? make_float2(x[0].y, x[1].y) : y[0];
    b[1] = kInterleaved ? make_float2(y[0].y, y[1].y) : y[1];
}

template <typename T, bool kInterleaved>
__device__ __forceinline__ void narrow_row(const float2 *a, const float2 *b, typename Piece<T>::Raw *r)
{
    float2 x[2], y[2];
    x[0] = kInterleaved ? make_float2(a[0].x, b[0].x) : a[0];
    x[1] = kInterleaved ? make_float2(a[0].y, b[0].y) : a[1];
    y[0] = kInterleaved ? make_float2(a[1].x, b[1].x) : b[0];
    y[1] = kInterleaved ? make_float2(a[1].y, b[1].y) : b[1];
    r[0] = Piece<T>::narrow(x);
    r[1] = Piece<T>::narrow(y);
}

// A piece global -> shared, asynchronously; zeros where there is none.
template <int kBytes>
__device__ __forceinline__ void copy_piece(void *to, const void *from, bool there)
{
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from), "r"(there ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(tc::smem_u32(to)), "l"(from), "r"(there ? 8 : 0)
                     : "memory");
}

// Copies a lane's pieces of a row (`base`: an address that may be named where
// there is none) to its place in a slot.
template <typename T, int GL>
__device__ __forceinline__ void copy_row(uint8_t *slot, const T *row, const void *base, bool there, const RowLane<GL> &at)
{
    constexpr int P = 4 * sizeof(T);
    copy_piece<P>(slot, there ? row + at.e0 : base, there);
    copy_piece<P>(slot + 32 * P, there ? row + at.e1 : base, there);
}

template <typename T>
__device__ __forceinline__ void read_row(const uint8_t *slot, typename Piece<T>::Raw *x)
{
    using Raw = typename Piece<T>::Raw;
    x[0] = *reinterpret_cast<const Raw *>(slot);
    x[1] = *reinterpret_cast<const Raw *>(slot + 32 * sizeof(Raw));
}

template <typename T, int GL>
__device__ __forceinline__ void store_row(T *row, bool there, const RowLane<GL> &at, const typename Piece<T>::Raw *x)
{
    using Raw = typename Piece<T>::Raw;
    if (there) {
        *reinterpret_cast<Raw *>(row + at.e0) = x[0];
        *reinterpret_cast<Raw *>(row + at.e1) = x[1];
    }
}

// Cosines and sines of a lane's four pairs; 1 and 0 where nothing turns.
struct Angles {
    float4 c, s;

    __device__ __forceinline__ Angles(const float4 *staged, bool turned)
    {
        c = make_float4(1.f, 1.f, 1.f, 1.f);
        s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turned) {
            c = staged[0];
            s = staged[1];
        }
    }
};

// Copies a token's angles to shared memory: 8 floats for each lane of a group,
// by the token's first group (`mine`).
template <int GL>
__device__ __forceinline__ void copy_angles(uint8_t *to, const float *row, int half, const RowLane<GL> &at, bool mine)
{
    if (mine && at.angle >= 0 && row) {
        copy_piece<16>(to + threadIdx.x % GL * 32, row + at.angle, true);
        copy_piece<16>(to + threadIdx.x % GL * 32 + 16, row + half + at.angle, true);
    }
}

// The heads of one side of a call (queries, keys, values) and what is done to
// them.  A kernel's parameters hold an array of these and a CTA works on one:
// indexed where they lie, in constant memory, they cost no registers.
struct NormSide {
    HeadsView x, dy, out;  // dy: of the gradient alone
    const float *w;
    int chunks;            // of a token's heads; the CTAs of chunk blockIdx.y
    int fold;              // tokens of a slot

    // 195312 tokens of 4 query heads and one key head of 64 bf16 elements: 81 us, 107 with one token a slot; 488281 of
    // one and one: 108 and 243
    void lay_out(int groups)
    {
        chunks = (x.heads + kSlots * groups - 1) / (kSlots * groups);
        for (fold = 1; x.heads > 0 && x.heads * fold * 2 <= groups;)
            fold *= 2;
    }
};

// Where a lane group works: its token of a slot, the first head of its chunk
// and its own, the slots of a token.
struct Fold {
    int token, head, slots;
    bool first;  // the token's first group

    __device__ __forceinline__ Fold(const NormSide &side, int chunk, int group, int groups)
    {
        const int per = groups / side.fold, base = chunk * kSlots * groups;
        token = group / per;
        head = base + group % per;
        first = group % per == 0;
        slots = min(kSlots, (side.x.heads - base + groups - 1) / groups);
    }
};

// The side of chunk `chunk`, which becomes the chunk's number within it.
__device__ __forceinline__ int side_of(const NormSide *side, int &chunk)
{
    int s = 0;
    while (chunk >= side[s].chunks)
        chunk -= side[s++].chunks;
    return s;
}

// The weight in shared memory, 8 floats a lane in the order of its pairs; ones
// where there is no weight.
template <bool kInterleaved, int GL>
__device__ __forceinline__ void stage_weights(const float *w, const RowLane<GL> &at, float2 (*sw)[4])
{
    if (threadIdx.x < GL) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[i] = w && at.active ? w[at.e0 + i] : 1.f;
            x[i + 4] = w && at.active ? w[at.e1 + i] : 1.f;
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            sw[threadIdx.x][i] = kInterleaved ? make_float2(x[4 * i], x[4 * i + 2]) : make_float2(x[2 * i], x[2 * i + 1]);
            sw[threadIdx.x][2 + i] =
                kInterleaved ? make_float2(x[4 * i + 1], x[4 * i + 3]) : make_float2(x[2 * i + 4], x[2 * i + 5]);
        }
    }
    __syncthreads();
}

// 1/sqrt(x) by the hardware's approximation (2 units in the last place; a
// subnormal x counts as zero).
__device__ __forceinline__ float rsqrt_approx(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int GL>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Weight and rotation as one linear map of a pair: y_a = x_a aa + x_b ab,
// y_b = x_b bb + x_a ba; made once for all rows of a token.
struct Turn {
    float2 aa[2], ab[2], bb[2], ba[2];

    __device__ __forceinline__ Turn(const Angles &t, const float2 *w)
    {
        const float2 *wa = w, *wb = w + 2;
        const float2 c[2] = {make_float2(t.c.x, t.c.y), make_float2(t.c.z, t.c.w)};
        const float2 s[2] = {make_float2(t.s.x, t.s.y), make_float2(t.s.z, t.s.w)};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            aa[i] = __fmul2_rn(wa[i], c[i]);
            ab[i] = __fmul2_rn(wb[i], make_float2(-s[i].x, -s[i].y));
            bb[i] = __fmul2_rn(wb[i], c[i]);
            ba[i] = __fmul2_rn(wa[i], s[i]);
        }
    }
};

// Norm and rotation of a lane's part of a row.
template <int GL>
__device__ __forceinline__ void norm_rope_lane(float2 *a, float2 *b, bool normed, float inv_d, float eps, const Turn &t)
{
    if (normed) {
        float2 sq = __fmul2_rn(a[0], a[0]);
        sq = __ffma2_rn(a[1], a[1], sq);
        sq = __ffma2_rn(b[0], b[0], sq);
        sq = __ffma2_rn(b[1], b[1], sq);
        const float r = rsqrt_approx(fmaf(group_sum<GL>(sq.x + sq.y), inv_d, eps));
        const float2 rr = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            a[i] = __fmul2_rn(a[i], rr);
            b[i] = __fmul2_rn(b[i], rr);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float2 x = a[i], y = b[i];
        a[i] = __ffma2_rn(x, t.aa[i], __fmul2_rn(y, t.ab[i]));
        b[i] = __ffma2_rn(y, t.bb[i], __fmul2_rn(x, t.ba[i]));
    }
}

// Whether rows can be moved as pieces of four elements.
static inline bool pieces_ok(const HeadsView &h, size_t es)
{
    return reinterpret_cast<uintptr_t>(h.ptr) % (4 * es) == 0 && h.ts % 4 == 0 && h.hs % 4 == 0;
}
static inline bool rope_pieces_ok(const RopeView &r)
{
    return !r.table || (r.rot % 8 == 0 && reinterpret_cast<uintptr_t>(r.table) % 16 == 0);
}

static inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens of a warp: as many as make one wave of CTAs (152 SMs of `resident`), so
// that a CTA's start and end are paid for once, or as few waves as keep them
// at `most`.
static inline int64_t run_tokens(int64_t n, int64_t chunks, int64_t resident, int64_t most)
{
    const int64_t places = kWarps * 152 * resident, work = n * chunks;
    const int64_t waves = div_up(div_up(work, places), most);
    const int64_t run = div_up(work, places * (waves < 1 ? 1 : waves));
    return run < 1 ? 1 : run;
}

// f<T, GL, interleaved>(...) of the call's type, width and layout: the fewest
// lanes that hold a row (97656 tokens of 16 and 4 heads of 32 bf16 elements: 53
// us with 4 lanes, 87 with 8).
#define DLRM_HEAD_DISPATCH(f, d, dtype, interleaved, ...)                                                             \
    do {                                                                                                              \
        if (dtype == DLRM_F32)                                                                                        \
            DLRM_HEAD_WIDTH(f, float, d, interleaved, __VA_ARGS__);                                                   \
        if (dtype == DLRM_F16)                                                                                        \
            DLRM_HEAD_WIDTH(f, __half, d, interleaved, __VA_ARGS__);                                                  \
        DLRM_HEAD_WIDTH(f, __nv_bfloat16, d, interleaved, __VA_ARGS__);                                               \
    } while (0)
#define DLRM_HEAD_WIDTH(f, T, d, interleaved, ...)                                                                    \
    do {                                                                                                              \
        if (d <= 32)                                                                                                  \
            return interleaved ? f<T, 4, true>(__VA_ARGS__) : f<T, 4, false>(__VA_ARGS__);                            \
        if (d <= 64)                                                                                                  \
            return interleaved ? f<T, 8, true>(__VA_ARGS__) : f<T, 8, false>(__VA_ARGS__);                            \
        if (d <= 128)                                                                                                 \
            return interleaved ? f<T, 16, true>(__VA_ARGS__) : f<T, 16, false>(__VA_ARGS__);                          \
        return interleaved ? f<T, 32, true>(__VA_ARGS__) : f<T, 32, false>(__VA_ARGS__);                              \
    } while (0)

}  // namespace dlrm
