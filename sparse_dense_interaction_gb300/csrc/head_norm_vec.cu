// Norm and rotation of query and key heads, and the append to the paged
// cache, by the vector path (head_norm.cuh).
//
// Memory bounds both: a row is read once and written once.  65536 tokens of 16
// query and 4 key heads of 128 bf16 elements take 116 us, 5.8 TB/s, 0.86 of the
// rate of a plain copy; the append of 26k tokens with their queries 103 us, 5.7 TB/s.
// With one slot loaded ahead in registers instead of the ring they took 146
// and 163 us: the loads in flight were what lacked.
#include "head_norm.cuh"

namespace dlrm {

// CTAs of an SM: with 4 the forward above takes 133 us (more rows of memory
// open at once), with 2 it takes 130.  Tokens of a warp at most: 27 in two waves
// take 116 us, 54 in one (which ends unevenly) 130.
constexpr int kResident = 3, kRun = kMaxRun;

struct NormParams {
    NormSide side[3];  // queries, keys, values; out: not of keys and values that go to the cache
    int fold;          // the largest of them
    RopeView rope;
    BatchView batch;   // of the append; else only n
    CacheView cache;
    int d, run;
    float eps;
    int32_t *err;
};

// The sequences of up to 32 neighbouring tokens, lane l's token being first + l
// and s0 the first's: the 32 sequence starts after s0 are read at once; beyond
// them (many sequences without tokens) a lane searches.  All lanes call it.
__device__ __forceinline__ int64_t lane_sequence(const BatchView &b, int64_t s0, int64_t i)
{
    const int64_t next = s0 + 1 + (threadIdx.x & 31);
    const int64_t start = next <= b.S ? b.offsets[next] : INT64_MAX;
    int count = 0;
#pragma unroll 8
    for (int j = 0; j < 32; j++)
        count += __shfl_sync(0xffffffffu, start, j) <= i;
    int64_t lo = min(s0 + count, b.S - 1), hi = b.S;
    if (count == 32)
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (b.offsets[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
    return lo;
}

template <typename T, int GL, bool kInterleaved, bool kAppend>
__global__ void __launch_bounds__(kWarps * 32, kResident)
norm_rope_vec_kernel(const __grid_constant__ NormParams p)
{
    using Raw = typename Piece<T>::Raw;
    using R = Ring<T, GL, 1>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float2 sw[GL][4];
    const int lane = threadIdx.x & 31;
    const RowLane<GL> at(p.d, p.rope);
    int chunk = blockIdx.y;
    const int which = side_of(p.side, chunk);
    const NormSide &me = p.side[which];
    const bool is_v = kAppend && which == 2, cached = kAppend && which > 0;
    const Fold my(me, chunk, at.group, at.kGroups);
    const int fold = me.fold, head = my.head, slots = my.slots;
    const int rows = at.active ? me.x.heads - head : 0;  // from this lane's group on
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.run;
    const int tokens = (int)max(min((int64_t)p.run, p.batch.n - first), (int64_t)0);
    const int steps = (tokens + fold - 1) / fold, angle_bytes = R::kAngles * fold;
    uint8_t *ring = smem + (threadIdx.x >> 5) * R::bytes(p.fold);
    uint8_t *angle_ring = ring + R::kDepth * R::kSlot + my.token * R::kAngles, *mine = ring + lane * R::kPiece;

    // lane i: token i's angles, and where its rows go (0: it is left out)
    const float *my_angles = nullptr;
    int64_t my_to = 0;
    const int64_t my_token = first + lane;
    int64_t s0 = -1, s = 0;
    if (kAppend && tokens > 0) {
        s0 = find_sequence(p.batch, first);
        if (s0 >= 0)
            s = lane_sequence(p.batch, s0, my_token);
    }
    if (lane < tokens) {
        int64_t position = -1;
        bool good = true;
        Sequence seq = {0, 0, 0};
        if (kAppend) {
            good = s0 >= 0 && read_sequence(p.batch, s, p.batch.n, p.batch.capacity, seq, p.err) &&
                   seq.has(my_token) && seq.count <= seq.length;
            position = seq.length - seq.count + my_token - seq.first;
            if (!good)
                raise_flag(p.err, DLRM_FLAG_BAD_OFFSETS);
        }
        if (good) {
            const int place = (int)position;
            if (p.rope.table) {
                position = p.rope.positions ? __ldg(p.rope.positions + my_token) : position;
                my_angles = rope_row(p.rope, position, p.err);
            }
            if (!cached) {
                my_to = reinterpret_cast<int64_t>(me.out.row<T>(my_token, 0));
            } else {
                const int64_t slot = slot_offset<T>(p.cache, p.batch.table + s * p.batch.table_stride, place, 0);
                if (slot < 0)
                    raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
                else if (!p.rope.table || my_angles)  // a token that cannot be turned is not stored
                    my_to = reinterpret_cast<int64_t>((is_v ? p.cache.v : p.cache.k) + slot);
            }
        }
    }

    // the copies run kDepth - 1 slots ahead
    const T *row = me.x.row<T>(first + my.token, head);
    const int64_t step = at.kGroups * me.x.hs, wrap = fold * me.x.ts - (slots - 1) * step;
    int ahead_step = 0, ahead_slot = 0, ahead = 0;
    auto copy = [&] {
        if (ahead_step < steps) {
            const int token = ahead_step * fold + my.token;
            if (ahead_slot == 0 && !is_v) {
                const float *a = reinterpret_cast<const float *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<int64_t>(my_angles), token));
                copy_angles<GL>(angle_ring + ahead_step % R::kDepth * angle_bytes, a, p.rope.rot >> 1, at, my.first);
            }
            copy_row<T, GL>(mine + ahead * R::kSlot, row, me.x.ptr,
                            ahead_slot * at.kGroups < rows && token < tokens, at);
            const bool last = ahead_slot + 1 == slots;
            row += last ? wrap : step;
            ahead_slot = last ? 0 : ahead_slot + 1;
            ahead_step += last;
        }
        ahead = ahead + 1 == R::kDepth ? 0 : ahead + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; i++)
        copy();
    if (kAppend)
        check_sequences(p.batch, ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                        (int64_t)gridDim.y * gridDim.x * blockDim.x, p.err);
    stage_weights<kInterleaved>(me.w, at, sw);

    const float inv_d = 1.f / (float)p.d;
    const int64_t to_step = at.kGroups * (cached ? p.cache.head_stride : me.out.hs);
    const int64_t to_head = head * (cached ? p.cache.head_stride : me.out.hs);
    int slot = 0;
#pragma unroll 1
    for (int t = 0; t < steps; t++) {
        const int token = t * fold + my.token;
        T *to = reinterpret_cast<T *>(__shfl_sync(0xffffffffu, my_to, token));  // none past the last token
        const bool there = to != nullptr;
        const bool turns = p.rope.table && !is_v;
        const bool zero = turns && !__shfl_sync(0xffffffffu, reinterpret_cast<int64_t>(my_angles), token);
        to += to_head;
        copy();
        asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
        __syncwarp();
        const Angles angles(reinterpret_cast<const float4 *>(angle_ring + t % R::kDepth * angle_bytes + lane % GL * 32),
                            at.angle >= 0 && turns && !zero);
        const Turn turn(angles, sw[lane % GL]);
#pragma unroll 1
        for (int s = 0; s < slots; s++) {
            if (s > 0) {
                copy();
                asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
            }
            Raw x[2];
            read_row<T>(mine + slot * R::kSlot, x);
            slot = slot + 1 == R::kDepth ? 0 : slot + 1;
            if (!is_v) {
                float2 a[2], b[2];
                widen_row<T, kInterleaved>(x, a, b);
                norm_rope_lane<GL>(a, b, me.w != nullptr, inv_d, p.eps, turn);
                narrow_row<T, kInterleaved>(a, b, x);
            }
            if (zero)
                x[0] = x[1] = Raw{};
            store_row<T, GL>(to, there && s * at.kGroups < rows, at, x);
            to += to_step;
        }
    }
}

template <typename T, int GL, bool kInterleaved, bool kAppend>
static int norm_launch(NormParams &p, cudaStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)norm_rope_vec_kernel<T, GL, kInterleaved, kAppend>,
                                     kWarps * Ring<T, GL, 1>::bytes(32 / GL), &done);
    if (s != DLRM_OK)
        return s;
    int64_t chunks = 0;
    p.fold = 1;
    for (NormSide &side : p.side) {
        side.lay_out(32 / GL);
        chunks += side.chunks;
        p.fold = side.fold > p.fold ? side.fold : p.fold;
    }
    p.run = (int)run_tokens(p.batch.n, chunks, kResident, kRun);
    norm_rope_vec_kernel<T, GL, kInterleaved, kAppend>
        <<<dim3((unsigned)div_up(p.batch.n, kWarps * p.run), (unsigned)chunks), kWarps * 32,
           kWarps * Ring<T, GL, 1>::bytes(p.fold), st>>>(p);
    count_launch(st);
    return launch_status();
}

template <typename T, int GL, bool kInterleaved>
static int norm_vec(NormParams &p, cudaStream_t st) { return norm_launch<T, GL, kInterleaved, false>(p, st); }
template <typename T, int GL, bool kInterleaved>
static int append_vec(NormParams &p, cudaStream_t st) { return norm_launch<T, GL, kInterleaved, true>(p, st); }

int launch_norm_rope_vec(const HeadsView &q, const HeadsView &k, int64_t n, int d, int dtype, const float *qw,
                         const float *kw, float eps, const RopeView &rope, const HeadsView &qo, const HeadsView &ko,
                         int32_t *err, cudaStream_t st)
{
    NormParams p = {};
    p.side[0] = {q, {}, qo, qw, 0, 1};
    p.side[1] = {k, {}, ko, kw, 0, 1};
    p.rope = rope;
    p.batch.n = n;
    p.d = d;
    p.eps = eps;
    p.err = err;
    DLRM_HEAD_DISPATCH(norm_vec, d, dtype, rope.interleaved, p, st);
}

int launch_kv_append_vec(const HeadsView &k, const HeadsView &v, const BatchView &batch, const CacheView &cache, int d,
                         int dtype, const float *kw, float eps, const RopeView &rope, const HeadsView &q,
                         const float *qw, const HeadsView &qo, int32_t *err, cudaStream_t st)
{
    NormParams p = {};
    p.side[0] = {q, {}, qo, qw, 0, 1};
    p.side[1] = {k, {}, {}, kw, 0, 1};
    p.side[2] = {v, {}, {}, nullptr, 0, 1};
    p.rope = rope;
    p.batch = batch;
    p.cache = cache;
    p.d = d;
    p.eps = eps;
    p.err = err;
    DLRM_HEAD_DISPATCH(append_vec, d, dtype, rope.interleaved, p, st);
}

}  // namespace dlrm
