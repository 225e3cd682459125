// Gradient of the norm and rotation of query and key heads by the vector path
// (head_norm.cuh).  A row's lanes turn dy back, and with two sums over the row
// (x^2 and g x) write dx; the weight's gradient gathers in 8 registers of a
// lane over all its rows, then over the CTA in shared memory, and a second
// kernel adds the CTAs' sums in a fixed order.
//
// Memory bounds it: dy and x are read once, dx is written once.  65536 tokens
// of 16 query and 4 key heads of 128 bf16 elements take 191 us, 5.3 TB/s,
// 0.78 of the rate of a plain copy (rows in registers, one slot ahead: 224 us).
#include "head_norm.cuh"

namespace dlrm {

// CTAs of an SM: 3 take 231 us, 2 take 191.  Tokens of a warp at most: 21 in four
// waves take 191 us, 41 in two 198.
constexpr int kBwdResident = 2, kBwdRun = 24;

struct NormBwdParams {
    NormSide side[2];
    int fold;  // the larger of theirs
    RopeView rope;
    int64_t n;
    int d, run;
    float eps;
    float *part;  // [gridDim.y][gridDim.x][d]: sums of the weight's gradient
    int32_t *err;
};

template <typename T, int GL, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, kBwdResident)
norm_rope_bwd_vec_kernel(const __grid_constant__ NormBwdParams p)
{
    using Raw = typename Piece<T>::Raw;
    using R = Ring<T, GL, 2>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sums[kWarps][GL * 8];
    __shared__ __align__(16) float2 sw[GL][4];
    const int lane = threadIdx.x & 31;
    const RowLane<GL> at(p.d, p.rope);
    int chunk = blockIdx.y;
    const NormSide &me = p.side[side_of(p.side, chunk)];
    const Fold my(me, chunk, at.group, at.kGroups);
    const int fold = me.fold, head = my.head, slots = my.slots;
    const int rows = at.active ? me.x.heads - head : 0;  // from this lane's group on
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.run;
    const int tokens = (int)max(min((int64_t)p.run, p.n - first), (int64_t)0);
    const int steps = (tokens + fold - 1) / fold, angle_bytes = R::kAngles * fold;
    uint8_t *ring = smem + (threadIdx.x >> 5) * R::bytes(p.fold);
    uint8_t *angle_ring = ring + R::kDepth * R::kSlot + my.token * R::kAngles, *mine = ring + lane * R::kPiece;

    int64_t position = 0;  // lane i: token i's
    if (p.rope.table && lane < tokens)
        position = __ldg(p.rope.positions + first + lane);

    // the copies run kDepth - 1 slots ahead; the first rows do not wait for the positions
    const T *x_row = me.x.row<T>(first + my.token, head), *y_row = me.dy.row<T>(first + my.token, head);
    const int64_t x_step = at.kGroups * me.x.hs, y_step = at.kGroups * me.dy.hs;
    int ahead_step = 0, ahead_slot = 0, ahead = 0;
    auto copy_slot = [&] {
        if (ahead_step < steps) {
            const bool there = ahead_slot * at.kGroups < rows && ahead_step * fold + my.token < tokens;
            copy_row<T, GL>(mine + ahead * R::kSlot, x_row, me.x.ptr, there, at);
            copy_row<T, GL>(mine + ahead * R::kSlot + R::kSlot / 2, y_row, me.x.ptr, there, at);
            const bool last = ahead_slot + 1 == slots;
            x_row += last ? fold * me.x.ts - (slots - 1) * x_step : x_step;
            y_row += last ? fold * me.dy.ts - (slots - 1) * y_step : y_step;
            ahead_slot = last ? 0 : ahead_slot + 1;
            ahead_step += last;
        }
        ahead = ahead + 1 == R::kDepth ? 0 : ahead + 1;
    };
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; i++)
        copy_slot();
    const float *my_angles = nullptr;
    if (p.rope.table && lane < tokens)
        my_angles = rope_row(p.rope, position, p.err);
    auto copy_turn = [&](int step) {
        if (step < steps) {
            const float *a = reinterpret_cast<const float *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<int64_t>(my_angles), step * fold + my.token));
            copy_angles<GL>(angle_ring + step % R::kDepth * angle_bytes, a, p.rope.rot >> 1, at, my.first);
        }
    };
    auto copy = [&] {
        if (ahead_slot == 0)
            copy_turn(ahead_step);
        copy_slot();
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; i++) {
        if (i % slots == 0)
            copy_turn(i / slots);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    stage_weights<kInterleaved>(me.w, at, sw);

    const float inv_d = 1.f / (float)p.d;
    const float2 *wa = sw[lane % GL], *wb = wa + 2;
    float2 da[2] = {}, db[2] = {};
    T *to = me.out.row<T>(first + my.token, head);
    const int64_t to_step = at.kGroups * me.out.hs, to_wrap = fold * me.out.ts - slots * to_step;
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < steps; i++, to += to_wrap) {
        const int token = i * fold + my.token;
        const bool bad = p.rope.table && !__shfl_sync(0xffffffffu, reinterpret_cast<int64_t>(my_angles), token);
        copy();
        asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
        __syncwarp();
        const Angles t(reinterpret_cast<const float4 *>(angle_ring + i % R::kDepth * angle_bytes + lane % GL * 32),
                       at.angle >= 0 && !bad);
        const float2 c[2] = {make_float2(t.c.x, t.c.y), make_float2(t.c.z, t.c.w)};
        const float2 s[2] = {make_float2(t.s.x, t.s.y), make_float2(t.s.z, t.s.w)};
#pragma unroll 1
        for (int u = 0; u < slots; u++) {
            if (u > 0) {
                copy();
                asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
            }
            Raw x[2], y[2];
            read_row<T>(mine + slot * R::kSlot, x);
            read_row<T>(mine + slot * R::kSlot + R::kSlot / 2, y);
            slot = slot + 1 == R::kDepth ? 0 : slot + 1;
            const bool there = u * at.kGroups < rows && token < tokens, counts = there && !bad;
            if (!counts)  // gives zeros, and adds nothing
                x[0] = x[1] = y[0] = y[1] = Raw{};
            float2 a[2], b[2], ga[2], gb[2];
            widen_row<T, kInterleaved>(x, a, b);
            widen_row<T, kInterleaved>(y, ga, gb);
#pragma unroll
            for (int i = 0; i < 2; i++) {  // turned back
                const float2 f = ga[i], g = gb[i];
                ga[i] = __ffma2_rn(f, c[i], __fmul2_rn(g, s[i]));
                gb[i] = __ffma2_rn(g, c[i], __fmul2_rn(make_float2(-f.x, -f.y), s[i]));
            }
            Raw z[2];
            if (me.w) {
                float2 va[2], vb[2], sq = make_float2(0.f, 0.f), gx = sq;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    va[i] = __fmul2_rn(ga[i], wa[i]);
                    vb[i] = __fmul2_rn(gb[i], wb[i]);
                    sq = __ffma2_rn(a[i], a[i], __ffma2_rn(b[i], b[i], sq));
                    gx = __ffma2_rn(va[i], a[i], __ffma2_rn(vb[i], b[i], gx));
                }
                float s1 = sq.x + sq.y, s2 = gx.x + gx.y;
#pragma unroll
                for (int o = GL / 2; o > 0; o >>= 1) {
                    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                    s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                }
                const float r = counts ? rsqrt_approx(fmaf(s1, inv_d, p.eps)) : 0.f, m = -s2 * inv_d * r * r;
                const float2 rr = make_float2(r, r), mm = make_float2(m, m);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    a[i] = __fmul2_rn(a[i], rr);
                    b[i] = __fmul2_rn(b[i], rr);
                    da[i] = __ffma2_rn(ga[i], a[i], da[i]);
                    db[i] = __ffma2_rn(gb[i], b[i], db[i]);
                    ga[i] = __ffma2_rn(va[i], rr, __fmul2_rn(a[i], mm));
                    gb[i] = __ffma2_rn(vb[i], rr, __fmul2_rn(b[i], mm));
                }
            }
            narrow_row<T, kInterleaved>(ga, gb, z);
            store_row<T, GL>(to, there, at, z);
            to += to_step;
        }
    }
    // the lane groups of a warp, then the warps
    float ra[4] = {da[0].x, da[0].y, da[1].x, da[1].y}, rb[4] = {db[0].x, db[0].y, db[1].x, db[1].y};
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int o = 16; o >= GL; o >>= 1) {
            ra[i] += __shfl_xor_sync(0xffffffffu, ra[i], o);
            rb[i] += __shfl_xor_sync(0xffffffffu, rb[i], o);
        }
    if (at.group == 0 && at.active)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float *row = sums[threadIdx.x >> 5];
            row[kInterleaved ? (i < 2 ? at.e0 : at.e1) + (2 * i & 3) : at.e0 + i] = ra[i];
            row[kInterleaved ? (i < 2 ? at.e0 : at.e1) + (2 * i & 3) + 1 : at.e1 + i] = rb[i];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < p.d; e += kWarps * 32) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; i++)
            t += sums[i][e];
        p.part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.d + e] = t;
    }
}

static int64_t bwd_run(int64_t n, int64_t chunks) { return run_tokens(n, chunks, kBwdResident, kBwdRun); }

size_t norm_bwd_vec_workspace(int64_t n, int qh, int kh, int d)
{
    const int64_t heads = kSlots * (d <= 32 ? 8 : (d <= 64 ? 4 : (d <= 128 ? 2 : 1)));
    const int64_t chunks = div_up(qh, heads) + div_up(kh, heads);
    return (size_t)(chunks * div_up(n, kWarps * bwd_run(n, chunks))) * d * sizeof(float) + 16;
}

void launch_norm_weight_sum(const float *, int64_t, int64_t, int, float *, float *, cudaStream_t);

template <typename T, int GL, bool kInterleaved>
static int norm_bwd_vec(const HeadsView &dqo, const HeadsView &dko, const HeadsView &q, const HeadsView &k, int64_t n,
                        int d, const float *qw, const float *kw, float eps, const RopeView &rope, const HeadsView &dq,
                        const HeadsView &dk, float *dqw, float *dkw, float *part, int32_t *err, cudaStream_t st)
{
    NormBwdParams p = {};
    p.side[0] = {q, dqo, dq, qw, 0, 1};
    p.side[1] = {k, dko, dk, kw, 0, 1};
    p.fold = 1;
    for (NormSide &side : p.side) {
        side.lay_out(32 / GL);
        p.fold = side.fold > p.fold ? side.fold : p.fold;
    }
    const int64_t qc = p.side[0].chunks, kc = p.side[1].chunks, run = bwd_run(n, qc + kc), x = div_up(n, kWarps * run);
    p.rope = rope;
    p.n = n;
    p.d = d;
    p.run = (int)run;
    p.eps = eps;
    p.part = part;
    p.err = err;
    static std::atomic<unsigned long long> done{0};
    const int s = allow_dynamic_smem((const void *)norm_rope_bwd_vec_kernel<T, GL, kInterleaved>,
                                     kWarps * Ring<T, GL, 2>::bytes(32 / GL), &done);
    if (s != DLRM_OK)
        return s;
    norm_rope_bwd_vec_kernel<T, GL, kInterleaved><<<dim3((unsigned)x, (unsigned)(qc + kc)), kWarps * 32,
                                                 kWarps * Ring<T, GL, 2>::bytes(p.fold), st>>>(p);
    count_launch(st);
    if (dqw || dkw)
        launch_norm_weight_sum(part, x * qc, x * kc, d, dqw, dkw, st);
    return launch_status();
}

int launch_norm_rope_bwd_vec(const HeadsView &dqo, const HeadsView &dko, const HeadsView &q, const HeadsView &k,
                             int64_t n, int d, int dtype, const float *qw, const float *kw, float eps,
                             const RopeView &rope, const HeadsView &dq, const HeadsView &dk, float *dqw, float *dkw,
                             float *part, int32_t *err, cudaStream_t st)
{
    DLRM_HEAD_DISPATCH(norm_bwd_vec, d, dtype, rope.interleaved, dqo, dko, q, k, n, d, qw, kw, eps, rope, dq, dk, dqw,
                       dkw, part, err, st);
}

}  // namespace dlrm
