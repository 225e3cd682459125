// Pages and slots for a step's new tokens, from the sequences' counts.
//
// Sequence s stores len tokens and gets c more: it needs
// ceil((len + c) / page) - ceil(len / page) pages.  Prefix sums of the counts are
// the batch's offsets; prefix sums of the needs say which entries of the free
// pages' ring a sequence takes, so no page is fought over and the result does
// not depend on the order in which threads run.  A token's page is then an
// entry of its table row or of the ring, found without a second pass.
//
// What bounds it is the launch and one prefix sum's latency (a step of 2048
// users writes 130 KB); a batch of prompts is bound by the 16 bytes written a
// token.  So there is one kernel of one CTA for short steps; for longer ones
// every CTA takes a run of tokens and sums up the sequences before it by itself
// (16 bytes a sequence from L2, which costs less than a second kernel that waits for
// the first).  Where lengths or the ring's state, which all CTAs read, are written in place,
// a launch of its own does that afterwards.  One event of each of 2048 users: 11 us from
// call to call, 9.5 in a graph; 512 users with up to 4096 new (14.4 MB): 16 and 13.5.
#include "history.cuh"

namespace dlrm {

constexpr int kResThreads = 1024, kResItems = 2, kResChunk = kResThreads * kResItems;
constexpr int kResTokens = kResThreads / 2;  // of a CTA, more where kResMaxCtas would not do
constexpr int kResMaxCtas = 152;
constexpr int kResLanes = 16, kResRun = 4;  // threads that look at a row given back; numbers that each asks for at once

struct ReserveParams {
    const int64_t *counts, *lengths;
    int64_t S, n;
    int32_t *table;
    int64_t table_stride, capacity;
    FastDiv page;
    int32_t *ring;
    int64_t pages;
    const int64_t *state;
    int64_t *new_state, *offsets, *new_lengths, *slots, *positions;
    int32_t *err;
};

// Sums over the sequences before one: new tokens, pages needed, pages given back.
struct ReserveSums {
    int64_t tokens, need, gone;
};

__device__ __forceinline__ ReserveSums operator+(const ReserveSums &a, const ReserveSums &b)
{
    return {a.tokens + b.tokens, a.need + b.need, a.gone + b.gone};
}

__device__ __forceinline__ ReserveSums shfl_up(const ReserveSums &x, int o)
{
    return {__shfl_up_sync(0xffffffffu, x.tokens, o), __shfl_up_sync(0xffffffffu, x.need, o),
            __shfl_up_sync(0xffffffffu, x.gone, o)};
}

// kTokens: this launch writes slots, positions, table entries and the ring;
// kSequences: its first CTA writes offsets, lengths and the state.
template <bool kTokens, bool kSequences>
__global__ void __launch_bounds__(kResThreads)
kv_reserve_kernel(const __grid_constant__ ReserveParams p)
{
    __shared__ ReserveSums warp_sums[kResThreads / 32];
    // of the chunk's sequences: tokens and needs before it (from the chunk's first), stored tokens, and whether
    // it has its pages (0: it is left out, -1: it has left, -2: and some numbers of its row are no pages)
    __shared__ uint32_t s_tokens[kResChunk + 1];
    __shared__ int32_t s_need[kTokens ? kResChunk : 1], s_gone[kTokens ? kResChunk : 1];
    __shared__ int32_t s_length[kTokens ? kResChunk : 1];
    __shared__ int8_t s_granted[kTokens ? kResChunk : 1];
    // those who give pages back, in any order, and how many (of this chunk, of the next)
    __shared__ uint16_t s_leavers[kResChunk];
    __shared__ int32_t s_held[kResChunk];
    __shared__ int s_leaving[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t head = p.state[0], tail = p.state[1];
    const bool sound = tail >= head && tail - head <= p.pages && head >= 0;
    const int64_t avail = sound ? tail - head : 0;
    const uint64_t ring_head = sound ? (uint64_t)head % (uint64_t)p.pages : 0;
    const uint64_t ring_tail = sound ? (uint64_t)tail % (uint64_t)p.pages : 0;
    // an entry of the ring, k < 2^31 places after one
    auto place = [&](uint64_t from, int64_t k) {
        const uint64_t at = from + (uint64_t)k;
        return at >= (uint64_t)p.pages ? at - (uint64_t)p.pages : at;
    };
    // pages of so many tokens, at most 2^30
    auto pages_of = [&](int tokens) { return (int)p.page.div((uint32_t)tokens + p.page.d - 1); };
    const int64_t slice = (p.n + gridDim.x - 1) / gridDim.x;
    const int64_t t0 = min(blockIdx.x * slice, p.n), t1 = min(t0 + slice, p.n);
    ReserveSums base = {0, 0, 0};
    int64_t taken = 0;  // this thread's largest granted sum
    const bool sequences = kSequences && blockIdx.x == 0;
    if (sequences && threadIdx.x == 0 && !sound)
        raise_flag(p.err, DLRM_FLAG_BAD_OFFSETS);
    auto is_page = [&](int32_t page) { return (uint32_t)page < (uint64_t)p.pages; };
    if (threadIdx.x < 2)
        s_leaving[threadIdx.x] = 0;
    for (int64_t c0 = 0; c0 < p.S; c0 += kResChunk) {
        int &leaving = s_leaving[c0 / kResChunk & 1], &next_leaving = s_leaving[~(c0 / kResChunk) & 1];
        const int64_t s0 = c0 + threadIdx.x * kResItems;
        int64_t take[kResItems], len[kResItems], need[kResItems], gone[kResItems];
        bool leaves[kResItems], fits[kResItems];
        ReserveSums mine = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < kResItems; i++) {
            const bool there = s0 + i < p.S;
            const int64_t count = there ? p.counts[s0 + i] : 0, x = there ? p.lengths[s0 + i] : 0;
            len[i] = x < 0 ? ~x : x;
            leaves[i] = count < 0;
            take[i] = count < 0 ? 0 : min(count, (int64_t)1 << 31);
            const bool stored = len[i] <= p.capacity;
            fits[i] = !leaves[i] && stored && take[i] <= p.capacity - len[i];
            const int64_t held = stored ? pages_of((int)len[i]) : 0;
            need[i] = fits[i] ? pages_of((int)(len[i] + take[i])) - held : 0;
            gone[i] = leaves[i] ? held : 0;
            if (sequences && !stored && leaves[i])
                raise_flag(p.err, DLRM_FLAG_BAD_OFFSETS);
            mine = mine + ReserveSums{take[i], need[i], gone[i]};
        }
        // Sums over the chunk.  Meanwhile 16 threads a row look for numbers that are no pages among those given back; they
        // are passed over, which moves all after them, so where there are any, the rows' pages are counted and summed up
        // again.  (One event of each of 2048 users, 128 of whom leave, and prompts of 512, of whom 64 leave, in a graph:
        // 9.5 and 13.5 us, without looking 8.2 and 12.5; where nobody leaves the same.  8 threads a row 9.5 and 14.0,
        // whole warps, before the sums, 10.3 and 16.7.)
        bool odd[kResItems] = {};
        ReserveSums sum;
        for (bool counted = false;; counted = true) {
            sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const ReserveSums x = shfl_up(sum, o);
                if (lane >= o)
                    sum = sum + x;
            }
            __syncthreads();  // the chunk before has been read
            if (lane == 31)
                warp_sums[warp] = sum;
#pragma unroll
            for (int i = 0; i < kResItems; i++)
                if (!counted && gone[i] > 0) {
                    const int in = threadIdx.x * kResItems + i;
                    s_held[in] = (int)gone[i];
                    s_leavers[atomicAdd(&leaving, 1)] = (uint16_t)in;
                }
            __syncthreads();
            if (warp == 0) {
                ReserveSums w = warp_sums[lane];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const ReserveSums x = shfl_up(w, o);
                    if (lane >= o)
                        w = w + x;
                }
                warp_sums[lane] = w;
            }
            bool bad = false;
            for (int r = threadIdx.x / kResLanes; !counted && r < leaving; r += kResThreads / kResLanes) {
                const int in = s_leavers[r], held = s_held[in];
                const int32_t *row = p.table + (c0 + in) * p.table_stride;
                for (int k = threadIdx.x % kResLanes; k < held; k += kResLanes * kResRun) {
                    int32_t page[kResRun];
#pragma unroll
                    for (int j = 0; j < kResRun; j++)
                        page[j] = k + j * kResLanes < held ? row[k + j * kResLanes] : 0;
#pragma unroll
                    for (int j = 0; j < kResRun; j++)
                        bad |= !is_page(page[j]);
                }
            }
            if (!__syncthreads_or(bad))
                break;
#pragma unroll
            for (int i = 0; i < kResItems; i++) {
                for (uint32_t left = __ballot_sync(0xffffffffu, gone[i] > 0); left != 0; left &= left - 1) {
                    const int who = __ffs(left) - 1, held = __shfl_sync(0xffffffffu, (int)gone[i], who);
                    const int32_t *row = p.table + (c0 + (warp * 32 + who) * kResItems + i) * p.table_stride;
                    int pages = 0;
                    for (int k = lane; k < held; k += 32)
                        pages += is_page(row[k]);
                    pages = __reduce_add_sync(0xffffffffu, pages);
                    if (lane == who && pages < held) {
                        odd[i] = true;
                        mine.gone -= held - pages;
                        gone[i] = pages;
                        if (sequences)
                            raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
                    }
                }
            }
        }
        if (threadIdx.x == 0)
            next_leaving = 0;
        ReserveSums at = warp > 0 ? warp_sums[warp - 1] : ReserveSums{0, 0, 0};  // from the chunk's first
        at = at + ReserveSums{sum.tokens - mine.tokens, sum.need - mine.need, sum.gone - mine.gone};
        const ReserveSums all = warp_sums[kResThreads / 32 - 1];
#pragma unroll
        for (int i = 0; i < kResItems; i++) {
            const int in = threadIdx.x * kResItems + i;
            const bool rows = take[i] == 0 || base.tokens + at.tokens + take[i] <= p.n;
            const bool granted = fits[i] && rows && (need[i] == 0 || base.need + at.need + need[i] <= avail);
            if (granted && need[i] > 0)
                taken = max(taken, base.need + at.need + need[i]);
            if (kTokens) {
                s_tokens[in] = (uint32_t)min(at.tokens, (int64_t)0xffffffffu);
                // beyond 2^31 they are past every granted need and every place of the ring
                s_need[in] = (int)min(at.need, (int64_t)0x7fffffff);
                s_gone[in] = (int)min(at.gone, (int64_t)0x7fffffff);
                s_length[in] = (int)min(len[i], (int64_t)0x7fffffff);
                s_granted[in] = leaves[i] ? (odd[i] ? -2 : -1) : (granted ? 1 : 0);
            }
            if (sequences && s0 + i < p.S) {
                p.offsets[s0 + i] = base.tokens + at.tokens;
                p.new_lengths[s0 + i] = leaves[i] ? 0 : (granted ? len[i] + take[i] : ~len[i]);
                if (!granted && !leaves[i])
                    raise_flag(p.err, fits[i] && rows ? DLRM_FLAG_CAPACITY : DLRM_FLAG_BAD_OFFSETS);
            }
            at = at + ReserveSums{take[i], need[i], gone[i]};
        }
        if (kTokens) {
            if (threadIdx.x == 0)
                s_tokens[kResChunk] = (uint32_t)min(all.tokens, (int64_t)0xffffffffu);
            __syncthreads();
            const int here = (int)min(p.S - c0, (int64_t)kResChunk);
            // the last of the chunk's sequences whose sum is at most x: those that add nothing come before
            auto owner = [&](const auto *sums, auto x) {
                int lo = 0, hi = here;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (sums[mid] <= x)
                        lo = mid;
                    else
                        hi = mid;
                }
                return lo;
            };
            // pages of those who leave, shared out over the CTAs
            for (int64_t k = (int64_t)blockIdx.x * kResThreads + threadIdx.x; k < all.gone; k += (int64_t)gridDim.x * kResThreads) {
                if (!sound || avail + base.gone + k >= p.pages) {
                    raise_flag(p.err, DLRM_FLAG_CAPACITY);
                    break;
                }
                const int in = owner(s_gone, (int)k);
                const int32_t *row = p.table + (c0 + in) * p.table_stride;
                int number = (int)k - s_gone[in];
                if (s_granted[in] == -2) {  // among those that are pages
                    int before = number;
                    const int last = pages_of(s_length[in]) - 1;
                    for (number = 0; number < last; number++)
                        if (is_page(row[number]) && before-- == 0)
                            break;
                }
                p.ring[place(ring_tail, base.gone + k)] = row[number];
            }
            // this CTA's tokens among the chunk's
            const int64_t from = max(t0, base.tokens), to = min(t1, base.tokens + all.tokens);
            for (int64_t t = from + threadIdx.x; t < to; t += kResThreads) {
                const uint32_t x = (uint32_t)(t - base.tokens);
                const int lo = owner(s_tokens, x);
                int64_t slot = -1, position = -1;
                if (s_granted[lo] > 0) {
                    const int length = s_length[lo], at_token = length + (int)(x - s_tokens[lo]);
                    const int number = (int)p.page.div((uint32_t)at_token), in_page = at_token - number * (int)p.page.d;
                    const int held = pages_of(length);
                    int32_t *entry = p.table + (c0 + lo) * p.table_stride + number;
                    int32_t page;
                    if (number < held) {
                        page = *entry;
                    } else {
                        page = p.ring[place(ring_head, base.need + s_need[lo] + number - held)];
                        if (in_page == 0)
                            *entry = page;
                    }
                    position = at_token;
                    if ((uint32_t)page < (uint64_t)p.pages)
                        slot = (int64_t)page * p.page.d + in_page;
                    else
                        raise_flag(p.err, DLRM_FLAG_INDEX_OOB);
                }
                if (p.slots)
                    p.slots[t] = slot;
                if (p.positions)
                    p.positions[t] = position;
            }
        }
        base = base + all;
    }
    if (sequences) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
        __syncthreads();
        if (lane == 0)
            warp_sums[warp].need = taken;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kResThreads / 32; w++)
                taken = max(taken, warp_sums[w].need);
            p.offsets[p.S] = base.tokens;
            p.new_state[0] = head + taken;
            p.new_state[1] = sound ? tail + min(base.gone, p.pages - avail) : tail;
        }
    }
}

int launch_kv_reserve(const int64_t *counts, const int64_t *lengths, int64_t S, int64_t n, int32_t *table,
                      int64_t table_stride, int64_t table_width, int page_size, int32_t *ring, int64_t pages,
                      const int64_t *state, int64_t *new_state, int64_t *offsets, int64_t *new_lengths, int64_t *slots,
                      int64_t *positions, int32_t *err, cudaStream_t st)
{
    const ReserveParams p = {counts, lengths, S, n, table, table_stride, table_width * page_size,
                             FastDiv::make((uint32_t)page_size), ring, pages, state, new_state, offsets, new_lengths,
                             slots, positions, err};
    // In place the second launch costs 4 us: one CTA takes up to 4096 tokens.  Steps of one event of 2048 users, of
    // 8192, us (in a graph; one CTA, many, many and a second launch): 12, 8, 12; 41, 21, 28; 64 users' prompts of up
    // to 200: 11, 7, 9; of one event of 8: 6.
    const bool in_place = new_lengths == lengths || new_state == state;
    const int64_t all = (n + kResTokens - 1) / kResTokens;
    const unsigned ctas = n <= (in_place ? 8 : 1) * kResTokens ? 1u : (unsigned)(all < kResMaxCtas ? all : kResMaxCtas);
    if (ctas == 1 || !in_place) {
        kv_reserve_kernel<true, true><<<ctas, kResThreads, 0, st>>>(p);
        count_launch(st);
        return launch_status();
    }
    kv_reserve_kernel<true, false><<<ctas, kResThreads, 0, st>>>(p);
    count_launch(st);
    kv_reserve_kernel<false, true><<<1, kResThreads, 0, st>>>(p);
    count_launch(st);
    return launch_status();
}

}  // namespace dlrm
