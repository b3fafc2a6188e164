// top_kernel.cu -- each row's most likely tokens with their logprobs, the mass of all
// others, and with them the logprob of a given token and the entropy.
//
// One pass over a row, in chunks of 16 KB that a producer warp brings into shared memory
// ahead of the eight warps that read them. What is above a bar is put into a list, what
// is not is added up, as 2^((x - ref) c) with ref the bar's value: no exponential is
// above 1, the running maximum is not needed, and the mass outside the top n is a sum
// of its own and not a difference that cancels.
//   The bar. At least n logits are above it, and all of those are in the list. The first
//   chunk gives one: of the 256 threads' largest, the n-th. A list that grows over
//   `trigger` is cut down to about n, whose least is the new bar; what falls out is added
//   to the sum, as whole multiples of 2^-40 of its largest, so that the order in which the
//   threads come does not matter.
//   Order. A logit and its token are one 64-bit key (the larger logit, then the lower
//   token, is the larger key), so that n keys are always exactly n tokens, whatever ties
//   there are. Tokens of later chunks lose ties, so the bar is passed by `x > bar` alone.
//   Chunks that overflow the list (rows that ascend, ties in the first chunk) are cut in
//   registers: a bisection over keys counts the list and the chunk together.
// Few rows are cut into parts, a CTA each, which leave their n keys and sums in the
// workspace; the part that ends last joins them, parts in order.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "row_loss.cuh"
#include "row_queue.cuh"
#include "row_vectors.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace top {

using namespace rows;

constexpr int kWarps = 8;
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kVecs = 4;                        // of a chunk in each consumer
constexpr int kChunkVecs = kConsumers * kVecs;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kSlots = 5;
constexpr int kMost = SAMPLER_MAX_ALTERNATIVES;
constexpr int kCap = 2048;                      // keys in the list
constexpr int kHeld = kCap / kConsumers;        // of them to a thread
constexpr double kLostUnit = 1099511627776.0;   // 2^40

struct Shared {
    uint64_t full[kSlots], empty[kSlots];
    RowQueue queue;
    uint64_t list[kCap];
    uint64_t sorted[kMost];
    float4 sums[kWarps];
    uint32_t tally[3];
    uint32_t count;             // keys put into the list (more than kCap: the last of them are not there)
    unsigned long long lost_s;  // what fell out of the list, relative to the largest of it, in multiples of 2^-40
    long long lost_t;
    uint32_t lost_most;         // its order
    uint32_t flag;
};
constexpr int kSmem = kSlots * kChunkBytes + int(sizeof(Shared));

__device__ __forceinline__ void bar_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

__device__ __forceinline__ uint32_t bar_count(bool p)
{
    uint32_t n;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.popc.u32 %0, 1, %2, p;\n\t}"
                 : "=r"(n)
                 : "r"(uint32_t(p)), "n"(kConsumers)
                 : "memory");
    return n;
}

__device__ __forceinline__ bool bar_any(bool p)
{
    uint32_t n;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(n)
        : "r"(uint32_t(p)), "n"(kConsumers)
        : "memory");
    return n != 0;
}

// Floats in the order of whole numbers (-0 is 0), and back.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// The largest float below that of order o.
__device__ __forceinline__ float below(uint32_t o)
{
    return value_of(o == 0x80000000u ? 0x7ffffffeu : o - 1);  // (0x7fffffff would be -0)
}

__device__ __forceinline__ uint64_t key_of(float x, int token) { return uint64_t(order_of(x)) << 32 | uint32_t(~token); }
__device__ __forceinline__ float key_value(uint64_t k) { return value_of(uint32_t(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) { return int(~uint32_t(k)); }

template <typename T>
__device__ __forceinline__ float element(const uint4& v, int j);
template <>
__device__ __forceinline__ float element<float>(const uint4& v, int j)
{
    return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w);
}
template <>
__device__ __forceinline__ float element<uint16_t>(const uint4& v, int j)
{
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
}

// Element j becomes -inf.
template <typename T>
__device__ __forceinline__ void clear(uint4& v, int j);
template <>
__device__ __forceinline__ void clear<float>(uint4& v, int j)
{
    (j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w) = 0xff800000u;
}
template <>
__device__ __forceinline__ void clear<uint16_t>(uint4& v, int j)
{
    uint32_t& w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    w = j & 1 ? (w & 0xffffu) | 0xff800000u : (w & 0xffff0000u) | 0xff80u;
}

// What of a unit (a row, or a part of one) a thread keeps.
struct Sums {
    float bar;     // logits above it go into the list
    float ref;     // of the sums
    float s, t;
};

// Add four vectors to the sums.
template <typename T, bool kEntropy>
__device__ __forceinline__ void add(Sums& st, const uint4 (&v)[kVecs], Two c_hi, Two c_lo)
{
    const Two ref = two(-st.ref, -st.ref);
    Two s = two(st.s, 0.f), t = two(st.t, 0.f);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        Two x[Elems<T>::kPer / 2];
        Elems<T>::widen(v[k], x);
#pragma unroll
        for (int j = 0; j < Elems<T>::kPer / 2; ++j) {
            const Two d = add2(x[j], ref);
            const Two u = fma2(d, c_hi, mul2(d, c_lo));
            const Two e = exp2_two(u);
            s = add2(s, e);
            if (kEntropy) t = fma2(e, clamp2(u), t);
        }
    }
    float a, b;
    split(s, a, b);
    st.s = a + b;
    if (kEntropy) {
        split(t, a, b);
        st.t = a + b;
    }
}

__device__ __forceinline__ void move(Sums& st, float ref, float c)
{
    Stats a{st.ref, st.s, st.t};
    stats_move(a, ref, c);
    st.ref = a.ref;
    st.s = a.s;
    st.t = a.t;
}

// The sum of all consumers' counts; `turn` goes round the three tallies, of which the one that it starts from is 0.
__device__ __forceinline__ uint32_t count_all(Shared& S, uint32_t mine, uint32_t& turn)
{
    mine = __reduce_add_sync(0xffffffffu, mine);
    const uint32_t next = turn == 2 ? 0 : turn + 1;
    if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&S.tally[turn], mine);
    if (threadIdx.x == 0) S.tally[next] = 0;
    bar_sync();
    const uint32_t n = S.tally[turn];
    turn = next;
    return n;
}

// A key that n to `most` of the list's `count` keys reach; count > most.
__device__ __noinline__ uint64_t select(Shared& S, uint32_t count, uint32_t n, uint32_t most)
{
    uint64_t lo = 0, hi = ~0ull;
    uint32_t turn = 0;
    if (threadIdx.x == 0) S.tally[0] = 0;
    bar_sync();
    while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        uint32_t mine = 0;
        for (uint32_t i = threadIdx.x; i < count; i += kConsumers) mine += S.list[i] >= mid;
        const uint32_t got = count_all(S, mine, turn);
        if (got >= n) {
            lo = mid;
            if (got <= most) break;
        } else {
            hi = mid;
        }
    }
    return lo;
}

// A key below `least` becomes part of the sums, relative to `ref`.
template <bool kEntropy>
__device__ __forceinline__ void lose(Shared& S, uint64_t key, float ref, float c_hi, float c_lo)
{
    const float d = key_value(key) - ref, u = fmaxf(fmaf(d, c_hi, d * c_lo), kLowest), e = exp2_fast(u);
    atomicAdd(&S.lost_s, static_cast<unsigned long long>(double(e) * kLostUnit));
    if (kEntropy) atomicAdd(reinterpret_cast<unsigned long long*>(&S.lost_t),
                            static_cast<unsigned long long>(static_cast<long long>(double(e) * double(u) * kLostUnit)));
}

// Keep the first `count` keys of the list that reach `least`; `before`: those of tokens before it (the others are not
// looked at). The others become part of the sums. Their place is free for more, which `more` puts in.
template <bool kEntropy, typename F>
__device__ __forceinline__ void cut(Shared& S, Sums& st, uint32_t count, uint64_t least, int before, const RowJob& h, F more)
{
    uint64_t mine[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const uint32_t at = threadIdx.x + i * kConsumers;
        mine[i] = at < count ? S.list[at] : 0;
        if (key_token(mine[i]) >= before) mine[i] = 0;
    }
    bar_sync();
    if (threadIdx.x == 0) {
        S.count = 0;
        S.lost_s = 0;
        S.lost_t = 0;
        S.lost_most = 0;
    }
    bar_sync();
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        if (mine[i] >= least) {
            S.list[atomicAdd(&S.count, 1u)] = mine[i];
            mine[i] = 0;
        }
        most = max(most, uint32_t(mine[i] >> 32));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0 && most) atomicMax(&S.lost_most, most);
    move(st, key_value(least), h.c);
    st.bar = st.ref;
    more();
    bar_sync();
    const uint32_t lost = S.lost_most;
    if (lost == 0) return;
    const float ref = value_of(lost);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (mine[i] != 0) lose<kEntropy>(S, mine[i], ref, h.c_hi, h.c_lo);
    bar_sync();
    if (threadIdx.x == 0) {
        Sums one{0.f, ref, float(double(S.lost_s) * (1.0 / kLostUnit)), float(double(S.lost_t) * (1.0 / kLostUnit))};
        move(one, st.ref, h.c);
        st.s += one.s;
        st.t += one.t;
    }
}

// A part of row r is done; true (in all consumers) for the one that is last, which sees what the others have left.
__device__ __forceinline__ bool leave(const TopParams& P, Shared& S, int64_t r, uint32_t part, const TopPart& q)
{
    if (threadIdx.x == 0) P.ws.parts[r * P.parts + part] = q;
    bar_sync();
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atomicAdd(P.ws.tickets + r, 1u) + 1 == uint32_t(P.parts);
        if (last) {
            P.ws.tickets[r] = 0;
            __threadfence();
        }
        S.flag = last;
    }
    bar_sync();
    return S.flag != 0;
}

// The outputs of a row that has no statistics: left out (zeros) or with a status (NaN).
__device__ __forceinline__ void write_none(const TopParams& P, int64_t r, int status)
{
    const sampler_rows_t& a = P.rows;
    const float x = status == SAMPLER_ROW_OK ? 0.f : quiet_nan();
    const int n = P.top.top_n;
    for (int j = threadIdx.x; j < n; j += kConsumers) {
        P.top.out_top_ids[r * n + j] = -1;
        P.top.out_top_logprobs[r * n + j] = x;
    }
    if (threadIdx.x == 0) {
        if (P.top.out_rest_logprob) P.top.out_rest_logprob[r] = x;
        if (a.out_logprob) a.out_logprob[r] = x;
        if (a.out_entropy) a.out_entropy[r] = x;
        if (a.out_status) a.out_status[r] = status;
    }
}

// Warp 0, with the row's `count` largest keys in order and the sums of the rest: its outputs.
template <bool kEntropy>
__device__ __forceinline__ void close_row(const TopParams& P, const uint64_t* sorted, int count, Sums st, const RowJob& h,
                                          int64_t r)
{
    const sampler_rows_t& a = P.rows;
    const int lane = threadIdx.x & 31, n = P.top.top_n;
    const float most = key_value(sorted[0]);
    float s = 0.f, t = 0.f;
    for (int j = lane; j < count; j += 32) {
        const float d = key_value(sorted[j]) - most, u = fmaxf(fmaf(d, h.c_hi, d * h.c_lo), kLowest), e = exp2f(u);
        s += e;
        if (kEntropy) t = fmaf(e, u, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (kEntropy) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    const float rest = st.s, ref = st.ref;
    Stats outside{ref, st.s, st.t};
    stats_move(outside, most, h.c);
    const Stats all{most, s + outside.s, t + outside.t};
    Pair ln_s = log_of(all.s);
    ln_s.lo = fmaf(kExp2Short, __fdividef(outside.s, all.s), ln_s.lo);
    for (int j = lane; j < n; j += 32) {
        const bool there = j < count;
        const uint64_t k = sorted[there ? j : 0];
        P.top.out_top_ids[r * n + j] = there ? key_token(k) : -1;
        P.top.out_top_logprobs[r * n + j] = there ? logprob_of(h, all, key_value(k), ln_s).hi : -pos_inf();
    }
    if (lane == 0) {
        if (P.top.out_rest_logprob) {
            float y = -pos_inf();
            if (rest > 0.f) {
                const Pair q = logprob_of(h, all, ref, ln_s), l = log_of(rest);
                const Pair z = two_sum(q.hi, l.hi);
                y = z.hi + (z.lo + (q.lo + l.lo + kExp2Short));
            }
            P.top.out_rest_logprob[r] = y;
        }
        if (a.out_logprob) a.out_logprob[r] = logprob_of(h, all, h.x_t, ln_s).hi;
        if (a.out_entropy) a.out_entropy[r] = ln_s.hi + fmaf(-kLn2, __fdiv_rn(all.t, all.s), ln_s.lo);
        if (a.out_status) a.out_status[r] = SAMPLER_ROW_OK;
    }
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kThreads, 2) top_kernel(const __grid_constant__ TopParams P)
{
    constexpr int kPer = Elems<T>::kPer;
    extern __shared__ __align__(128) unsigned char ring[];
    Shared& S = *reinterpret_cast<Shared*>(ring + kSlots * kChunkBytes);
    const sampler_rows_t& a = P.rows;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t part = blockIdx.x % P.parts, q = blockIdx.x / P.parts, n_clusters = gridDim.x / P.parts;
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], kWarps);
        }
        queue_open(S.queue, kWarps);
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kWarps) {
        RingPlace slot{0, 0};
        uint32_t issued = 0;
        // (wait_ns 0: nothing begins, and the consumers' waits give up)
        if (P.wait_ns != 0)
            queue_fill<T>(S.queue, a, q, n_clusters, a.out_logprob != nullptr, P.wait_ns, [&](int64_t r) {
                const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
                const RowSpan span = row_span(x, a.vocab);
                const unsigned char* from = reinterpret_cast<const unsigned char*>(x - span.head);
                const int first = int(part) * P.part_vecs, last = min(first + P.part_vecs, span.count);
                for (int v = first; v < last; v += kChunkVecs) {
                    if (!wait(&S.empty[slot.at], slot.phase ^ 1u, P.wait_ns)) return false;
                    const uint32_t bytes = uint32_t(min(kChunkVecs, last - v)) * 16u;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&S.full[slot.at], bytes);
                        bulk_copy_g2s(ring + slot.at * kChunkBytes, from + size_t(v) * 16, bytes, &S.full[slot.at]);
                    }
                    __syncwarp();
                    slot.next(kSlots);
                    ++issued;
                }
                return true;
            });
        // copies in flight land before the CTA may exit
        for (uint32_t j = issued > kSlots ? issued - kSlots : 0; j < issued; ++j)
            wait(&S.full[j % kSlots], j / kSlots & 1u, kWaitNs);
        return;
    }

    const uint32_t n = uint32_t(P.top.top_n);
    const uint32_t trigger = max(256u, 3 * n), about = n + n / 4 + 8;
    RingPlace slot{0, 0};
    QueuePlace place{{0, 0}, 0};
    int64_t done = 0;  // rows that this CTA has ended with
    for (;; ++done) {
        RowItem row;
        // a wait that gives up gives up for all warps
        if (bar_any(!queue_next(S.queue, place, P.wait_ns, row))) break;
        if (row.row < 0) return;
        const int64_t r = row.row;
        if (!row.live) {
            if (part == 0) write_none(P, r, SAMPLER_ROW_OK);
            continue;
        }
        bool failed = false;
        RowJob h;
        h.token = row.token;
        row_scale(h, a, row.temperature);
        const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
        h.x_t = row.x_t;
        const RowSpan span = row_span(x, a.vocab);
        const int first = int(part) * P.part_vecs, last = min(first + P.part_vecs, span.count);
        const int end = span.head + int(a.vocab);  // elements of the span up to the row's end
        const Two c_hi = two(h.c_hi, h.c_hi), c_lo = two(h.c_lo, h.c_lo);
        Sums st{-pos_inf(), -kFloatMax, 0.f, 0.f};
        bool has_n = false, bad = false;
        if (tid == 0) S.count = 0;
        bar_sync();
        for (int base = first; base < last; base += kChunkVecs) {
            bool ok = wait(&S.full[slot.at], slot.phase, P.wait_ns);
            const uint4* chunk = reinterpret_cast<const uint4*>(ring + slot.at * kChunkBytes);
            uint4 v[kVecs];
            auto load = [&] {
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int i = base + k * kConsumers + tid;
                    v[k] = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
                    if (sizeof(T) == 2) v[k] = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
                    if (ok && i < last) {
                        v[k] = chunk[k * kConsumers + tid];
                        const int at = i * kPer;
                        if (at < span.head || at + kPer > end) Elems<T>::mask(v[k], span.head - at, end - at);
                    }
                }
            };
            load();
            float m[kVecs];
#pragma unroll
            for (int k = 0; k < kVecs; ++k) m[k] = Elems<T>::largest(v[k]);
            const float most = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
            bad |= !(most < pos_inf());
            if (!has_n) {
                // n of the threads' largest reach `lo`
                uint32_t lo = order_of(-kFloatMax), hi = order_of(pos_inf());
                const uint32_t mine = order_of(most);
                uint32_t got = bar_count(most >= -kFloatMax);
                if (got >= n) {
                    while (got > about && hi - lo > 1) {
                        const uint32_t mid = lo + (hi - lo) / 2;
                        const uint32_t c = bar_count(mine >= mid);
                        if (c >= n) {
                            lo = mid;
                            got = c;
                        } else {
                            hi = mid;
                        }
                    }
                    has_n = true;
                    move(st, value_of(lo), h.c);
                    st.bar = below(lo);
                }
            }
            const float s_before = st.s, t_before = st.t;
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                if (!(m[k] <= st.bar)) {
                    const int at = (base + k * kConsumers + tid) * kPer - span.head;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const float y = element<T>(v[k], j);
                        if (y > st.bar) {
                            top = atomicAdd(&S.count, 1u) + 1;
                            if (top <= kCap) S.list[top - 1] = key_of(y, at + j);
                            clear<T>(v[k], j);
                        }
                    }
                }
            }
            add<T, kEntropy>(st, v, c_hi, c_lo);
            if (bar_any(top >= trigger || !ok)) {
                failed = bar_any(!ok);
                if (failed) break;
                const uint32_t count = S.count;
                if (count > kCap) {
                    // the list has no place for this chunk: it is cut together with what the list had before
                    st.s = s_before;
                    st.t = t_before;
                    load();
                    const int before = base * kPer - span.head;
                    uint64_t lo = 0, hi = ~0ull;
                    uint32_t turn = 0;
                    if (tid == 0) S.tally[0] = 0;
                    bar_sync();
                    while (hi - lo > 1) {
                        const uint64_t mid = lo + (hi - lo) / 2;
                        uint32_t c = 0;
                        for (int i = tid; i < kCap; i += kConsumers) c += key_token(S.list[i]) < before && S.list[i] >= mid;
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) {
                            const int at = (base + k * kConsumers + tid) * kPer - span.head;
#pragma unroll
                            for (int j = 0; j < kPer; ++j) {
                                const float y = element<T>(v[k], j);
                                c += y > -pos_inf() && key_of(y, at + j) >= mid;
                            }
                        }
                        const uint32_t got = count_all(S, c, turn);
                        if (got >= n) {
                            lo = mid;
                            if (got <= about) break;
                        } else {
                            hi = mid;
                        }
                    }
                    cut<kEntropy>(S, st, kCap, lo, before, h, [&] {
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) {
                            const int at = (base + k * kConsumers + tid) * kPer - span.head;
#pragma unroll
                            for (int j = 0; j < kPer; ++j) {
                                const float y = element<T>(v[k], j);
                                if (y > -pos_inf() && key_of(y, at + j) >= lo) {
                                    S.list[atomicAdd(&S.count, 1u)] = key_of(y, at + j);
                                    clear<T>(v[k], j);
                                }
                            }
                        }
                        add<T, kEntropy>(st, v, c_hi, c_lo);
                    });
                } else {
                    const uint64_t least = select(S, count, n, about);
                    cut<kEntropy>(S, st, count, least, 0x7fffffff, h, [] {});
                }
                has_n = true;
                bar_sync();
            } else if (has_n) {
                st.bar = st.ref;  // later tokens lose ties
            }
            if (lane == 0) mbar_arrive(&S.empty[slot.at]);
            slot.next(kSlots);
        }
        if (failed) break;
        bad = bar_any(bad);
        uint32_t count = S.count;
        if (count > n) {
            const uint64_t least = select(S, count, n, n);
            cut<kEntropy>(S, st, count, least, 0x7fffffff, h, [] {});
            bar_sync();
            count = n;
        }
        // the sums of all threads, in order
        {
            float s = st.s, t = st.t;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                if (kEntropy) t += __shfl_xor_sync(0xffffffffu, t, o);
            }
            if (lane == 0) S.sums[warp] = make_float4(s, t, 0.f, 0.f);
            bar_sync();
            st.s = st.t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                st.s += S.sums[w].x;
                st.t += S.sums[w].y;
            }
        }
        if (P.parts > 1) {
            uint64_t* keys = P.ws.keys + (r * P.parts + part) * kMost;
            if (uint32_t(tid) < count) __stcg(reinterpret_cast<unsigned long long*>(keys + tid), S.list[tid]);
            const bool joins = leave(P, S, r, part, TopPart{st.ref, st.s, st.t, int(count), bad, 0});
            if (!joins) continue;
            // all parts: their keys into the list, their sums in order
            count = 0;
            bool some_failed = false;
            Sums sum{0.f, -kFloatMax, 0.f, 0.f};
            for (int p = 0; p < P.parts; ++p) {
                const volatile TopPart& from = P.ws.parts[r * P.parts + p];
                Sums one{0.f, from.ref, from.s, from.t};
                const uint32_t c = uint32_t(from.count);
                bad |= from.bad != 0;
                some_failed |= from.failed != 0;
                const float ref = fmaxf(sum.ref, one.ref);
                move(sum, ref, h.c);
                move(one, ref, h.c);
                sum.s += one.s;
                sum.t += one.t;
                if (uint32_t(tid) < c)
                    S.list[count + tid] = __ldcg(reinterpret_cast<const unsigned long long*>(P.ws.keys + (r * P.parts + p) * kMost + tid));
                count += c;
            }
            st = sum;
            if (some_failed) {
                write_none(P, r, SAMPLER_ROW_TIMEOUT);
                bar_sync();
                continue;
            }
            bar_sync();
            if (count > n) {
                const uint64_t least = select(S, count, n, n);
                cut<kEntropy>(S, st, count, least, 0x7fffffff, h, [] {});  // (thread 0 has the sums with what is lost)
                count = n;
                if (tid == 0) S.sums[0] = make_float4(st.s, st.t, 0.f, 0.f);
                bar_sync();
                st.s = S.sums[0].x;
                st.t = S.sums[0].y;
            }
        }
        const int status = h.bad_param    ? SAMPLER_ROW_BAD_PARAM
                           : bad          ? SAMPLER_ROW_NONFINITE
                           : count == 0   ? SAMPLER_ROW_ALL_NEG_INF
                                          : SAMPLER_ROW_OK;
        if (status != SAMPLER_ROW_OK) {
            write_none(P, r, status);
            bar_sync();
            continue;
        }
        if (uint32_t(tid) < count) {
            const uint64_t k = S.list[tid];
            uint32_t rank = 0;
            for (uint32_t j = 0; j < count; ++j) rank += S.list[j] > k;
            S.sorted[rank] = k;
        }
        bar_sync();
        if (warp == 0) close_row<kEntropy>(P, S.sorted, int(count), st, h, r);
    }

    // A wait gave up. The rows that this CTA has not ended with are written as TIMEOUT, those that it shares with other
    // CTAs by the last of them.
    RowDealer d;
    dealer_open(d, a, q);
    for (int64_t i = 0;; ++i) {
        bool counts;
        const int64_t r = dealer_next(d, a, q, n_clusters, counts);
        if (r < 0) return;
        if (i < done) continue;
        if (!counts) {
            if (part == 0) write_none(P, r, SAMPLER_ROW_OK);
        } else if (P.parts == 1 || leave(P, S, r, part, TopPart{0.f, 0.f, 0.f, 0, 0, 1})) {
            write_none(P, r, SAMPLER_ROW_TIMEOUT);
        }
    }
}

}  // namespace top

int top_launch(const TopParams& params, int sms, TopGrants* grants, cudaStream_t stream)
{
    using namespace top;
    TopParams p = params;
    const bool bf16 = p.rows.dtype == SAMPLER_DTYPE_BF16, entropy = p.rows.out_entropy != nullptr;
    const int per = bf16 ? 8 : 4;
    const int64_t vecs = (p.rows.vocab + 2 * per - 2) / per;  // the most that a row touches, wherever it starts
    const int64_t slots = 2 * int64_t(sms);
    // parts of a row: as many as give every place on the GPU one, where rows are few; not so small that their joining is
    // what takes the time, and so many that their keys fit the list
    int64_t parts = std::max<int64_t>(1, slots / p.rows.n_rows);
    parts = std::min({parts, int64_t(kCap / p.top.top_n), std::max<int64_t>(1, vecs / 256)});
    if (p.rows.n_rows * parts > kTopUnits) parts = 1;
    p.part_vecs = int((vecs + parts - 1) / parts);
    p.parts = int((vecs + p.part_vecs - 1) / p.part_vecs);
    const auto kernel = bf16 ? entropy ? top_kernel<uint16_t, true> : top_kernel<uint16_t, false>
                             : entropy ? top_kernel<float, true> : top_kernel<float, false>;
    bool& granted = grants->granted[bf16][entropy];
    if (!granted && cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem) != cudaSuccess)
        return SAMPLER_ERR_CUDA;
    granted = true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min(slots / p.parts, p.rows.n_rows) * p.parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
