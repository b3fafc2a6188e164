// top_kernel.cu -- each row's most likely tokens with their logprobs, the mass of all
// others, and with them the logprob of a given token and the entropy.
//
// One pass over a row, in chunks of 16 KB that a producer warp brings into shared memory
// ahead of the eight warps that read them. What is above a bar is put into a list, what
// is not is added up, as 2^((x - ref) c) with ref the bar's value: no exponential is
// above 1, the running maximum is not needed, and the mass outside the top n is a sum
// of its own and not a difference that cancels.
//   The first bar. Of the 256 threads' largest in the first five chunks, the n-th,
//   rounded down to bf16, by counts of two to an instruction. At least n logits reach
//   it. (Of the first chunk alone: 331 us for 281 at 4096 x 128000 bf16, n = 64, and 61 for
//   46 at 517 x 40961 fp32, n = 128, for the many keys that come in a row's first part.)
//   Later bars. A list of `trigger` keys or more goes to the closer, a warp that cuts it
//   down to about n, whose least is the new bar, while the next chunks are read and put
//   theirs into the row's other list; two chunks later what it has left comes back. What
//   falls out is added to the sums as whole multiples of 2^-40 of its largest, so that
//   the order in which the threads come does not matter.
//   Order. A logit and its token are one 64-bit key (the larger logit, then the lower
//   token, is the larger key), so that n keys are always exactly n tokens, whatever ties
//   there are. Tokens of later chunks lose ties, so the bar is passed by `x > bar` alone.
//   Chunks that overflow the list (rows that ascend, ties in the first chunks) are looked
//   at again, an element of each thread at a time, and cut by bisection over keys.
//   A row's end: the closer again, under the next row: the exact n, in order, their
//   logprobs and the row's outputs, and a second look where the others' mass is too little
//   for sums relative to the list.
// Few rows are cut into parts, a CTA each, which leave their n keys and sums in the
// workspace; the part that ends last joins them, parts in order. Short rows are a warp's
// each, with a kernel of their own.
//
// Two CTAs an SM. 4096 x 128000 bf16, n = 64: 281 us, 0.49 of the copy rate. What bounds it
// is the barrier for each chunk, at which all warps wait for the few that have keys to put:
// issue slots are 0.56 busy, warps 0.28 active. (51000 instructions of a warp a row, of which
// exponentials and sums are 14000, loads, peaks and comparisons with the bar 19000, keys and
// cuts 15000.) Tried besides: one CTA of sixteen warps (425 us), four of four (339), two
// chunks for each step (292).
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
constexpr int kProducer = kWarps, kCloser = kWarps + 1;
constexpr int kThreads = kConsumers + 64;
constexpr int kVecs = 4;                        // of a chunk in each consumer
constexpr int kChunkVecs = kConsumers * kVecs;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kSlots = 5;
constexpr int kLook = kSlots;                    // chunks that are looked at for a row's first bar
constexpr int kJobs = 4;                         // of the closer
constexpr int kLane = 8;                         // keys of a list in each of its lanes, at most
constexpr int kClosable = 32 * kLane;            // keys of a list that it takes
constexpr int kMost = SAMPLER_MAX_ALTERNATIVES;
constexpr int kCap = 512;                       // keys in a list
constexpr int kMaxToken = 262143;
constexpr int kMaxTopParts = 8;                 // of a row
constexpr float kLostUnit = 1099511627776.f;    // 2^40

// What the closer is asked for: to cut a list down, to close a row, or to end.
enum JobKind : int { kCut, kClose, kEnd };
struct Job {
    int kind, list, count;
    int ordered;  // kClose: the list is the row's, in order
    int row, token;
    float ref;    // of the sums of what is not in the list
    float bar;    // the list's keys have values of that or above
    float c_hi, c_lo, inv_t, inv_t_lo, x_t;
};

struct Shared {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t ready[kJobs], ended[kJobs];
    uint64_t closed[2];  // the rows that had a pair of lists
    RowQueue queue;
    // two for a row, whose successor has the other two: one is filled, the other is what it is cut into, or what is filled
    // while the closer cuts it
    __align__(16) uint64_t list[4][kCap];
    uint64_t sorted[kMost];
    Job jobs[kJobs];
    uint64_t cut_least;   // what a cut has left: its least key, how many, and the sums of the others
    uint32_t cut_count;
    float cut_ref, cut_s, cut_t;
    __align__(16) uint16_t largest[kConsumers];  // of a chunk, in each thread, in bf16
    float4 state[kConsumers];   // sums, on their way into functions out of line and back
    float2 sums[2][kWarps];     // of a row's consumers, for the closer
    uint32_t tops[kWarps];
    uint32_t tally[3];
    uint32_t count[4];          // keys put into a list (functions out of line)
    uint32_t pushed[4];         // keys put into the row's list since it was last changed; used in turn
    unsigned long long lost_s[kWarps];  // what fell out of a list, relative to the largest of it, in multiples of 2^-40
    long long lost_t[kWarps];
    uint32_t lost_most;                 // its order; 0 between cuts
    uint32_t flag;
    float part_ref[kMaxTopParts], part_s[kMaxTopParts], part_t[kMaxTopParts];
    int part_count[kMaxTopParts], part_flags[kMaxTopParts];
};
constexpr int kSmem = kSlots * kChunkBytes + int(sizeof(Shared));

__device__ __forceinline__ unsigned char* ring_of()
{
    extern __shared__ __align__(128) unsigned char ring[];
    return ring;
}

// (Asked for wherever it is needed, so that functions that stay out of line know it to be in shared memory.)
__device__ __forceinline__ Shared& shared() { return *reinterpret_cast<Shared*>(ring_of() + kSlots * kChunkBytes); }

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

// A bar as vectors are compared with it: `x > bar` for every x of the type.
template <typename T>
__device__ __forceinline__ uint32_t packed_bar(float bar);
template <>
__device__ __forceinline__ uint32_t packed_bar<float>(float bar)
{
    return __float_as_uint(bar);
}
template <>
__device__ __forceinline__ uint32_t packed_bar<uint16_t>(float bar)
{
    uint32_t u = __float_as_uint(bar);  // rounded down: the same bf16 values are above it
    if ((u >> 31) && (u & 0xffffu)) u += 0x10000u;
    u >>= 16;
    return u << 16 | u;
}

// The largest element of a vector, NaN where there is one, as it is compared: fp32 a float, bf16 those of the even and of
// the odd elements.
template <typename T>
struct Peak;
template <>
struct Peak<float> {
    static __device__ __forceinline__ uint32_t none() { return 0xff800000u; }
    static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b)
    {
        return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ bool above(uint32_t a, uint32_t bar) { return __uint_as_float(a) > __uint_as_float(bar); }
    static __device__ __forceinline__ float value(uint32_t a) { return __uint_as_float(a); }
};
template <>
struct Peak<uint16_t> {
    static __device__ __forceinline__ uint32_t none() { return 0xff80ff80u; }
    static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b)
    {
        uint32_t y;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    static __device__ __forceinline__ bool above(uint32_t a, uint32_t bar)
    {
        uint32_t m;
        asm("set.gt.u32.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(bar));
        return m != 0;
    }
    static __device__ __forceinline__ float value(uint32_t a)
    {
        return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    }
};

template <typename T>
__device__ __forceinline__ uint32_t peak(const uint4& v)
{
    return Peak<T>::join(Peak<T>::join(v.x, v.y), Peak<T>::join(v.z, v.w));
}

// Which elements of a vector are above the bar (a bit for each); those become -inf.
template <typename T>
__device__ __forceinline__ uint32_t take_above(uint4& v, uint32_t bar);
template <>
__device__ __forceinline__ uint32_t take_above<float>(uint4& v, uint32_t bar)
{
    const float b = __uint_as_float(bar);
    uint32_t bits = 0;
    auto word = [&](uint32_t& w, uint32_t bit) {
        if (__uint_as_float(w) > b) {
            w = 0xff800000u;
            bits |= bit;
        }
    };
    word(v.x, 1u);
    word(v.y, 2u);
    word(v.z, 4u);
    word(v.w, 8u);
    return bits;
}
template <>
__device__ __forceinline__ uint32_t take_above<uint16_t>(uint4& v, uint32_t bar)
{
    uint32_t bits = 0;
    auto word = [&](uint32_t& w, int shift) {
        uint32_t m;  // 0xffff in each half that is above
        asm("set.gt.u32.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w), "r"(bar));
        w = (w & ~m) | (0xff80ff80u & m);
        bits |= ((m & 1u) | (m >> 15 & 2u)) << shift;
    };
    word(v.x, 0);
    word(v.y, 2);
    word(v.z, 4);
    word(v.w, 6);
    return bits;
}

// What of a unit (a row, or a part of one) a thread keeps.
struct Sums {
    float bar;     // logits above it go into the list
    float ref;     // of the sums
    float s, t;
};

// Add four vectors to the sums. (By log2(e) / T as one float, c, the nearest. The pair takes 6 % longer: 4096 x 128000
// bf16, n = 64, 324 us for 306 with a cold L2. Mean errors of 2048 logprobs of rows of 128000 bf16 whose mass is 8 nats
// below one token: 0.8e-7 at T = 1.44, where the product of rounded log2(e) and 1 / T, 1.9 units of 2^-24 off, had -7.4e-7;
// 0.7 and 7.5e-7 at T = 0.7195. sampler_score, which moves its sums by that product, has -7.2e-7 and 6.4e-7.)
template <typename T, bool kEntropy>
__device__ __forceinline__ void add(Sums& st, const uint4 (&v)[kVecs], Two c)
{
    const Two ref = two(-st.ref, -st.ref);
    Two s = two(0.f, 0.f), t = s;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        Two x[Elems<T>::kPer / 2];
        Elems<T>::widen(v[k], x);
#pragma unroll
        for (int j = 0; j < Elems<T>::kPer / 2; ++j) {
            const Two u = mul2(add2(x[j], ref), c);
            const Two e = exp2_two(u);
            s = add2(s, e);
            if (kEntropy) t = fma2(e, clamp2(u), t);
        }
    }
    // (four vectors by themselves first: the roundings of long sums of equal terms go one way)
    float a, b;
    split(s, a, b);
    st.s += a + b;
    if (kEntropy) {
        split(t, a, b);
        st.t += a + b;
    }
}

// The sums relative to a higher reference; a lower one is not taken. (A list's keys may be below the reference: what came in
// before a cut ended, and what parts leave that are far below another. A key that some of those reach may be, too, and sums
// relative to it beyond all numbers.)
__device__ __forceinline__ void move(Sums& st, float ref, const Scale& q)
{
    Stats a{st.ref, st.s, st.t};
    stats_move(a, fmaxf(ref, st.ref), q);
    st.ref = a.ref;
    st.s = a.s;
    st.t = a.t;
}

// The sum of all consumers' counts; `turn` goes round the three tallies, of which the one that it starts from is 0.
__device__ __forceinline__ uint32_t count_all(uint32_t mine, uint32_t& turn)
{
    Shared& S = shared();
    mine = __reduce_add_sync(0xffffffffu, mine);
    const uint32_t next = turn == 2 ? 0 : turn + 1;
    if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&S.tally[turn], mine);
    if (threadIdx.x == 0) S.tally[next] = 0;
    bar_sync();
    const uint32_t n = S.tally[turn];
    turn = next;
    return n;
}

// A key that n to `most` of the first `count` keys of a list reach; count > most. A bisection, over the values first and,
// where ties do not leave it a number in between, over the tokens of the value that it ends at. (Each step is a barrier
// that counts, of a key in each thread; longer lists take the tallies.) What has been put into the list before is seen
// by all after it.
__device__ __forceinline__ uint64_t select(const uint64_t* list, uint32_t count, uint32_t n, uint32_t most)
{
    Shared& S = shared();
    const int tid = threadIdx.x;
    const bool single = count <= uint32_t(kConsumers);
    const uint64_t mine = uint32_t(tid) < count ? list[tid] : 0;
    uint32_t top = uint32_t(mine >> 32), turn = 0;
    for (uint32_t i = tid + kConsumers; i < count; i += kConsumers) top = max(top, uint32_t(list[i] >> 32));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) S.tops[tid >> 5] = top;
    if (tid == 0) S.tally[0] = 0;
    bar_sync();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, S.tops[w]);
    auto reach = [&](uint64_t key) {
        if (single) return bar_count(mine >= key);
        uint32_t c = 0;
        for (uint32_t i = tid; i < count; i += kConsumers) c += list[i] >= key;
        return count_all(c, turn);
    };
    uint64_t lo = uint64_t(order_of(-kFloatMax)) << 32, hi = (uint64_t(top) + 1) << 32, step = 1ull << (32 + 21);
    bool found = false;  // a lower end that is near: steps down from the top, each four times the one before
    for (int part = 0; part < 2; ++part) {
        const uint64_t last = part == 0 ? 1ull << 32 : 1;
#pragma unroll 1
        while (hi - lo > last) {
            uint64_t mid = lo + ((hi - lo) / 2 & ~(last - 1));
            if (!found && step != 0 && step < hi - lo) mid = max(mid, hi - step);
            step <<= 2;  // (0 at last: halves from then on)
            const uint32_t got = reach(mid);
            if (got >= n) {
                lo = mid;
                found = true;
                if (got <= most) return mid;
            } else {
                hi = mid;
            }
        }
        if (part == 0) lo |= uint32_t(~uint32_t(kMaxToken));  // the lowest key of the value
    }
    return lo;
}

// The next `want` places in a list for a lane by itself. (Written so that the lanes that want some, a few of a warp, are
// not put together first.)
__device__ __forceinline__ uint32_t next_places(uint32_t* count, uint32_t want)
{
    uint32_t at;
    asm volatile("atom.shared.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(smem_addr(count)), "r"(want) : "memory");
    return at;
}

// Places in a list for the lanes of a warp that want one (kCap and above: there is none); the warp is whole.
__device__ __forceinline__ uint32_t places(uint32_t* count, bool want)
{
    const uint32_t lanes = __ballot_sync(0xffffffffu, want), lane = threadIdx.x & 31;
    uint32_t first = 0;
    if (lane == 0 && lanes) first = atomicAdd(count, uint32_t(__popc(lanes)));
    return __shfl_sync(0xffffffffu, first, 0) + __popc(lanes & ((1u << lane) - 1u));
}

// Those of the first `count` keys of a list for which goes(key, the place in turn) become part of thread 0's sums, as
// whole multiples of 2^-40 of the largest of them, so that it does not matter in what order they are. S.lost_most is
// their largest order, seen by all.
template <bool kEntropy, typename F>
__device__ __forceinline__ void lose(const uint64_t* from, uint32_t count, Sums& st, const Scale& q, F goes)
{
    Shared& S = shared();
    const int tid = threadIdx.x;
    const uint32_t lost = S.lost_most;
    if (lost == 0) return;
    const float ref = value_of(lost);
    unsigned long long s = 0;
    long long t = 0;
#pragma unroll 1
    for (uint32_t i = tid; i < count; i += kConsumers) {
        const uint64_t k = from[i];
        if (!goes(k)) continue;
        const float d = key_value(k) - ref, u = fmaxf(fmaf(d, q.c_hi, d * q.c_lo), kLowest), e = exp2_fast(u);
        s += __float2ull_rn(e * kLostUnit);
        if (kEntropy) t += __float2ll_rn(e * u * kLostUnit);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (kEntropy) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if ((tid & 31) == 0) {
        S.lost_s[tid >> 5] = s;
        S.lost_t[tid >> 5] = t;
    }
    bar_sync();
    if (tid == 0) {
        s = 0;
        t = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s += S.lost_s[w];
            t += S.lost_t[w];
        }
        Sums one{0.f, ref, __ull2float_rn(s) * (1.f / kLostUnit), __ll2float_rn(t) * (1.f / kLostUnit)};
        move(one, st.ref, q);
        st.s += one.s;
        st.t += one.t;
        S.lost_most = 0;
    }
}

// The n largest of a list's first `count` keys (as many as there are threads at most), in order, into `to`; the others
// become part of thread 0's sums. Each thread counts the keys above its own. (Ends without a barrier for S.lost_most,
// which the next use comes two barriers after.)
template <bool kEntropy>
__device__ __forceinline__ void rank(const uint64_t* from, uint32_t count, uint32_t n, uint64_t* to, Sums& st, const Scale& q)
{
    Shared& S = shared();
    const uint32_t tid = threadIdx.x;
    if ((tid & ~31u) < count) {
        const uint64_t mine = tid < count ? from[tid] : 0;
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(from);
        uint32_t above = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < count / 2; ++j) {
            const ulonglong2 k = pairs[j];
            above += k.x > mine;
            above += k.y > mine;
        }
        if (count & 1) above += from[count - 1] > mine;
        const bool stays = above < n;
        if (tid < count && stays) to[above] = mine;
        const uint32_t most = __reduce_max_sync(0xffffffffu, stays ? 0 : uint32_t(mine >> 32));
        if ((tid & 31) == 0 && most) atomicMax(&S.lost_most, most);
    }
    bar_sync();
    if (count <= n) return;
    const uint64_t least = to[n - 1];
    move(st, key_value(least), q);
    st.bar = st.ref;
    lose<kEntropy>(from, count, st, q, [&](uint64_t k) { return k < least; });
}

// Cuts the first `count` keys of list `at` into the other one, which is empty: those that reach `least`. The others
// become part of thread 0's sums. List `at` is then empty, and the other one is seen by all. (Between two cuts there is
// a select.)
template <bool kEntropy>
__device__ __forceinline__ void cut(uint32_t at, uint32_t count, uint64_t least, Sums& st, const Scale& q)
{
    Shared& S = shared();
    const int tid = threadIdx.x;
    const uint64_t* from = S.list[at];
    uint32_t most = 0;
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < count; i0 += kConsumers) {
        const uint64_t k = i0 + tid < count ? from[i0 + tid] : 0;
        const bool stays = k >= least;
        const uint32_t to = places(&S.count[at ^ 1], stays);
        if (stays)
            S.list[at ^ 1][to] = k;
        else
            most = max(most, uint32_t(k >> 32));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((tid & 31) == 0 && most) atomicMax(&S.lost_most, most);
    move(st, key_value(least), q);
    st.bar = st.ref;
    bar_sync();
    lose<kEntropy>(from, count, st, q, [&](uint64_t k) { return k < least; });
    if (tid == 0) S.count[at] = 0;
}

// A list that is longer than there are threads is cut down to n to `most` keys. Sums come and go in S.state; the list that
// is filled in the end is returned.
template <bool kEntropy>
__device__ __noinline__ uint32_t cut_long(uint32_t at, uint32_t count, uint32_t n, uint32_t most, float c_hi, float c_lo)
{
    Shared& S = shared();
    const float4 in = S.state[threadIdx.x];
    Sums st{in.x, in.y, in.z, in.w};
    const uint64_t least = select(S.list[at], count, n, most);
    cut<kEntropy>(at, count, least, st, Scale{c_hi, c_lo});
    S.state[threadIdx.x] = make_float4(st.bar, st.ref, st.s, st.t);
    bar_sync();
    return at ^ 1;
}

// Adds 1 to each half of `count` (in bf16) whose value of `a` is above `b`'s.
__device__ __forceinline__ void count_above(uint32_t& count, uint32_t a, uint32_t b)
{
    uint32_t one;
    asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(one) : "r"(a), "r"(b));
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(count) : "r"(one));
}

// Where a chunk of a row is: its place in the ring, the first of its vectors in the span, the end of the part's, and the
// span's elements that the row begins and ends at.
struct Chunk {
    int at, base, last, head, end;
};

template <typename T>
__device__ __forceinline__ void load(uint4 (&v)[kVecs], const Chunk& p)
{
    constexpr int kPer = Elems<T>::kPer;
    const uint4* in = reinterpret_cast<const uint4*>(ring_of() + p.at) + threadIdx.x;
    const uint32_t none = Peak<T>::none();
    if (p.base + kChunkVecs <= p.last && p.base * kPer >= p.head && (p.base + kChunkVecs) * kPer <= p.end) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) v[k] = in[k * kConsumers];
        return;
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int i = k * kConsumers + int(threadIdx.x);
        v[k] = make_uint4(none, none, none, none);
        if (p.base + i < p.last) {
            v[k] = in[k * kConsumers];
            const int at = (p.base + i) * kPer;
            if (at < p.head || at + kPer > p.end) Elems<T>::mask(v[k], p.head - at, p.end - at);
        }
    }
}

// The list has had no place for all that a chunk put into it (rows that rise, ties in the first chunk). What it had
// before is kept, and the chunk's elements are looked at again, one of each thread at a time, as keys. Sums come and go
// in S.state (before the chunk; after it); the list that is filled in the end is returned.
template <typename T, bool kEntropy>
__device__ __noinline__ uint32_t slow_chunk(uint32_t at, uint32_t valid, int chunk_at, int base, int last, int head, int end,
                                            uint32_t n, float c_hi, float c_lo)
{
    constexpr int kPer = Elems<T>::kPer;
    Shared& S = shared();
    const int tid = threadIdx.x, before = base * kPer - head;
    const Scale q{c_hi, c_lo};
    const float4 in = S.state[tid];
    Sums st{in.x, in.y, in.z, in.w};
    bar_sync();
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < valid; i0 += kConsumers) {
        const uint64_t k = i0 + tid < valid ? S.list[at][i0 + tid] : 0;
        const bool stays = k != 0 && key_token(k) < before;
        const uint32_t to = places(&S.count[at ^ 1], stays);
        if (stays) S.list[at ^ 1][to] = k;
    }
    bar_sync();
    if (tid == 0) S.count[at] = 0;
    at ^= 1;
    uint64_t least = st.bar > -pos_inf() ? uint64_t(order_of(st.bar) + 1) << 32 : 0;  // (of the list, where it has n keys)
    const T* x = reinterpret_cast<const T*>(ring_of() + chunk_at);
#pragma unroll 1
    for (int e = 0;; ++e) {
        // Room for a key of each thread. (What was there before may leave none: the keys of a cut that has just come back, and
        // those that were put in meanwhile, are up to kCap.) In the end the list is cut down in any case.
        const bool end_of_chunk = e == kVecs * kPer;
        const uint32_t count = S.count[at];
        if (count > (end_of_chunk ? n : uint32_t(kCap - kConsumers))) {
            least = select(S.list[at], count, n, n + n / 4 + 8 < count ? n + n / 4 + 8 : n);
            cut<kEntropy>(at, count, least, st, q);
            at ^= 1;
        }
        bar_sync();
        if (end_of_chunk) break;
        const int i = e / kPer * kConsumers + tid, j = (base + i) * kPer + e % kPer;
        const bool there = base + i < last && j >= head && j < end;
        const float y = there ? load_logit(x + i * kPer + e % kPer) : -pos_inf();
        const uint64_t k = key_of(y, j - head);
        const bool wants = y > -pos_inf() && k >= least;
        const uint32_t to = places(&S.count[at], wants);
        if (wants) {
            S.list[at][to] = k;
        } else {
            const float d = y - st.ref, u = fmaf(d, q.c_hi, d * q.c_lo), f = exp2_fast(u);
            st.s += f;
            if (kEntropy) st.t = fmaf(f, fmaxf(u, kLowest), st.t);
        }
        bar_sync();
    }
    S.state[tid] = make_float4(st.bar, st.ref, st.s, st.t);
    return at;
}

// A part of row r is done; true (in all consumers) for the one that is last, which sees what the others have left.
__device__ __forceinline__ bool leave(const TopParams& P, int64_t r, uint32_t part, const TopPart& q)
{
    Shared& S = shared();
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
__device__ __forceinline__ void write_none(const TopParams& P, int64_t r, int status, int thread, int threads)
{
    const sampler_rows_t& a = P.rows;
    const float x = status == SAMPLER_ROW_OK ? 0.f : quiet_nan();
    const int n = P.top.top_n;
    for (int j = thread; j < n; j += threads) {
        P.top.out_top_ids[r * n + j] = -1;
        P.top.out_top_logprobs[r * n + j] = x;
    }
    if (thread == 0) {
        if (P.top.out_rest_logprob) P.top.out_rest_logprob[r] = x;
        if (a.out_logprob) a.out_logprob[r] = x;
        if (a.out_entropy) a.out_entropy[r] = x;
        if (a.out_status) a.out_status[r] = status;
    }
}

__device__ __forceinline__ void write_none(const TopParams& P, int64_t r, int status)
{
    write_none(P, r, status, int(threadIdx.x), kConsumers);
}

// The mass outside a row's list is added up relative to references that are the n-th key's value in the end, and no term
// is kept that is below 2^-126 of those: 2^-108 of a row is lost at most. Below this much the sum is not good for its
// digits (2^-24 of it), and the row is looked at again.
constexpr float kFaint = 5.169878828e-26f;  // 2^-84

// The sum of what is below the value of key `least`, relative to its own largest (x: the reference, y: the sum, 0 where
// there is none); a whole warp. (Where a list is as long as was asked for and what is outside is faint, there are no ties
// with the key. Rows like that come with a low temperature and a short list, or where all tokens but a few are forbidden.
// One of 151936 bf16 takes 49 us more; 4096 x 128000 bf16, n = 1, T = 0.05, all of them such: 703 us, without any 232.)
template <typename T>
__device__ __noinline__ float2 far_outside(const TopParams& P, int64_t r, uint64_t least, float c_hi, float c_lo)
{
    constexpr int kPer = Elems<T>::kPer, kAhead = 8;
    const sampler_rows_t& a = P.rows;
    const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
    const RowSpan span = row_span(x, a.vocab);
    const uint4* from = reinterpret_cast<const uint4*>(x - span.head);
    const int lane = threadIdx.x & 31, end = span.head + int(a.vocab);
    const uint32_t none = Peak<T>::none(), bar = packed_bar<T>(below(uint32_t(least >> 32)));
    const Scale q{c_hi, c_lo};
    Stats st = stats_empty();
    bool bad = false;
    for (int base = lane; base < span.count; base += 32 * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = base + 32 * k;
            v[k] = i < span.count ? __ldg(from + i) : make_uint4(none, none, none, none);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int at = (base + 32 * k) * kPer;
            if (at < span.head || at + kPer > end) Elems<T>::mask(v[k], span.head - at, end - at);
            take_above<T>(v[k], bar);
        }
        fold<T, false, kAhead>(st, bad, v, two(c_hi, c_hi), two(c_lo, c_lo), q);
    }
    stats_warp<false>(st, q);
    return make_float2(st.ref, st.s);
}

// The closer (a warp), with a row's `count` largest keys in order and the sums of the rest: its outputs.
template <typename T, bool kEntropy>
__device__ __forceinline__ void close_row(const TopParams& P, const uint64_t* sorted, int count, const Sums& st,
                                          const RowJob& h, int64_t r)
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
    float rest = st.s, ref = st.ref;
    Sums outside = st;
    move(outside, most, Scale{h.c_hi, h.c_lo});
    const Stats all{most, s + outside.s, t + outside.t};
    Pair ln_s = log_of(all.s);
    ln_s.lo = fmaf(kExp2Short, __fdividef(outside.s, all.s), ln_s.lo);
    for (int j = lane; j < n; j += 32) {
        const bool there = j < count;
        const uint64_t k = sorted[there ? j : 0];
        P.top.out_top_ids[r * n + j] = there ? key_token(k) : -1;
        P.top.out_top_logprobs[r * n + j] = there ? logprob_of(h, all, key_value(k), ln_s).hi : -pos_inf();
    }
    // (fewer keys than n: the row has no others above -inf)
    if (P.top.out_rest_logprob && rest < kFaint && count == n) {
        const float2 far = far_outside<T>(P, r, sorted[n - 1], h.c_hi, h.c_lo);
        ref = far.x;
        rest = far.y;
    }
    if (lane == 0) {
        if (P.top.out_rest_logprob) {
            float y = -pos_inf();
            if (rest > 0.f) {
                const Pair q = logprob_of(h, all, ref, ln_s), l = log_of(rest);
                const Pair z = two_sum(q.hi, l.hi);
                if (q.hi >= -kFloatMax) y = z.hi + (z.lo + (q.lo + l.lo + kExp2Short));  // (else below fp32's range)
            }
            P.top.out_rest_logprob[r] = y;
        }
        if (a.out_logprob) a.out_logprob[r] = logprob_of(h, all, h.x_t, ln_s).hi;
        if (a.out_entropy) a.out_entropy[r] = ln_s.hi + fmaf(-kLn2, __fdiv_rn(all.t, all.s), ln_s.lo);
        if (a.out_status) a.out_status[r] = SAMPLER_ROW_OK;
    }
}

// ---------------------------------------------------------------- the closer
// A list of up to 32 * kLane keys in a warp's lanes.
struct Keys {
    uint64_t k[kLane];
};

__device__ __forceinline__ void take_keys(Keys& a, const uint64_t* list, int count)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kLane; ++i) a.k[i] = lane + 32 * i < count ? list[lane + 32 * i] : 0;
}

__device__ __forceinline__ uint32_t reaching(const Keys& a, uint64_t key)
{
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < kLane; ++i) c += a.k[i] >= key;
    return __reduce_add_sync(0xffffffffu, c);
}

// How many reach each of three orders, ten bits for each.
__device__ __forceinline__ uint32_t reaching(const Keys& a, uint32_t o1, uint32_t o2, uint32_t o3)
{
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
        const uint32_t o = uint32_t(a.k[i] >> 32);
        c += (o >= o1 ? 1u : 0u) + (o >= o2 ? 1u << 10 : 0u) + (o >= o3 ? 1u << 20 : 0u);
    }
    return __reduce_add_sync(0xffffffffu, c);
}

// As select: a key that n to `most` of the lanes' keys reach (exact), or that at least n reach and no other value's with
// fewer (not exact: more than `most` where ties are). There are more than `most` keys, all of order `lo` or above. The
// values' steps cut the range in four.
__device__ __forceinline__ uint64_t select_warp(const Keys& a, uint32_t n, uint32_t most, bool exact, uint32_t lo)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kLane; ++i) top = max(top, uint32_t(a.k[i] >> 32));
    uint32_t hi = __reduce_max_sync(0xffffffffu, top) + 1;
#pragma unroll 1
    while (hi - lo > 1) {
        const uint32_t q = max((hi - lo) / 4, 1u), o1 = lo + q, o2 = min(o1 + q, hi), o3 = min(o2 + q, hi);
        const uint32_t got = reaching(a, o1, o2, o3), c1 = got & 1023u, c2 = got >> 10 & 1023u, c3 = got >> 20;
        uint32_t c;
        if (c3 >= n) {
            lo = o3;
            c = c3;
        } else if (c2 >= n) {
            lo = o2;
            hi = o3;
            c = c2;
        } else if (c1 >= n) {
            lo = o1;
            hi = o2;
            c = c1;
        } else {
            hi = o1;
            continue;
        }
        if (c <= most) return uint64_t(lo) << 32;
    }
    if (!exact) return uint64_t(lo) << 32;
    // among the tokens of that value: the lowest n of them that are still wanted
    uint64_t l = uint64_t(lo) << 32 | uint32_t(~uint32_t(kMaxToken)), h = uint64_t(lo + 1) << 32;
#pragma unroll 1
    while (h - l > 1) {
        const uint64_t mid = l + (h - l) / 2;
        const uint32_t got = reaching(a, mid);
        if (got >= n) {
            l = mid;
            if (got <= most) break;
        } else {
            h = mid;
        }
    }
    return l;
}

// The keys that reach `least` go to the front of the list; the sums of the others, relative to their largest, as whole
// multiples of 2^-40. Their number.
template <bool kEntropy>
__device__ __forceinline__ int split_keys(const Keys& a, uint64_t least, uint64_t* list, const Scale& q, Sums& lost)
{
    const int lane = threadIdx.x & 31;
    int count = 0;
    uint32_t most = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
        const bool stays = a.k[i] >= least;
        const uint32_t lanes = __ballot_sync(0xffffffffu, stays);
        if (stays)
            list[count + __popc(lanes & ((1u << lane) - 1u))] = a.k[i];
        else
            most = max(most, uint32_t(a.k[i] >> 32));
        count += __popc(lanes);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    lost = Sums{0.f, -kFloatMax, 0.f, 0.f};
    if (most != 0) {
        lost.ref = value_of(most);
        unsigned long long s = 0;
        long long t = 0;
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
            if (a.k[i] >= least || a.k[i] == 0) continue;
            const float d = key_value(a.k[i]) - lost.ref, u = fmaxf(fmaf(d, q.c_hi, d * q.c_lo), kLowest), e = exp2_fast(u);
            s += __float2ull_rn(e * kLostUnit);
            if (kEntropy) t += __float2ll_rn(e * u * kLostUnit);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            if (kEntropy) t += __shfl_xor_sync(0xffffffffu, t, o);
        }
        lost.s = __ull2float_rn(s) * (1.f / kLostUnit);
        lost.t = __ll2float_rn(t) * (1.f / kLostUnit);
    }
    __syncwarp();
    return count;
}

// The keys at the front of a list in order.
__device__ __forceinline__ void sort_keys(const uint64_t* list, int count, uint64_t* to)
{
    const int lane = threadIdx.x & 31;
    uint64_t mine[kMost / 32];
    int rank[kMost / 32];
#pragma unroll
    for (int i = 0; i < kMost / 32; ++i) {
        mine[i] = lane + 32 * i < count ? list[lane + 32 * i] : 0;
        rank[i] = 0;
    }
    if (count <= 32) {
#pragma unroll 4
        for (int j = 0; j < count; ++j) rank[0] += list[j] > mine[0];
    } else {
#pragma unroll 2
        for (int j = 0; j < count; ++j) {
            const uint64_t k = list[j];
#pragma unroll
            for (int i = 0; i < kMost / 32; ++i) rank[i] += k > mine[i];
        }
    }
#pragma unroll
    for (int i = 0; i < kMost / 32; ++i)
        if (lane + 32 * i < count) to[rank[i]] = mine[i];
    __syncwarp();
}

// A row that is done, of whose list (of 32 * kLane keys at most, none below `bar`) n at most are wanted; a whole warp.
template <typename T, bool kEntropy>
__device__ __forceinline__ void close_list(const TopParams& P, uint64_t* list, int count, uint64_t* sorted, float bar, Sums st,
                                           const RowJob& h, int64_t r)
{
    const uint32_t n = uint32_t(P.top.top_n);
    if (uint32_t(count) > n) {
        Keys keys;
        take_keys(keys, list, count);
        const uint64_t least = select_warp(keys, n, n, true, order_of(bar));
        Sums lost;
        const Scale q{h.c_hi, h.c_lo};
        count = split_keys<kEntropy>(keys, least, list, q, lost);
        // (relative to the largest of both and not to the list's least, which may be far above)
        const float ref = fmaxf(st.ref, lost.ref);
        move(st, ref, q);
        move(lost, ref, q);
        st.s += lost.s;
        st.t += lost.t;
    }
    sort_keys(list, count, sorted);
    close_row<T, kEntropy>(P, sorted, count, st, h, r);
}

template <typename T, bool kEntropy>
__device__ __forceinline__ void run_closer(const TopParams& P)
{
    Shared& S = shared();
    const int lane = threadIdx.x & 31;
    const uint32_t n = uint32_t(P.top.top_n);
    for (uint32_t j = 0;; ++j) {
        const uint32_t slot = j % kJobs;
        // (the consumers give up before it does, and say so)
        if (!wait(&S.ready[slot], j / kJobs & 1u, 8 * kWaitNs)) return;
        const Job job = S.jobs[slot];
        if (job.kind == kEnd) return;
        const Scale q{job.c_hi, job.c_lo};
        uint64_t* list = S.list[job.list];
        int count = job.count;
        if (job.kind == kCut) {
            Keys keys;
            take_keys(keys, list, count);
            const uint64_t least = select_warp(keys, n, n + n / 4 + 8, false, order_of(job.bar));
            Sums lost;
            count = split_keys<kEntropy>(keys, least, list, q, lost);
            if (lane == 0) {
                S.cut_least = least;
                S.cut_count = uint32_t(count);
                S.cut_ref = lost.ref;
                S.cut_s = lost.s;
                S.cut_t = lost.t;
            }
        } else {
            Sums st{0.f, job.ref, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {  // in order
                st.s += S.sums[job.list >> 1][w].x;
                st.t += S.sums[job.list >> 1][w].y;
            }
            RowJob h;
            h.token = job.token;
            h.x_t = job.x_t;
            h.c_hi = job.c_hi;
            h.c_lo = job.c_lo;
            h.inv_t = job.inv_t;
            h.inv_t_lo = job.inv_t_lo;
            if (job.ordered)
                close_row<T, kEntropy>(P, list, count, st, h, job.row);
            else
                close_list<T, kEntropy>(P, list, count, S.sorted, job.bar, st, h, job.row);
        }
        __syncwarp();
        if (lane == 0) {
            if (job.kind == kClose) mbar_arrive(&S.closed[job.list >> 1]);
            mbar_arrive(&S.ended[slot]);
        }
    }
}

// Whether job j has ended; a whole warp. (Job -1 and before: there is none. The job that has its place after it must not
// have been asked for.)
__device__ __forceinline__ bool wait_job(int j, uint64_t ns)
{
    return j < 0 || wait(&shared().ended[j % kJobs], uint32_t(j / kJobs) & 1u, ns);
}

// Asks for job j; a whole warp, of which lane 0 has it. False where a wait gave up.
__device__ __forceinline__ bool post_job(int j, const Job& job, uint64_t ns)
{
    Shared& S = shared();
    const bool ok = wait_job(j - kJobs, ns);
    if (ok && (threadIdx.x & 31) == 0) {
        S.jobs[j % kJobs] = job;
        mbar_arrive(&S.ready[j % kJobs]);
    }
    __syncwarp();
    return ok;
}

// The last part of a row joins them all: its largest keys, in order, are then in list `at` + 1, and the others' sums
// thread 0's, in S.state. How many keys; -1: a part has failed; -2: it has a NaN or +inf.
template <bool kEntropy>
__device__ __noinline__ int join_parts(const TopParams& P, int64_t r, uint32_t at, float c_hi, float c_lo)
{
    Shared& S = shared();
    const int tid = threadIdx.x, parts = P.parts;
    const uint32_t n = uint32_t(P.top.top_n);
    const Scale q{c_hi, c_lo};
    if (tid < 2) S.count[at + tid] = 0;
    // all that the parts have left at once: the keys' places, two a thread (kCap at most), before their numbers are known (32 x 151936 bf16
    // in eight parts, n = 20: 16.5 us; one part after the other 17.5)
    uint64_t key[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t i = uint32_t(tid + j * kConsumers), p = i / n;
        key[j] = p < uint32_t(parts)
                     ? __ldcg(reinterpret_cast<const unsigned long long*>(P.ws.keys + (r * parts + p) * kMost + i % n))
                     : 0;
    }
    if (tid < parts) {
        const volatile TopPart& from = P.ws.parts[r * parts + tid];
        S.part_ref[tid] = from.ref;
        S.part_s[tid] = from.s;
        S.part_t[tid] = from.t;
        S.part_count[tid] = from.count;
        S.part_flags[tid] = (from.bad ? 1 : 0) | (from.failed ? 2 : 0);
    }
    bar_sync();
    // keys into the list; the parts' sums, in order, are thread 0's
    uint32_t count = 0;
    int flags = 0;
    Sums st{0.f, -kFloatMax, 0.f, 0.f};
    for (int p = 0; p < parts; ++p) {
        const uint32_t c = uint32_t(S.part_count[p]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t i = uint32_t(tid + j * kConsumers) - uint32_t(p) * n;  // (of this part's)
            if (i < c) S.list[at][count + i] = key[j];
        }
        count += c;
        flags |= S.part_flags[p];
        st.ref = fmaxf(st.ref, S.part_ref[p]);
    }
    for (int p = 0; p < parts; ++p) {
        Sums one{0.f, S.part_ref[p], S.part_s[p], S.part_t[p]};
        move(one, st.ref, q);
        st.s += tid == 0 ? one.s : 0.f;
        st.t += tid == 0 ? one.t : 0.f;
    }
    bar_sync();
    if (flags) return flags & 2 ? -1 : -2;
    if (count > uint32_t(kConsumers)) {
        // More than are ranked at once. A bar for them all: of the first of each part's (which are in order), as many as
        // there are threads, the n-th. What does not reach it is lost. (17 rows of 18557 bf16 in five parts, n = 99: 18 us
        // in place of 28 by bisection.)
        const uint32_t each = uint32_t(kConsumers / parts), p = uint32_t(tid) / each, i = uint32_t(tid) % each;
        uint32_t before = 0;
        for (uint32_t k = 0; k < p && k < uint32_t(parts); ++k) before += uint32_t(S.part_count[k]);
        const bool there = p < uint32_t(parts) && i < uint32_t(S.part_count[p]);
        const uint64_t mine = there ? S.list[at][before + i] : 0;
        S.list[at + 1][tid] = mine;
        if (tid == 0) S.cut_least = 0;
        bar_sync();
        uint32_t above = 0;
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(S.list[at + 1]);
#pragma unroll 8
        for (int j = 0; j < kConsumers / 2; ++j) {
            const ulonglong2 k = pairs[j];
            above += k.x > mine;
            above += k.y > mine;
        }
        if (there && above == n - 1) S.cut_least = mine;
        bar_sync();
        const uint64_t least = S.cut_least;
        uint32_t from = at;
        if (least != 0) {
            cut<kEntropy>(at, count, least, st, q);
            bar_sync();
            count = S.count[at + 1];
            from = at + 1;
        }
        if (count > uint32_t(kConsumers)) {
            S.state[tid] = make_float4(st.bar, st.ref, st.s, st.t);
            from = cut_long<kEntropy>(from, count, n, n, c_hi, c_lo);
            const float4 in = S.state[tid];
            st = Sums{in.x, in.y, in.z, in.w};
            count = n;
        }
        if (from != at) {  // back into the list that the ranking reads
            const uint64_t k = uint32_t(tid) < count ? S.list[from][tid] : 0;
            bar_sync();
            if (uint32_t(tid) < count) S.list[at][tid] = k;
        }
        bar_sync();
    }
    rank<kEntropy>(S.list[at], count, n, S.list[at + 1], st, q);
    S.state[tid] = make_float4(st.bar, st.ref, st.s, st.t);
    bar_sync();
    return int(min(count, n));
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kThreads, 2) top_kernel(const __grid_constant__ TopParams P)
{
    constexpr int kPer = Elems<T>::kPer;
    constexpr int kLag = 2;  // chunks that the closer has for a cut
    unsigned char* ring = ring_of();
    Shared& S = shared();
    const sampler_rows_t& a = P.rows;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t part = blockIdx.x % P.parts, q = blockIdx.x / P.parts, n_clusters = gridDim.x / P.parts;
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], kWarps);
        }
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&S.ready[i], 1);
            mbar_init(&S.ended[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&S.closed[i], 1);
        queue_open(S.queue, kWarps);
        S.lost_most = 0;
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kProducer) {
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

    if (warp == kCloser) {
        run_closer<T, kEntropy>(P);
        return;
    }

    const uint32_t n = uint32_t(P.top.top_n);
    const uint32_t trigger = min(n + 96, 208u), about = n + n / 4 + 8;
    RingPlace slot{0, 0};
    QueuePlace place{{0, 0}, 0};
    int job = 0;                    // jobs that the closer has been asked for
    uint32_t pair = 0;              // of lists that the row has: 0 or 2
    uint32_t rows_of[2] = {0, 0};   // rows that have gone to the closer with either pair
    int64_t done = 0;   // rows that this CTA has ended with
    bool failed = false;
    for (;; ++done) {
        RowItem row;
        // a wait that gives up gives up for all warps
        failed = bar_any(!queue_next(S.queue, place, P.wait_ns, row));
        if (failed || row.row < 0) break;
        const int64_t r = row.row;
        if (!row.live) {
            if (part == 0) write_none(P, r, SAMPLER_ROW_OK);
            continue;
        }
        const RowJob h = job_of(row);
        const RowSpan span{row.head, row.count};
        const int first = int(part) * P.part_vecs, last = min(first + P.part_vecs, span.count);
        const Scale scale{h.c_hi, h.c_lo};
        const Two c = two(scale.nearest(), scale.nearest());
        Sums st{-pos_inf(), -kFloatMax, 0.f, 0.f};
        bool has_n = false;
        uint32_t worst = Peak<T>::none();  // NaN, or +inf, where the row has one
        uint32_t at = pair, count = 0;  // the list that is filled, and the keys in it
        uint32_t kept = 0;              // keys that the list had before the present counter of S.pushed was begun
        int cutting = -1, age = 0;      // the job that cuts the other one, which was filled before, and the chunks since
        const Job job_of_row{kClose, 0, 0, 0, row.row, row.token, 0.f, 0.f, h.c_hi, h.c_lo, h.inv_t, h.inv_t_lo, h.x_t};
        // the row's lists are the ones of two rows ago
        const uint32_t gone = pair ? rows_of[1] : rows_of[0];
        failed = bar_any(gone != 0 && !wait(&S.closed[pair >> 1], (gone - 1) & 1u, P.wait_ns));
        if (failed) break;
        if (tid < 2) S.count[pair + tid] = 0;
        if (tid < 4) S.pushed[tid] = 0;
        uint32_t counter = 0;
        // The first bar: of the first chunks' largest in each thread, the n-th, rounded down to bf16 (two to an instruction,
        // whose counts are exact in bf16 up to 256); where fewer threads have any, all are taken. (Of the first chunk
        // alone: four times as many keys of the first quarter of a row, which cost more than this second look.)
        const int looked = min(last, first + kLook * kChunkVecs);
        {
            uint32_t peaks = Peak<T>::none();
            RingPlace ahead = slot;
            bool ok = true;
            for (int base = first; base < looked; base += kChunkVecs) {
                ok = ok && wait(&S.full[ahead.at], ahead.phase, P.wait_ns);
                uint4 v[kVecs];
                load<T>(v, Chunk{int(ahead.at) * kChunkBytes, base, ok ? last : 0, span.head, span.head + int(a.vocab)});
#pragma unroll
                for (int k = 0; k < kVecs; ++k) peaks = Peak<T>::join(peaks, peak<T>(v[k]));
                ahead.next(kSlots);
            }
            const float most = Peak<T>::value(peaks);
            const uint32_t mine = packed_bar<uint16_t>(most);
            S.largest[tid] = uint16_t(mine);
            failed = bar_any(!ok);
            if (failed) break;
            uint32_t n0 = 0, n1 = 0;
            const uint4* all = reinterpret_cast<const uint4*>(S.largest);
#pragma unroll 8
            for (int j = 0; j < kConsumers / 8; ++j) {
                const uint4 o = all[j];
                count_above(n0, o.x, mine);
                count_above(n1, o.y, mine);
                count_above(n0, o.z, mine);
                count_above(n1, o.w, mine);
            }
            const float above = __uint_as_float(n0 << 16) + __uint_as_float(n0 & 0xffff0000u) + __uint_as_float(n1 << 16) +
                                __uint_as_float(n1 & 0xffff0000u);
            // (of equal ones all have the first's place: the least of those that come before the n-th or on it)
            const bool within = above < float(n);
            const uint32_t least = __reduce_min_sync(0xffffffffu, within ? order_of(__uint_as_float(mine << 16)) : 0xffffffffu);
            if (lane == 0) S.tops[warp] = least;
            has_n = bar_count(within && most >= -kFloatMax) >= n;
            if (has_n) {
                uint32_t lo = 0xffffffffu;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) lo = min(lo, S.tops[w]);
                lo = max(lo, order_of(-kFloatMax));
                st.ref = value_of(lo);
                st.bar = below(lo);
            }
        }
        bool loose = has_n;  // n of the looked at tokens, not of those that are in the list, are at the bar or above
        for (int base = first; base < last; base += kChunkVecs) {
            const bool ok = wait(&S.full[slot.at], slot.phase, P.wait_ns);
            const Chunk chunk{int(slot.at) * kChunkBytes, base, ok ? last : 0, span.head, span.head + int(a.vocab)};
            uint4 v[kVecs];
            load<T>(v, chunk);
            uint32_t peaks[kVecs];
#pragma unroll
            for (int k = 0; k < kVecs; ++k) peaks[k] = peak<T>(v[k]);
            worst = Peak<T>::join(worst, Peak<T>::join(Peak<T>::join(peaks[0], peaks[1]), Peak<T>::join(peaks[2], peaks[3])));
            const float s_before = st.s, t_before = st.t, ref_before = st.ref;
            uint32_t top = 0, above = 0;
            const uint32_t bar = packed_bar<T>(st.bar);
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
                if (Peak<T>::above(peaks[k], bar)) above |= take_above<T>(v[k], bar) << k * kPer;
            uint32_t to = kCap;
            if (above) {
                const uint32_t want = uint32_t(__popc(above));
                to = kept + next_places(&S.pushed[counter], want);
                top = to + want;
            }
            add<T, kEntropy>(st, v, c);
            for (; above && to < kCap; ++to, above &= above - 1) {
                const int bit = __ffs(above) - 1, i = bit / kPer * kConsumers + tid, j = bit % kPer;
                S.list[at][to] = key_of(load_logit(reinterpret_cast<const T*>(ring + chunk.at) + i * kPer + j),
                                        (base + i) * kPer - span.head + j);
            }
            __syncwarp();
            const bool end = base + kChunkVecs >= last;
            const bool joins = cutting >= 0 && (++age == kLag || end);  // what the closer has cut is wanted now
            bool cut_ended = !joins || wait_job(cutting, P.wait_ns);
            const bool any = bar_any(top >= trigger || !ok || !cut_ended);
            if (any && bar_any(!ok || !cut_ended)) {
                failed = true;
                break;
            }
            if (any || end || joins) {
                // (Nobody waits for anybody here, but where a function out of line or the closer takes over: counters are
                // used in turn, and the one after the next is cleared.)
                count = kept + S.pushed[counter];
                bool over = count > uint32_t(kCap);
                float bar_before = st.bar;  // of this chunk, should it be looked at again
                // (with what the closer leaves, 256 at most, the other list's keys of the chunks before have to fit)
                if (cutting >= 0 && (joins || count > uint32_t(kCap - kClosable))) {
                    if (!joins) {  // the cut is wanted early
                        cut_ended = wait_job(cutting, P.wait_ns);
                        failed = bar_any(!cut_ended);
                        if (failed) break;
                    }
                    // what has been cut meanwhile, and, after it, what the chunks since have put into the other list
                    const uint32_t left = S.cut_count, full = at ^ 1;
                    const uint64_t least = S.cut_least;
                    over |= left + count > uint32_t(kCap);
                    if (over) {
                        // this chunk's are taken again
                        const int before = base * kPer - span.head;
                        const uint32_t valid = min(count, uint32_t(kCap));
                        if (tid == 0) S.count[full] = left;
                        bar_sync();
#pragma unroll 1
                        for (uint32_t i0 = 0; i0 < valid; i0 += kConsumers) {
                            const uint64_t k = i0 + tid < valid ? S.list[at][i0 + tid] : 0;
                            const bool stays = k != 0 && key_token(k) < before;
                            const uint32_t place = places(&S.count[full], stays);
                            if (stays && place < kCap) S.list[full][place] = k;
                        }
                        bar_sync();
                        count = min(S.count[full], uint32_t(kCap));
                        st.s = s_before;
                        st.t = t_before;
                    } else {
                        for (uint32_t i = tid; i < count; i += kConsumers) S.list[full][left + i] = S.list[at][i];
                        count += left;
                    }
                    move(st, key_value(least), scale);
                    if (tid == 0) {
                        Sums lost{0.f, S.cut_ref, S.cut_s, S.cut_t};
                        move(lost, st.ref, scale);
                        st.s += lost.s;
                        st.t += lost.t;
                    }
                    cutting = -1;
                    at = full;
                    bar_before = st.ref;
                } else if (over) {  // (no cut is under way)
                    st.s = s_before;
                    st.t = t_before;
                }
                if (cutting >= 0) {
                    kept = count;
                } else if (over || count > uint32_t(kClosable)) {
                    if (tid == 0) S.count[at ^ 1] = 0;
                    S.state[tid] = make_float4(bar_before, st.ref, st.s, st.t);
                    bar_sync();
                    at = over ? slow_chunk<T, kEntropy>(at, min(count, uint32_t(kCap)), chunk.at, base, last, chunk.head, chunk.end, n,
                                                        h.c_hi, h.c_lo)
                              : cut_long<kEntropy>(at, count, n, about, h.c_hi, h.c_lo);
                    const float4 q = S.state[tid];
                    st = Sums{q.x, q.y, q.z, q.w};
                    count = S.count[at];
                    has_n = true;
                    kept = count;
                } else if (!end && count >= trigger) {
                    // the closer cuts it, while the next chunks go into the other one
                    has_n = true;
                    cutting = job++;
                    age = 0;
                    bar_sync();
                    if (warp == 0) {
                        Job j = job_of_row;
                        j.kind = kCut;
                        j.list = int(at);
                        j.count = int(count);
                        j.bar = bar_before;
                        post_job(cutting, j, P.wait_ns);  // (where that gives up, the wait for its end does)
                    }
                    at ^= 1;
                    kept = 0;
                } else {
                    kept = count;
                }
                counter = (counter + 1) & 3;
                if (tid == 0) S.pushed[(counter + 1) & 3] = 0;
                if (end) bar_sync();
            }
            loose = loose && st.ref == ref_before && base + kChunkVecs < looked;
            if (has_n && !loose) st.bar = st.ref;  // later tokens lose ties
            if (lane == 0) mbar_arrive(&S.empty[slot.at]);
            slot.next(kSlots);
        }
        if (failed) break;
        const bool bad = bar_any(!(Peak<T>::value(worst) < pos_inf()));
        int status = h.bad_param ? SAMPLER_ROW_BAD_PARAM : bad ? SAMPLER_ROW_NONFINITE : SAMPLER_ROW_OK;
        bool ordered = false;
        if (P.parts > 1) {
            // this part's n largest keys and sums go into the workspace, for the part of the row that ends last
            rank<kEntropy>(S.list[at], count, n, S.list[at ^ 1], st, scale);
            count = min(count, n);
            float s = st.s, t = st.t;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                if (kEntropy) t += __shfl_xor_sync(0xffffffffu, t, o);
            }
            if (lane == 0) S.sums[pair >> 1][warp] = make_float2(s, t);
            if (uint32_t(tid) < count)
                __stcg(reinterpret_cast<unsigned long long*>(P.ws.keys + (r * P.parts + part) * kMost + tid), S.list[at ^ 1][tid]);
            bar_sync();
            s = t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                s += S.sums[pair >> 1][w].x;
                t += S.sums[pair >> 1][w].y;
            }
            if (!leave(P, r, part, TopPart{st.ref, s, t, int(count), bad, 0})) continue;
            const int joined = join_parts<kEntropy>(P, r, pair, h.c_hi, h.c_lo);
            const float4 q = S.state[tid];
            st = Sums{q.x, q.y, q.z, q.w};
            count = uint32_t(max(joined, 0));
            at = pair + 1;
            ordered = true;
            if (status == SAMPLER_ROW_OK && joined < 0) status = joined == -1 ? SAMPLER_ROW_TIMEOUT : SAMPLER_ROW_NONFINITE;
            if (joined == -1) status = SAMPLER_ROW_TIMEOUT;
        }
        if (status == SAMPLER_ROW_OK && count == 0) status = SAMPLER_ROW_ALL_NEG_INF;
        if (status != SAMPLER_ROW_OK) {
            write_none(P, r, status);
            bar_sync();
            continue;
        }
        // the rest of the row's work is the closer's
        float s = st.s, t = st.t;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            if (kEntropy) t += __shfl_xor_sync(0xffffffffu, t, o);
        }
        if (lane == 0) S.sums[pair >> 1][warp] = make_float2(s, t);
        bar_sync();
        const int closing = job++;
        if (pair)
            ++rows_of[1];
        else
            ++rows_of[0];
        pair ^= 2;
        bool posted = true;
        if (warp == 0) {
            Job j = job_of_row;
            j.list = int(at);
            j.count = int(count);
            j.ordered = ordered;
            j.ref = st.ref;
            j.bar = st.bar;
            posted = post_job(closing, j, P.wait_ns);
        }
        failed = bar_any(!posted);
        if (failed) {
            if (P.parts > 1) {  // the row's parts have all been counted
                write_none(P, r, SAMPLER_ROW_TIMEOUT);
                ++done;
            }
            break;
        }
    }
    if (warp == 0) {
        Job j;
        j.kind = kEnd;
        post_job(job, j, kWaitNs);
    }
    if (!failed) return;

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
        } else if (P.parts == 1 || leave(P, r, part, TopPart{0.f, 0.f, 0.f, 0, 0, 1})) {
            write_none(P, r, SAMPLER_ROW_TIMEOUT);
        }
    }
}

// ---------------------------------------------------------------- short rows
// A warp by itself takes a row of 32 KB at most, all of it in shared memory, with the next one on its way there while the
// row's keys are put in order.
constexpr int kShortWarps = 4;
constexpr int kShortVecs = 2049;   // of a row, where rows are many
constexpr int kShortFew = 513;     // where each has a place in the other kernel
constexpr int kShortResident = 5;  // CTAs of kShortWarps that an SM's registers hold
constexpr int kGroups = 8;         // of a lane's vectors

struct Short {
    uint64_t list[kClosable];
    uint64_t sorted[kMost];
    uint32_t count;
    uint32_t pad[3];
};
constexpr int kSmemOfSm = 228 * 1024;
constexpr int kShortSmem = kShortWarps * (kShortVecs * 16 + int(sizeof(Short)));

__device__ __forceinline__ void copy_vector(uint4* to, const uint4* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

// The largest elements that a lane's groups have: of a group one in fp32, two in bf16 (of the even and the odd ones).
template <typename T>
struct Largest {
    static constexpr int kCount = sizeof(T) == 2 ? 2 * kGroups : kGroups;
    float x[kCount];
};

template <typename T>
__device__ __forceinline__ Largest<T> largest_of(const uint32_t (&peaks)[kGroups])
{
    Largest<T> y;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (sizeof(T) == 2) {
            y.x[2 * g] = __uint_as_float(peaks[g] << 16);
            y.x[(2 * g + 1) % Largest<T>::kCount] = __uint_as_float(peaks[g] & 0xffff0000u);
        } else {
            y.x[g] = __uint_as_float(peaks[g]);
        }
    }
    return y;
}

// The order of a value that n of the lanes' largest reach, and not many more than n; `top` is the largest's. The lowest
// finite value's where there are fewer than n.
template <typename T>
__device__ __forceinline__ uint32_t first_bar(const Largest<T>& a, uint32_t n, uint32_t top)
{
    auto reach = [&](float b1, float b2, float b3) {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < Largest<T>::kCount; ++i)
            c += (a.x[i] >= b1 ? 1u : 0u) + (a.x[i] >= b2 ? 1u << 10 : 0u) + (a.x[i] >= b3 ? 1u << 20 : 0u);
        return __reduce_add_sync(0xffffffffu, c);
    };
    uint32_t lo = order_of(-kFloatMax), hi = top + 1;
#pragma unroll 1
    while (hi - lo > 1) {
        const uint32_t q = max((hi - lo) / 4, 1u), o1 = lo + q, o2 = min(o1 + q, hi), o3 = min(o2 + q, hi);
        const uint32_t got = reach(value_of(o1), value_of(o2), value_of(o3)), c1 = got & 1023u, c2 = got >> 10 & 1023u,
                       c3 = got >> 20;
        uint32_t c;
        if (c3 >= n) {
            lo = o3;
            c = c3;
        } else if (c2 >= n) {
            lo = o2;
            hi = o3;
            c = c2;
        } else if (c1 >= n) {
            lo = o1;
            hi = o2;
            c = c1;
        } else {
            hi = o1;
            continue;
        }
        if (c <= n + n / 8) break;
    }
    return lo;
}

// The least key of those that n to kClosable of the row's reach; more than kClosable reach the value of order `lo`.
template <typename T>
__device__ __forceinline__ uint64_t least_of_row(const T* x, int vocab, uint32_t n, uint32_t lo, uint32_t top)
{
    const int lane = threadIdx.x & 31;
    auto reach = [&](uint64_t key) {
        uint32_t c = 0;
        for (int j = lane; j < vocab; j += 32) c += key_of(load_logit(x + j), j) >= key;
        return __reduce_add_sync(0xffffffffu, c);
    };
    uint64_t l = uint64_t(lo) << 32, h = (uint64_t(top) + 1) << 32;
    for (int part = 0; part < 2; ++part) {
        const uint64_t last = part == 0 ? 1ull << 32 : 1;
#pragma unroll 1
        while (h - l > last) {
            const uint64_t mid = l + ((h - l) / 2 & ~(last - 1));
            const uint32_t got = reach(mid);
            if (got >= n) {
                l = mid;
                if (got <= uint32_t(kClosable)) return l;
            } else {
                h = mid;
            }
        }
        if (part == 0) l |= uint32_t(~uint32_t(kMaxToken));  // the lowest key of the value
    }
    return l;
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kShortWarps * 32, kShortResident) top_short_kernel(const __grid_constant__ TopParams P)
{
    constexpr int kPer = Elems<T>::kPer;
    const sampler_rows_t& a = P.rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vocab = int(a.vocab);
    unsigned char* mine = ring_of() + warp * (P.part_vecs * 16 + int(sizeof(Short)));
    uint4* vecs = reinterpret_cast<uint4*>(mine);
    Short& S = *reinterpret_cast<Short*>(mine + P.part_vecs * 16);
    const uint32_t n = uint32_t(P.top.top_n);
    const int64_t step = int64_t(gridDim.x) * (blockDim.x >> 5);

    // What comes with a row, and its vectors where it counts.
    struct Next {
        float weight, temperature;
        int token;
    };
    auto look = [&](int64_t r) {
        Next y{0.f, 1.f, 0};
        if (r >= a.n_rows) return y;
        y.weight = a.weight ? a.weight[r] : 1.f;
        if (a.temperature) y.temperature = a.temperature[r];
        if (a.tokens) y.token = a.tokens[r];
        return y;
    };
    auto fetch = [&](int64_t r) {
        const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
        const RowSpan span = row_span(x, a.vocab);
        const uint4* from = reinterpret_cast<const uint4*>(x - span.head);
        for (int i = lane; i < span.count; i += 32) copy_vector(vecs + i, from + i);
    };

    int64_t r = int64_t(blockIdx.x) + int64_t(gridDim.x) * warp;
    Next now = look(r);
    if (now.weight != 0.f) fetch(r);
    for (; r < a.n_rows; r += step) {
        const Next next = look(r + step);
        // (the row's vectors have been read when this is called)
        auto ahead = [&] {
            __syncwarp();
            if (next.weight != 0.f) fetch(r + step);
        };
        const Next given = now;
        now = next;
        if (given.weight == 0.f) {
            write_none(P, r, SAMPLER_ROW_OK, lane, 32);
            ahead();
            continue;
        }
        RowJob h;
        h.token = given.token;
        row_scale(h, a, given.temperature);
        const RowSpan span = row_span(static_cast<const T*>(a.logits) + r * a.row_stride, a.vocab);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        // what is not the row's becomes -inf
        if (lane == 0) {
            uint4 v = vecs[0];
            Elems<T>::mask(v, span.head, span.head + vocab);
            vecs[0] = v;
            const int at = (span.count - 1) * kPer;
            v = vecs[span.count - 1];
            Elems<T>::mask(v, span.head - at, span.head + vocab - at);
            vecs[span.count - 1] = v;
            S.count = 0;
        }
        __syncwarp();
        const T* x = reinterpret_cast<const T*>(vecs) + span.head;
        h.x_t = a.out_logprob && !h.bad_param ? load_logit(x + h.token) : 0.f;

        uint32_t peaks[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) peaks[g] = Peak<T>::none();
        for (int base = 0; base < span.count; base += 32 * kGroups)
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int i = base + 32 * g + lane;
                if (i < span.count) peaks[g] = Peak<T>::join(peaks[g], peak<T>(vecs[i]));
            }
        uint32_t most = peaks[0];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) most = Peak<T>::join(most, peaks[g]);
        const float largest = Peak<T>::value(most);
        const bool bad = __any_sync(0xffffffffu, !(largest < pos_inf()));
        const uint32_t top = __reduce_max_sync(0xffffffffu, order_of(largest));
        const int status = h.bad_param            ? SAMPLER_ROW_BAD_PARAM
                           : bad                  ? SAMPLER_ROW_NONFINITE
                           : top < order_of(-kFloatMax) ? SAMPLER_ROW_ALL_NEG_INF
                                                  : SAMPLER_ROW_OK;
        if (status != SAMPLER_ROW_OK) {
            write_none(P, r, status, lane, 32);
            ahead();
            continue;
        }
        const uint32_t lo = first_bar<T>(largest_of<T>(peaks), n, top);
        Sums st{below(lo), value_of(lo), 0.f, 0.f};
        const uint32_t bar = packed_bar<T>(st.bar);
        const float nearest = Scale{h.c_hi, h.c_lo}.nearest();
        const Two c = two(nearest, nearest);
        for (int base = 0; base < span.count; base += 32 * kVecs) {
            uint4 v[kVecs];
            uint32_t above = 0;
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int i = base + 32 * k + lane;
                v[k] = i < span.count ? vecs[i] : make_uint4(Peak<T>::none(), Peak<T>::none(), Peak<T>::none(), Peak<T>::none());
                if (Peak<T>::above(peak<T>(v[k]), bar)) above |= take_above<T>(v[k], bar) << k * kPer;
            }
            if (above) {
                uint32_t to = next_places(&S.count, uint32_t(__popc(above)));
                for (; above && to < uint32_t(kClosable); ++to, above &= above - 1) {
                    const int bit = __ffs(above) - 1, j = (base + 32 * (bit / kPer) + lane) * kPer + bit % kPer - span.head;
                    S.list[to] = key_of(load_logit(x + j), j);
                }
            }
            add<T, kEntropy>(st, v, c);
        }
        __syncwarp();
        uint32_t count = S.count;
        if (count > uint32_t(kClosable)) {
            // ties, or a row whose largest are close together: a key for a bar, and all of it once more
            const uint64_t least = least_of_row<T>(x, vocab, n, lo, top);
            st = Sums{0.f, key_value(least), 0.f, 0.f};
            st.bar = st.ref;
            count = 0;
            Pair s{0.f, 0.f}, t{0.f, 0.f};  // (one after the other: 440 a lane, alike where there are ties)
            for (int base = 0; base < vocab; base += 32) {
                const int j = base + lane;
                const float y = j < vocab ? load_logit(x + j) : -pos_inf();
                const uint64_t k = key_of(y, j);
                const bool stays = j < vocab && k >= least;
                const uint32_t lanes = __ballot_sync(0xffffffffu, stays);
                if (stays) {
                    S.list[count + __popc(lanes & ((1u << lane) - 1u))] = k;
                } else {
                    const float d = y - st.ref, u = fmaf(d, h.c_hi, d * h.c_lo), f = exp2_fast(u);
                    const Pair p = two_sum(s.hi, f);
                    s = Pair{p.hi, s.lo + p.lo};
                    if (kEntropy) {
                        const Pair w = two_sum(t.hi, f * fmaxf(u, kLowest));
                        t = Pair{w.hi, t.lo + w.lo};
                    }
                }
                count += uint32_t(__popc(lanes));
            }
            st.s = s.hi + s.lo;
            st.t = t.hi + t.lo;
        }
        ahead();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
            if (kEntropy) st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
        }
        st.bar = st.ref;
        close_list<T, kEntropy>(P, S.list, int(count), S.sorted, st.ref, st, h, r);
        __syncwarp();
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
    // Rows of 8 KB at most, and of 32 KB where there are more than the other kernel holds at once, are a warp's each. Measured,
    // us by chunks and by warps (bf16, n = 64; of one row n = 20):
    //   1 x 1000       8.9   7.5      4096 x 4096   121   38
    //   1 x 4096       9.1   8.0      4096 x 8186   121   65
    //   1 x 8186       7.8  10.4      4096 x 12000  131   73
    //   100 x 4096    13.0  12.9      4096 x 16000  132  120
    //   100 x 8186    13.6  15.4      350 x 12000    23   18
    // (A handle whose waits all give up takes the kernel that waits.)
    if (vecs <= (p.rows.n_rows > 2 * sms ? kShortVecs : kShortFew) && p.wait_ns != 0) {
        const auto kernel = bf16 ? entropy ? top_short_kernel<uint16_t, true> : top_short_kernel<uint16_t, false>
                                 : entropy ? top_short_kernel<float, true> : top_short_kernel<float, false>;
        bool& granted = grants->short_granted[bf16][entropy];
        if (!granted && cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kShortSmem) != cudaSuccess)
            return SAMPLER_ERR_CUDA;
        granted = true;
        p.parts = 1;
        p.part_vecs = int(vecs);
        // rows on as many SMs as there are
        const int64_t warps = std::min<int64_t>(kShortWarps, (p.rows.n_rows + sms - 1) / sms);
        const int smem = int(warps) * (p.part_vecs * 16 + int(sizeof(Short)));
        const int64_t resident = std::min<int64_t>(kShortResident * kShortWarps / warps, kSmemOfSm / (smem + 1024));
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(std::min((p.rows.n_rows + warps - 1) / warps, resident * sms)));
        cfg.blockDim = dim3(unsigned(warps) * 32);
        cfg.dynamicSmemBytes = size_t(smem);
        cfg.stream = stream;
        return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
    }
    const int64_t slots = 2 * int64_t(sms);
    // parts of a row, where rows are few: eight at most, of two chunks at least, as their joining takes as long as some
    // chunks do (32 of 4 KB, 32 x 151936 bf16 and n = 20: 18.2 for 16.4 us; 1 row: 21.2 for 15.1; 1 x 16384: 13.4 for 7.9
    // in one part), and so many that their keys fit the list
    int64_t parts = std::max<int64_t>(1, slots / p.rows.n_rows);
    parts = std::min({parts, int64_t(kMaxTopParts), int64_t(kCap / p.top.top_n), std::max<int64_t>(1, vecs / (2 * kChunkVecs))});
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
