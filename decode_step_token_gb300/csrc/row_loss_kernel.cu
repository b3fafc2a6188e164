// row_loss_kernel.cu -- scoring and the losses over logits rows: logprob,
// entropy, the clipped policy loss, the preference loss, and the logits'
// gradients.
//
// A row's gradient needs the row's sums, so a row is wanted twice, and is read
// from memory once: a cluster of C CTAs takes a row, each CTA a part of it in
// shared memory, where the second pass finds it. Warp roles of a CTA:
//   producer   goes ahead over the cluster's rows: it reads their parameters and
//              brings their parts in with bulk copies, through a ring of 16 KB chunks;
//   consumers  (sixteen) pass 1, two vectors of each chunk in every thread: the
//              running reference and the sums of exponentials, which each warp puts
//              into every CTA of the cluster (distributed shared memory);
//   closer     combines the cluster's sums, works out the gradient's factors and
//              writes the row's outputs;
//   consumers  pass 2, with a gradient: the same vectors again from the ring,
//              16-byte stores, and each chunk's slot goes back to the producer.
// Where two parts fit in the ring, the consumers take pass 1 of a row before pass 2
// of the row before it, so that the join and the closer's work (3 to 4 us a row,
// most of it latency) run under pass 1.
// The rows that count are dealt to the clusters evenly whatever rows are left
// out: each producer counts them, 32 weights at a time.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "row_loss.cuh"

namespace dst {
namespace rows {

constexpr int kWarps = 16;                       // consumers
constexpr int kConsumers = kWarps * 32;
constexpr int kProducer = kWarps, kCloser = kWarps + 1;
constexpr int kThreads = kConsumers + 64;
constexpr int kVecs = 2;                         // 16-byte vectors of a chunk in each consumer
constexpr int kChunkVecs = kConsumers * kVecs;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kMaxSlots = 6;
constexpr int kPartChunks = 6;                   // of a row in a CTA, where the row allows it
constexpr int kMaxParts = 16;                    // CTAs of a cluster
constexpr int kJobs = 4;                         // rows that a CTA has in hand
constexpr int kSums = 4;                         // rows whose sums are in shared memory
constexpr int kSmemMax = 113 * 1024;             // of a CTA: two on an SM
constexpr uint64_t kWaitNs = 2000000000ull;      // a wait gives up after 2 s

// The ring (slots * kChunkBytes), the sums [kSums][parts * kWarps] and this.
struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t job_full[kJobs], job_empty[kJobs];
    uint64_t join[kSums], closed[kSums];
    RowJob jobs[kJobs];
    RowRecord rec[kSums];
    double scratch[kThreads / 32];
    uint32_t flag, failed;  // failed: a wait of this CTA gave up
};

constexpr int smem_of(int slots, int parts)
{
    return slots * kChunkBytes + kSums * parts * kWarps * int(sizeof(float4)) + int(sizeof(Shared));
}

constexpr int slots_for(int parts)
{
    int slots = kMaxSlots;
    while (smem_of(slots, parts) > kSmemMax) --slots;
    return slots;
}

// How the rows of a call are cut.
struct RowPlan {
    int part_vecs;  // vectors of a row in each CTA
    int slots;
    int deep;       // two parts fit in the ring
};

// A ring's place and the parity of its phase.
struct Place {
    uint32_t at, phase;
    __device__ __forceinline__ void next(uint32_t n)
    {
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// A whole warp waits for the phase of `bar` with the given parity, for kWaitNs at
// most; all of its lanes get the same answer.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity)
{
    const uint64_t until = now_ns() + kWaitNs;
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 63u) == 63u && __any_sync(0xffffffffu, now_ns() > until)) return false;
    }
    return false;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_slow(bar, parity);
}

__device__ __forceinline__ void arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Put 16 bytes into a CTA of the cluster and count them on its barrier. (Ordinary
// stores and a release of the cluster would wait for all that the thread has
// stored, the last row's gradient included.)
__device__ __forceinline__ void put_sums(uint32_t addr, uint32_t bar, float a, float b, float c, float d)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
                 : "memory");
}

// A wait for row r (-1: for no row yet) gave up: the row says so, and the loss
// becomes NaN.
__device__ __noinline__ void gave_up(Shared& S, const LossParams& P, int64_t r)
{
    if ((threadIdx.x & 31) != 0) return;
    S.failed = 1;
    if (r >= 0 && P.rows.out_status) P.rows.out_status[r] = SAMPLER_ROW_TIMEOUT;
    if (P.mode == kModePolicy) atomicOr(P.ws.ticket, kGaveUp);
}

// ---------------------------------------------------------------- vectors
// The 16-byte vectors that a row touches: vector 0 starts at or before the row's
// first element (`head` elements of it lie before), `count` cover the row.
struct RowSpan {
    int head;
    int count;
};

template <typename T>
__device__ __forceinline__ RowSpan row_span(const T* x, int64_t vocab)
{
    constexpr int kPer = 16 / int(sizeof(T));
    RowSpan s;
    s.head = int((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    s.count = int((s.head + vocab + kPer - 1) / kPer);
    return s;
}

template <typename T>
struct Elems;
template <>
struct Elems<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ void widen(const uint4& v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float largest(const uint4& v)  // NaN where there is one
    {
        float a, b;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w)));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(b));
        return a;
    }
    static __device__ __forceinline__ uint4 round(const float (&y)[4])
    {
        return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
    }
    // elements before `lo` and from `hi` on become -inf
    static __device__ __forceinline__ void mask(uint4& v, int lo, int hi)
    {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < lo || j >= hi) w[j] = 0xff800000u;
    }
};
template <>
struct Elems<uint16_t> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ void widen(const uint4& v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ float largest(const uint4& v)
    {
        uint32_t a, b;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        float m;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(__uint_as_float(a << 16)), "f"(__uint_as_float(a & 0xffff0000u)));
        return m;
    }
    static __device__ __forceinline__ uint4 round(const float (&y)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(y[2 * j + 1]), "f"(y[2 * j]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void mask(uint4& v, int lo, int hi)
    {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < lo || j >= hi)
                w[j / 2] = (j & 1) ? (w[j / 2] & 0xffffu) | 0xff800000u : (w[j / 2] & 0xffff0000u) | 0xff80u;
    }
};

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two fp32 operations in one instruction: both passes are bound by the number of
// instructions before they are by memory.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 y;
    asm("{\n\t.reg .b64 s, t;\n\tmov.b64 s, {%2, %3};\n\tmov.b64 t, {%4, %5};\n\tadd.rn.f32x2 s, s, t;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return y;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 y;
    asm("{\n\t.reg .b64 s, t;\n\tmov.b64 s, {%2, %3};\n\tmov.b64 t, {%4, %5};\n\tmul.rn.f32x2 s, s, t;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return y;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 y;
    asm("{\n\t.reg .b64 s, t, u;\n\tmov.b64 s, {%2, %3};\n\tmov.b64 t, {%4, %5};\n\tmov.b64 u, {%6, %7};\n\t"
        "fma.rn.f32x2 s, s, t, u;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return y;
}

// Pass 1 over N vectors. The reference moves only when one holds a larger
// element, which is rare after the first few.
template <typename T, bool kEntropy, int N>
__device__ __forceinline__ void fold(Stats& st, bool& bad, const uint4 (&v)[N], float c_hi, float c_lo)
{
    constexpr int kPer = Elems<T>::kPer;
    float m = Elems<T>::largest(v[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) m = max_nan(m, Elems<T>::largest(v[k]));
    if (!(m <= st.ref)) {
        if (m < pos_inf())
            stats_move(st, m, c_hi);
        else
            bad = true;
    }
    const float2 ref = make_float2(-st.ref, -st.ref), hi = make_float2(c_hi, c_hi), lo = make_float2(c_lo, c_lo);
    float2 s = make_float2(st.s, 0.f), t = make_float2(st.t, 0.f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float x[kPer];
        Elems<T>::widen(v[k], x);
#pragma unroll
        for (int j = 0; j < kPer; j += 2) {
            const float2 d = add2(make_float2(x[j], x[j + 1]), ref);
            float2 u = fma2(d, hi, mul2(d, lo));
            const float2 e = make_float2(exp2_fast(u.x), exp2_fast(u.y));
            s = add2(s, e);
            if (kEntropy) {
                u.x = fmaxf(u.x, kLowest);
                u.y = fmaxf(u.y, kLowest);
                t = fma2(e, u, t);
            }
        }
    }
    st.s = s.x + s.y;
    if (kEntropy) st.t = t.x + t.y;
}

// Pass 2 of one vector; `at` is the token's place in it (outside [0, kPer): not in it).
template <typename T, bool kEntropy>
__device__ __forceinline__ uint4 gradient(const uint4& v, const RowRecord& rec, int at)
{
    constexpr int kPer = Elems<T>::kPer;
    const float2 ref = make_float2(-rec.ref, -rec.ref), c = make_float2(rec.c, rec.c);
    const float2 k0 = make_float2(rec.k0, rec.k0), k1 = make_float2(rec.k1, rec.k1);
    float x[kPer];
    Elems<T>::widen(v, x);
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
        float2 u = mul2(add2(make_float2(x[j], x[j + 1]), ref), c);
        float2 y;
        if (kEntropy) {
            u.x = fmaxf(u.x, kLowest);
            u.y = fmaxf(u.y, kLowest);
            y = mul2(make_float2(exp2_fast(u.x), exp2_fast(u.y)), fma2(k1, u, k0));
        } else {
            y = mul2(make_float2(exp2_fast(u.x), exp2_fast(u.y)), k0);
        }
        x[j] = y.x;
        x[j + 1] = y.y;
    }
    if (unsigned(at) < unsigned(kPer)) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j == at) x[j] += rec.at_token;
    }
    return Elems<T>::round(x);
}

// Store vector `i` of a row's span to the gradient: as one where it lies wholly
// inside the row and the gradient's vectors lie as the logits' do (`whole`), else
// by element.
template <typename T>
__device__ __forceinline__ void put_vector(T* g, int vocab, const RowSpan& span, int i, bool whole, const uint4& y)
{
    constexpr int kPer = Elems<T>::kPer;
    const int first = i * kPer - span.head;
    if (whole && first >= 0 && first + kPer <= vocab) {
        __stcs(reinterpret_cast<uint4*>(g + first), y);
    } else {
        const T* e = reinterpret_cast<const T*>(&y);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (first + j >= 0 && first + j < vocab) g[first + j] = e[j];
    }
}

// ---------------------------------------------------------------- the kernel
// The rows of cluster `q` of `n_clusters`, in order: every n_clusters-th of those
// that count, and every n_clusters-th of those that are left out. One warp.
struct RowDealer {
    int64_t base;            // first row of the 32 in `mine`; without weights: the next row
    uint32_t mine;           // those of them that are this cluster's and have not been given out
    uint32_t live, dead;     // rows of either kind before `base`, modulo n_clusters
    uint32_t group;          // of the four in `counts`
    uint32_t counts;         // bit k: this lane's row of group k of 32 has a weight
    float ahead[4];          // weights of the next 128 rows
};

__device__ __forceinline__ void dealer_load(RowDealer& d, const sampler_rows_t& a, int64_t base)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = base + 32 * k + (threadIdx.x & 31);
        d.ahead[k] = r < a.n_rows ? a.weight[r] : 1.f;
    }
}

__device__ __forceinline__ void dealer_open(RowDealer& d, const sampler_rows_t& a, uint32_t q)
{
    d.base = a.weight ? -32 : int64_t(q);
    d.mine = d.live = d.dead = d.counts = 0;
    d.group = 3;
    if (a.weight) dealer_load(d, a, 0);
}

// The next row, -1 at the end.
__device__ __forceinline__ int64_t dealer_next(RowDealer& d, const sampler_rows_t& a, uint32_t q, uint32_t n_clusters)
{
    if (!a.weight) {
        const int64_t r = d.base;
        d.base += n_clusters;
        return r < a.n_rows ? r : -1;
    }
    const uint32_t lane = threadIdx.x & 31;
    while (d.mine == 0) {
        d.base += 32;
        if (d.base >= a.n_rows) return -1;
        if (++d.group == 4) {
            d.group = 0;
            d.counts = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) d.counts |= d.ahead[k] != 0.f ? 1u << k : 0u;
            dealer_load(d, a, d.base + 128);
        }
        const bool in = d.base + lane < a.n_rows, counts = d.counts >> d.group & 1u;
        const uint32_t live = __ballot_sync(0xffffffffu, in && counts), dead = __ballot_sync(0xffffffffu, in && !counts);
        const uint32_t before = (1u << lane) - 1u;
        uint32_t rank = counts ? d.live + __popc(live & before) : d.dead + __popc(dead & before);
        rank %= n_clusters;
        d.mine = __ballot_sync(0xffffffffu, in && rank == q);
        d.live = (d.live + __popc(live)) % n_clusters;
        d.dead = (d.dead + __popc(dead)) % n_clusters;
    }
    const int bit = __ffs(d.mine) - 1;
    d.mine &= d.mine - 1u;
    return d.base + bit;
}

// What a producer reads of a row ahead of its turn.
struct RowAhead {
    int64_t row;     // -1: none
    int32_t token;
    float weight, T, in0, in1, in2;
    float x_t;
};

__device__ __forceinline__ void ahead_load(RowAhead& h, const LossParams& P, int64_t r)
{
    const sampler_rows_t& a = P.rows;
    h.row = r;
    if (r < 0) return;
    h.token = a.tokens[r];
    h.weight = a.weight ? a.weight[r] : 1.f;
    h.T = a.temperature ? a.temperature[r] : 1.f;
    h.in0 = h.in1 = h.in2 = 0.f;
    if (P.mode == kModeScoreGrad) {
        h.in0 = P.grad_logprob[r];
        if (P.grad_entropy) h.in1 = P.grad_entropy[r];
    } else if (P.mode == kModePolicy) {
        h.in0 = P.policy.advantage[r];
        h.in1 = P.policy.old_logprob[r];
        if (P.policy.ref_logprob) h.in2 = P.policy.ref_logprob[r];
    }
}

// The token's logit. It is read before the row is taken up, and so before any
// CTA can write the row's gradient in the logits' place.
template <typename T>
__device__ __forceinline__ void ahead_token(RowAhead& h, const sampler_rows_t& a)
{
    h.x_t = 0.f;
    if (h.row >= 0 && h.weight != 0.f && h.token >= 0 && int64_t(h.token) < a.vocab)
        h.x_t = load_logit(static_cast<const T*>(a.logits) + h.row * a.row_stride + h.token);
}

// A CTA's part of a row: vectors first .. last, in chunks that end at `end`
// (counted for the consumer: every one of them takes part in each chunk).
struct RowPart {
    RowSpan span;
    int first, last, end;
};

template <typename T>
__device__ __forceinline__ RowPart row_part(const T* x, int64_t vocab, uint32_t rank, int part_vecs)
{
    RowPart p;
    p.span = row_span(x, vocab);
    p.first = int(rank) * part_vecs;
    p.last = max(p.first, min(p.first + part_vecs, p.span.count));
    p.end = p.first + (p.last - p.first + kChunkVecs - 1) / kChunkVecs * kChunkVecs;
    return p;
}

// kGrad: with the logits' gradient. kEntropy: with the sum t. The grid is whole
// clusters.
template <typename T, bool kGrad, bool kEntropy>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const __grid_constant__ LossParams P, const RowPlan plan)
{
    extern __shared__ __align__(128) unsigned char ring[];
    const sampler_rows_t& a = P.rows;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t parts = cluster_nctarank(), rank = cluster_ctarank();
    const uint32_t q = blockIdx.x / parts, n_clusters = gridDim.x / parts;
    const uint32_t slots = uint32_t(plan.slots);
    float4* sums = reinterpret_cast<float4*>(ring + slots * kChunkBytes);
    Shared& S = *reinterpret_cast<Shared*>(sums + kSums * parts * kWarps);

    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], kWarps);
        }
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&S.job_full[i], 1);
            mbar_init(&S.job_empty[i], kWarps + 1);
        }
        for (int i = 0; i < kSums; ++i) {
            mbar_init(&S.join[i], 1);
            mbar_init(&S.closed[i], 1);
        }
        S.failed = 0;
        fence_mbar_init();
    }
    cluster_sync();

    if (warp == kProducer) {
        RowDealer d;
        dealer_open(d, a, q);
        Place slot{0, 0}, job{0, 0};
        uint32_t issued = 0;
        bool ok = true;
        auto copy_in = [&](const RowAhead& h) {
            const T* x = static_cast<const T*>(a.logits) + h.row * a.row_stride;
            const RowPart part = row_part(x, a.vocab, rank, plan.part_vecs);
            const unsigned char* from = reinterpret_cast<const unsigned char*>(x - part.span.head);
            for (int v = part.first; ok && v < part.last; v += kChunkVecs) {
                ok = wait(&S.empty[slot.at], slot.phase ^ 1u);
                if (ok && lane == 0) {
                    const uint32_t bytes = uint32_t(min(kChunkVecs, part.last - v)) * 16u;
                    mbar_arrive_expect_tx(&S.full[slot.at], bytes);
                    bulk_copy_g2s(ring + slot.at * kChunkBytes, from + size_t(v) * 16, bytes, &S.full[slot.at]);
                }
                __syncwarp();
                slot.next(slots);
                ++issued;
            }
        };
        RowAhead now, next;
        ahead_load(now, P, dealer_next(d, a, q, n_clusters));
        if (now.row >= 0 && now.weight != 0.f) copy_in(now);
        ahead_token<T>(now, a);
        ahead_load(next, P, now.row < 0 ? -1 : dealer_next(d, a, q, n_clusters));
        for (bool first = true; ok; first = false) {
            ahead_token<T>(next, a);
            RowAhead after;
            ahead_load(after, P, next.row < 0 ? -1 : dealer_next(d, a, q, n_clusters));
            ok = wait(&S.job_empty[job.at], job.phase ^ 1u);
            if (!ok) break;
            if (lane == 0) {
                RowJob& j = S.jobs[job.at];
                j.row = int32_t(now.row);
                if (now.row >= 0) {
                    j.token = now.token;
                    j.live = now.weight != 0.f;
                    j.weight = now.weight;
                    j.x_t = now.x_t;
                    j.in0 = now.in0;
                    j.in1 = now.in1;
                    j.in2 = now.in2;
                    row_scale(j, a, now.T);
                }
                arrive(&S.job_full[job.at]);
            }
            __syncwarp();
            job.next(kJobs);
            if (now.row < 0) break;
            if (!first && now.weight != 0.f) copy_in(now);
            now = next;
            next = after;
        }
        if (!ok) {
            gave_up(S, P, -1);
            // copies in flight land before the CTA may exit
            for (uint32_t j = issued > slots ? issued - slots : 0; j < issued; ++j) wait(&S.full[j % slots], j / slots & 1u);
        }
    } else if (warp == kCloser) {
        const float grad_scale =
            kGrad && P.mode == kModePolicy ? scale_of_grad(P.policy.grad_scale, P.policy.grad_scale_dev) : 1.f;
        Place jp{0, 0}, sp{0, 0};
        for (;;) {
            if (!wait(&S.job_full[jp.at], jp.phase)) {
                gave_up(S, P, -1);
                break;
            }
            const RowJob job = S.jobs[jp.at];
            if (job.row < 0) break;
            Stats st = stats_empty();
            if (job.live) {
                if (lane == 0) mbar_arrive_expect_tx(&S.join[sp.at], kWarps * parts * 16u);
                __syncwarp();
                if (!wait(&S.join[sp.at], sp.phase)) {
                    gave_up(S, P, job.row);
                    break;
                }
                const float4* in = sums + sp.at * parts * kWarps;
                for (uint32_t i = lane; i < parts * kWarps; i += 32) {
                    const float4 p = in[i];
                    Stats o{p.x, p.y, p.z};
                    const float ref = fmaxf(st.ref, o.ref);
                    stats_move(st, ref, job.c);
                    stats_move(o, ref, job.c);
                    st.s += o.s;
                    st.t += o.t;
                }
                stats_warp<kEntropy>(st, job.c);
            }
            RowRecord rec;
            RowOut out;
            row_close(P, job, st, grad_scale, rec, out);
            if (job.live) {
                if (lane == 0) {
                    if (kGrad) S.rec[sp.at] = rec;
                    arrive(&S.closed[sp.at]);
                }
                sp.next(kSums);
            }
            if (rank == 0 && lane == 0) row_write(P, job.row, rec, out);
            __syncwarp();
            if (lane == 0) arrive(&S.job_empty[jp.at]);
            jp.next(kJobs);
        }
    } else {
        // pass 1's row, pass 2's row (the same, or the one before), and what has been waited for of `closed`
        Place jp{0, 0}, slot1{0, 0}, slot2{0, 0}, sp{0, 0}, cp{0, 0};
        uint32_t behind = 0;  // rows taken in pass 1 and not finished
        int32_t prev = -1;    // job of the row before, where it waits for pass 2
        uint32_t prev_at = 0;
        bool ok = true;
        // pass 2 of a job's row, or its fill where it is left out
        auto finish = [&](uint32_t at) {
            const RowJob& job = S.jobs[at];
            const int64_t r = job.row;
            const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
            T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
            const RowPart part = row_part(x, a.vocab, rank, plan.part_vecs);
            const bool whole = ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
            if (!job.live) {
                for (int i = part.first + tid; i < part.last; i += kConsumers)
                    put_vector(g, int(a.vocab), part.span, i, whole, make_uint4(0u, 0u, 0u, 0u));
                return true;
            }
            if (!wait(&S.closed[cp.at], cp.phase)) return false;
            const RowRecord rec = S.rec[cp.at];
            cp.next(kSums);
            const int tok = rec.token < kNoToken ? rec.token + part.span.head : -1;
            for (int i = part.first + tid; i < part.end; i += kChunkVecs) {
                const uint4* in = reinterpret_cast<const uint4*>(ring + slot2.at * kChunkBytes) + tid;
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int ik = i + k * kConsumers;
                    if (ik < part.last)
                        put_vector(g, int(a.vocab), part.span, ik, whole,
                                   gradient<T, kEntropy>(in[k * kConsumers], rec, tok - ik * Elems<T>::kPer));
                }
                __syncwarp();
                if (lane == 0) arrive(&S.empty[slot2.at]);
                slot2.next(slots);
            }
            return true;
        };
        for (;;) {
            if (!wait(&S.job_full[jp.at], jp.phase)) {
                gave_up(S, P, -1);
                break;
            }
            const RowJob& job = S.jobs[jp.at];
            const int32_t row = job.row;
            if (row >= 0 && job.live) {
                const T* x = static_cast<const T*>(a.logits) + int64_t(row) * a.row_stride;
                const RowPart part = row_part(x, a.vocab, rank, plan.part_vecs);
                const float c_hi = job.c_hi, c_lo = job.c_lo;
                Stats st = stats_empty();
                bool bad = false;
                for (int i = part.first + tid; i < part.end; i += kChunkVecs) {
                    ok = wait(&S.full[slot1.at], slot1.phase);
                    if (!ok) break;
                    const uint4* in = reinterpret_cast<const uint4*>(ring + slot1.at * kChunkBytes) + tid;
                    const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
                    uint4 v[kVecs];
                    bool edge = i == 0;
#pragma unroll
                    for (int k = 0; k < kVecs; ++k) {
                        const int ik = i + k * kConsumers;
                        v[k] = make_uint4(none, none, none, none);
                        if (ik < part.last) v[k] = in[k * kConsumers];
                        edge = edge || ik == part.span.count - 1;
                    }
                    if (edge) {
                        constexpr int kPer = Elems<T>::kPer;
                        const int hi = int(a.vocab) + part.span.head;
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) {
                            const int at = (i + k * kConsumers) * kPer;
                            Elems<T>::mask(v[k], part.span.head - at, hi - at);
                        }
                    }
                    fold<T, kEntropy, kVecs>(st, bad, v, c_hi, c_lo);
                    if (!kGrad) {
                        __syncwarp();
                        if (lane == 0) arrive(&S.empty[slot1.at]);
                    }
                    slot1.next(slots);
                }
                if (bad) st.s = quiet_nan();
                stats_warp<kEntropy>(st, job.c);
                // A buffer of sums is written again four rows later. By then this CTA has closed the row two
                // before this one, so every warp of the cluster had come to that row's join, and each had
                // seen the row two before that closed in its own CTA: all closers are done with the buffer.
                // (With a gradient, finish() has waited for it.)
                if (!kGrad) {
                    if (behind == 2) {
                        ok = ok && wait(&S.closed[cp.at], cp.phase);
                        cp.next(kSums);
                    } else {
                        ++behind;
                    }
                }
                if (!ok) {
                    gave_up(S, P, row);
                    break;
                }
                if (uint32_t(lane) < parts)
                    put_sums(dsmem_map(smem_addr(sums + (sp.at * parts + rank) * kWarps + warp), lane),
                             dsmem_map(smem_addr(&S.join[sp.at]), lane), st.ref, st.s, st.t, 0.f);
                sp.next(kSums);
            }
            const uint32_t at = jp.at;
            jp.next(kJobs);
            if (kGrad) {
                const bool held = plan.deep != 0;
                const int32_t target = held ? prev : row;
                const uint32_t target_at = held ? prev_at : at;
                prev = row;
                prev_at = at;
                if (target >= 0) {
                    if (!finish(target_at)) {
                        gave_up(S, P, target);
                        break;
                    }
                    __syncwarp();
                    if (lane == 0) arrive(&S.job_empty[target_at]);
                }
            } else if (row >= 0) {
                __syncwarp();
                if (lane == 0) arrive(&S.job_empty[at]);
            }
            if (row < 0) break;
        }
    }
    // no CTA leaves while another may still write to its shared memory
    __syncwarp();
    cluster_sync();
    if (P.mode == kModePolicy && rank == 0) {  // the first CTAs have written the rows' shares
        const uint32_t end = last_block(P.ws.ticket, n_clusters, &S.flag);
        if (end) {
            const double loss = sum_terms<kThreads>(P.ws.terms, a.n_rows, S.scratch);
            if (tid == 0) *P.policy.out_loss = end & kGaveUp ? quiet_nan() : float(loss);
        }
    }
}

// ---------------------------------------------------------------- pairs
constexpr int kPairThreads = 256;

// Sums of one answer's rows: weight * (logprob - ref_logprob), and weight.
__device__ __forceinline__ void answer_sums(const sampler_rows_t& a, const sampler_preference_t& q, const double* lp,
                                            int64_t begin, int64_t end, double* scratch, double* sum, double* count)
{
    double s = 0.0, n = 0.0;
    for (int64_t r = begin + threadIdx.x; r < end; r += kPairThreads) {
        const float w = a.weight ? a.weight[r] : 1.f;
        if (w == 0.f) continue;
        s += double(w) * (lp[r] - (q.ref_logprob ? double(q.ref_logprob[r]) : 0.0));
        n += double(w);
    }
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        scratch[warp] = s;
        scratch[kPairThreads / 32 + warp] = n;
    }
    __syncthreads();
    s = n = 0.0;
    for (int w = 0; w < kPairThreads / 32; ++w) {
        s += scratch[w];
        n += scratch[kPairThreads / 32 + w];
    }
    *sum = s;
    *count = n;
}

// One block for a pair: the two answers' sums, the pair's share of the loss,
// and the gradient's factors of their rows.
__global__ void __launch_bounds__(kPairThreads) pairs_kernel(const sampler_rows_t a, const sampler_preference_t q,
                                                             const RowWorkspace ws)
{
    __shared__ double scratch[2 * kPairThreads / 32];
    __shared__ uint32_t flag;
    const int64_t i = blockIdx.x;
    int64_t at[2][2];
    double sum[2], share[2], reward[2];
    for (int k = 0; k < 2; ++k) {
        const int64_t b = q.seq_offsets[2 * i + k], e = q.seq_offsets[2 * i + k + 1];
        const bool ok = b >= 0 && b <= e && e <= a.n_rows;
        at[k][0] = ok ? b : 0;
        at[k][1] = ok ? e : 0;
        double count;
        answer_sums(a, q, ws.terms, at[k][0], at[k][1], scratch, &sum[k], &count);
        share[k] = !q.mean_over_tokens ? 1.0 : count != 0.0 ? 1.0 / count : 0.0;
        reward[k] = ok ? double(q.beta) * (sum[k] * share[k]) : double(quiet_nan());
        if (threadIdx.x == 0 && q.out_reward) q.out_reward[2 * i + k] = float(reward[k]);
    }
    const double z = reward[0] - reward[1] - double(q.margin);
    const double eps = double(q.label_smoothing);
    if (threadIdx.x == 0) {
        // -ln sigmoid(z) = max(-z, 0) + ln(1 + exp(-|z|)); a share of 0 takes no part, even of an infinity
        const double tail = log1p(exp(-fabs(z)));
        const double chosen = eps != 1.0 ? (1.0 - eps) * (fmax(-z, 0.0) + tail) : 0.0;
        const double other = eps != 0.0 ? eps * (fmax(z, 0.0) + tail) : 0.0;
        ws.pair_terms[i] = isnan(z) ? z : chosen + other;
    }
    if (a.out_grad) {
        const double by_z = 1.0 / (1.0 + exp(-z)) - (1.0 - eps);
        const float scale = scale_of_grad(q.grad_scale, q.grad_scale_dev);
        for (int k = 0; k < 2; ++k) {
            const float by_sum = float((k ? -by_z : by_z) * double(q.beta) * share[k] / double(q.n_pairs)) * scale;
            for (int64_t r = at[k][0] + threadIdx.x; r < at[k][1]; r += kPairThreads) {
                RowRecord rec = ws.records[r];
                if (rec.token < 0) continue;
                set_factors(rec, (a.weight ? a.weight[r] : 1.f) * by_sum, 0.f, 0.f, 0.f);
                ws.records[r] = rec;
            }
        }
    }
    if (last_block(ws.ticket, gridDim.x, &flag) != 0u) {
        const double loss = sum_terms<kPairThreads>(ws.pair_terms, q.n_pairs, scratch);
        if (threadIdx.x == 0) *q.out_loss = float(loss / double(q.n_pairs));
    }
}

// The gradient of rows whose records are complete, the last rows first: those
// are what the pass before this one has left in L2. One block a row and part.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;  // vectors of a thread in flight

template <typename T>
__global__ void __launch_bounds__(kGradThreads) pairs_grad_kernel(const sampler_rows_t a, const RowWorkspace ws)
{
    const int64_t r = a.n_rows - 1 - int64_t(blockIdx.y);
    const RowRecord rec = ws.records[r];
    const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
    T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
    const RowSpan span = row_span(x, a.vocab);
    const bool whole = ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
    const uint4* from = reinterpret_cast<const uint4*>(x - span.head);
    const int first = int(blockIdx.x) * kGradThreads * kGradVecs + threadIdx.x;
    const bool zero = rec.token < 0 || (rec.k0 == 0.f && rec.at_token == 0.f);
    const int tok = rec.token < kNoToken ? rec.token + span.head : -1;
    uint4 v[kGradVecs];
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
        const int i = first + k * kGradThreads;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (!zero && i < span.count) v[k] = __ldcs(from + i);
    }
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
        const int i = first + k * kGradThreads;
        if (i < span.count)
            put_vector(g, int(a.vocab), span, i, whole,
                       zero ? v[k] : gradient<T, false>(v[k], rec, tok - i * Elems<T>::kPer));
    }
}

}  // namespace rows

namespace {

using RowsKernel = void (*)(const LossParams, const rows::RowPlan);

template <typename T>
RowsKernel rows_kernel_for(bool grad, bool entropy)
{
    return grad ? entropy ? rows::rows_kernel<T, true, true> : rows::rows_kernel<T, true, false>
           : entropy ? rows::rows_kernel<T, false, true>
                     : rows::rows_kernel<T, false, false>;
}

}  // namespace

int rows_launch(const LossParams& p, int sms, RowOccupancy* occ, cudaStream_t stream)
{
    const bool grad = p.rows.out_grad && p.mode != kModePairs;
    const bool entropy = p.rows.out_entropy || (p.mode == kModeScoreGrad && p.grad_entropy) ||
                         (p.mode == kModePolicy && p.policy.entropy_coef != 0.f);
    const int es = p.rows.dtype == SAMPLER_DTYPE_BF16 ? 2 : 4;
    const RowsKernel kernel = es == 2 ? rows_kernel_for<uint16_t>(grad, entropy) : rows_kernel_for<float>(grad, entropy);
    // vectors of a row that starts anywhere
    const int64_t vecs = (p.rows.vocab + 2 * (16 / es - 1)) * es / 16 + 1;
    // parts of at most kPartChunks chunks, of which two fit in the ring; smaller ones while few rows leave the
    // device unfilled
    int parts = 1;
    while (parts < rows::kMaxParts && ((vecs + parts - 1) / parts > rows::kPartChunks * rows::kChunkVecs ||
                                       p.rows.n_rows * parts * 2 <= sms))
        parts *= 2;
    rows::RowPlan plan;
    plan.part_vecs = int((vecs + parts - 1) / parts);
    plan.slots = rows::slots_for(parts);
    plan.deep = 2 * ((plan.part_vecs + rows::kChunkVecs - 1) / rows::kChunkVecs) <= plan.slots;
    const int smem = rows::smem_of(plan.slots, parts);
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(rows::kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {unsigned(parts), 1u, 1u};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int& resident = occ->clusters[es == 2][grad][entropy][parts == 1 ? 0 : parts == 2 ? 1 : parts == 4 ? 2 : parts == 8 ? 3 : 4];
    if (resident < 1) {  // once for each kernel and cluster size of a handle
        const void* k = reinterpret_cast<const void*>(kernel);
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, rows::kSmemMax) !=
                cudaSuccess ||
            (parts > 8 && cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess))
            return SAMPLER_ERR_CUDA;
        cfg.gridDim = dim3(unsigned(parts));
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return SAMPLER_ERR_CUDA;
        resident = n;
    }
    const int clusters = int(std::min<int64_t>(p.rows.n_rows, resident));
    cfg.gridDim = dim3(unsigned(clusters * parts));
    return cudaLaunchKernelEx(&cfg, kernel, p, plan) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

int pairs_launch(const sampler_rows_t& rows, const sampler_preference_t& pref, const RowWorkspace& ws,
                 cudaStream_t stream)
{
    rows::pairs_kernel<<<unsigned(pref.n_pairs), rows::kPairThreads, 0, stream>>>(rows, pref, ws);
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

int pairs_grad_launch(const sampler_rows_t& rows, const RowWorkspace& ws, cudaStream_t stream)
{
    const int es = rows.dtype == SAMPLER_DTYPE_BF16 ? 2 : 4;
    const int64_t vecs = (rows.vocab + 2 * (16 / es - 1)) * es / 16 + 1;
    constexpr int kPer = rows::kGradThreads * rows::kGradVecs;
    sampler_rows_t some = rows;
    RowWorkspace at = ws;
    for (int64_t done = 0; done < rows.n_rows; done += 65535) {  // the last rows first
        some.n_rows = std::min<int64_t>(rows.n_rows - done, 65535);
        const int64_t base = rows.n_rows - done - some.n_rows;
        some.logits = static_cast<const char*>(rows.logits) + base * rows.row_stride * es;
        some.out_grad = static_cast<char*>(rows.out_grad) + base * rows.grad_stride * es;
        at.records = ws.records + base;
        const dim3 grid(unsigned((vecs + kPer - 1) / kPer), unsigned(some.n_rows));
        if (es == 2)
            rows::pairs_grad_kernel<uint16_t><<<grid, rows::kGradThreads, 0, stream>>>(some, at);
        else
            rows::pairs_grad_kernel<float><<<grid, rows::kGradThreads, 0, stream>>>(some, at);
    }
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
