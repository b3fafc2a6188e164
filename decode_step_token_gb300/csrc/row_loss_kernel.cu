// row_loss_kernel.cu -- scoring and the losses over logits rows: logprob,
// entropy, the clipped policy loss, the preference loss, and the logits'
// gradients.
//
// A row's gradient needs the row's sums, so a row is wanted twice, and is read
// from memory once: a cluster of C CTAs takes a row, each CTA a part of it in
// shared memory, where the second pass finds it. One warp of a CTA (the
// producer) goes ahead over the cluster's rows and brings their parts in with
// bulk copies through a ring of 8 KB chunks; sixteen (the consumers) take
//   pass 1   a vector of each chunk in every thread: the running reference and
//            the sums of exponentials;
//   join     each warp puts its sums into every CTA of the cluster (distributed
//            shared memory) and arrives there on a barrier; one warp of each CTA
//            combines all of them and works out the gradient's factors;
//   pass 2   (with a gradient) the same vectors again from the ring: 16-byte
//            stores of the gradient, and each chunk's slot goes back to the
//            producer, which fills it for the next row.
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
constexpr int kThreads = kConsumers + 32;
constexpr int kChunkVecs = kConsumers;           // 16-byte vectors of a chunk: one for each consumer
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kSlots = 12;
constexpr int kMaxParts = 16;                    // CTAs of a cluster
constexpr int kJobs = 4;                         // rows that the producer may be ahead, in shared memory
constexpr uint64_t kWaitNs = 2000000000ull;      // a wait gives up after 2 s

struct Shared {
    alignas(128) unsigned char ring[kSlots][kChunkBytes];
    float4 sums[2][kMaxParts * kWarps];          // ref, s, t of each warp of the cluster, x_t of a CTA's first
    uint64_t full[kSlots], empty[kSlots];
    uint64_t job_full[kJobs], job_empty[kJobs];
    uint64_t join[2], closed[2];
    RowJob jobs[kJobs];
    RowRecord rec[2];
    double scratch[kThreads / 32];
    uint32_t flag, failed;  // failed: a wait of this CTA gave up
};

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase of `bar` with the given parity, for kWaitNs at most.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity)
{
    const uint64_t until = now_ns() + kWaitNs;
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u && now_ns() > until) return false;
    }
    return false;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity)
{
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity);
}

__device__ __forceinline__ void arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// The same wait with the cluster's writes before the arrivals made visible.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity)
{
    uint64_t until = 0;
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63u) == 63u) {
            const uint64_t now = now_ns();
            if (until == 0) until = now + kWaitNs;
            if (now > until) return false;
        }
    }
    return false;
}

__device__ __forceinline__ void put_sums(uint32_t addr, float a, float b, float c, float d)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
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

// Pass 1 over kVecs vectors. The reference moves only when a vector holds a
// larger element, which is rare after the first few.
template <typename T, bool kEntropy, int kVecs>
__device__ __forceinline__ void fold(Stats& st, bool& bad, const uint4 (&v)[kVecs], float c_hi, float c_lo)
{
    constexpr int kPer = Elems<T>::kPer;
    float m = Elems<T>::largest(v[0]);
#pragma unroll
    for (int k = 1; k < kVecs; ++k) m = max_nan(m, Elems<T>::largest(v[k]));
    if (!(m <= st.ref)) {
        if (m < pos_inf())
            stats_move(st, m, c_hi);
        else
            bad = true;
    }
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        float x[kPer];
        Elems<T>::widen(v[k], x);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float d = x[j] - st.ref;
            const float u = fmaf(d, c_hi, d * c_lo);
            const float e = exp2_fast(u);
            if (j & 1)
                s1 += e;
            else
                s0 += e;
            if (kEntropy) st.t = fmaf(e, fmaxf(u, kLowest), st.t);
        }
    }
    st.s += s0 + s1;
}

// Pass 2 of one vector; `at` is the token's place in it (outside [0, kPer): not in it).
template <typename T, bool kEntropy>
__device__ __forceinline__ uint4 gradient(const uint4& v, const RowRecord& rec, int at)
{
    constexpr int kPer = Elems<T>::kPer;
    float x[kPer];
    Elems<T>::widen(v, x);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const float d = x[j] - rec.ref;
        if (kEntropy) {
            const float u = fmaxf(d * rec.c, kLowest);
            x[j] = exp2_fast(u) * fmaf(rec.k1, u, rec.k0);
        } else {
            x[j] = exp2_fast(d * rec.c) * rec.k0;
        }
    }
    if (unsigned(at) < unsigned(kPer)) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j == at) x[j] += rec.at_token;
    }
    return Elems<T>::round(x);
}

// Store vector `i` of a row's span to the gradient: as one where it lies wholly
// inside the row and the gradient's vectors lie as the logits' do, else by element.
template <typename T>
__device__ __forceinline__ void put_vector(T* g, int64_t vocab, int head, int64_t i, bool whole, const uint4& y)
{
    constexpr int kPer = Elems<T>::kPer;
    const int64_t first = i * kPer - head;
    if (whole && first >= 0 && first + kPer <= vocab) {
        __stcs(reinterpret_cast<uint4*>(g + first), y);
    } else {
        const T* e = reinterpret_cast<const T*>(&y);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (first + j >= 0 && first + j < vocab) g[first + j] = e[j];
    }
}

// A CTA's part of a row's gradient, all the same value (zeros, or NaN).
template <typename T>
__device__ __forceinline__ void fill(T* g, const RowSpan& span, int64_t vocab, int first, int last, int tid, bool whole,
                                     bool nan)
{
    const uint32_t w = !nan ? 0u : sizeof(T) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
    for (int i = first + tid; i < last; i += kConsumers)
        put_vector(g, vocab, span.head, i, whole, make_uint4(w, w, w, w));
}

// ---------------------------------------------------------------- the kernel
// The rows of cluster `q` of `n_clusters`, in order: every n_clusters-th of those
// that count, and every n_clusters-th of those that are left out. One warp.
struct RowDealer {
    int64_t base;            // first row of the 32 in `mine`
    uint32_t mine;           // those of them that are this cluster's and have not been given out
    uint32_t live, dead;     // rows of either kind before `base`, modulo n_clusters
    float weight;            // this lane's row of the next 32
};

__device__ __forceinline__ void dealer_load(RowDealer& d, const sampler_rows_t& a, int64_t base)
{
    const int64_t r = base + (threadIdx.x & 31);
    d.weight = a.weight && r < a.n_rows ? a.weight[r] : 1.f;
}

// The next row, -1 at the end.
__device__ __forceinline__ int64_t dealer_next(RowDealer& d, const sampler_rows_t& a, uint32_t q, uint32_t n_clusters)
{
    const uint32_t lane = threadIdx.x & 31;
    while (d.mine == 0) {
        d.base += 32;
        if (d.base >= a.n_rows) return -1;
        const bool in = d.base + lane < a.n_rows;
        const bool counts = d.weight != 0.f;
        const uint32_t live = __ballot_sync(0xffffffffu, in && counts), dead = __ballot_sync(0xffffffffu, in && !counts);
        const uint32_t before = (1u << lane) - 1u;
        const uint32_t rank = counts ? d.live + __popc(live & before) : d.dead + __popc(dead & before);
        d.mine = __ballot_sync(0xffffffffu, in && rank % n_clusters == q);
        d.live = (d.live + __popc(live)) % n_clusters;
        d.dead = (d.dead + __popc(dead)) % n_clusters;
        dealer_load(d, a, d.base + 32);
    }
    const int bit = __ffs(d.mine) - 1;
    d.mine &= d.mine - 1u;
    return d.base + bit;
}

// kGrad: with the logits' gradient. kEntropy: with the sum t. The grid is whole
// clusters of `parts` CTAs; part_vecs: vectors of a row in each CTA.
template <typename T, bool kGrad, bool kEntropy>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const __grid_constant__ LossParams P, int part_vecs)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Shared& S = *reinterpret_cast<Shared*>(smem_raw);
    const sampler_rows_t& a = P.rows;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t parts = cluster_nctarank(), rank = cluster_ctarank();
    const uint32_t q = blockIdx.x / parts, n_clusters = gridDim.x / parts;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], kWarps);
        }
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&S.job_full[i], 1);
            mbar_init(&S.job_empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.join[i], kWarps * parts);
            mbar_init(&S.closed[i], 1);
        }
        S.failed = 0;
        fence_mbar_init();
    }
    cluster_sync();

    if (warp == kWarps) {  // producer
        RowDealer d{-32, 0, 0, 0, 1.f};
        dealer_load(d, a, 0);
        uint32_t chunk = 0;  // of all rows
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            const int64_t r = dealer_next(d, a, q, n_clusters);
            RowJob job;
            if (r >= 0)
                job = row_open(P, r);
            else
                job.row = -1;
            const uint32_t slot = n % kJobs;
            ok = wait(&S.job_empty[slot], (n / kJobs & 1u) ^ 1u);
            if (lane == 0) {
                S.jobs[slot] = job;
                arrive(&S.job_full[slot]);
            }
            __syncwarp();
            if (!ok || r < 0) break;
            if (!job.live || job.bad_param) continue;
            const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
            const RowSpan span = row_span(x, a.vocab);
            const int first = int(rank) * part_vecs, last = min(first + part_vecs, span.count);
            const unsigned char* from = reinterpret_cast<const unsigned char*>(x - span.head);
            for (int v = first; ok && v < last; v += kChunkVecs, ++chunk) {
                const uint32_t s = chunk % kSlots;
                ok = wait(&S.empty[s], (chunk / kSlots & 1u) ^ 1u);
                if (ok && lane == 0) {
                    const uint32_t bytes = uint32_t(min(kChunkVecs, last - v)) * 16u;
                    mbar_arrive_expect_tx(&S.full[s], bytes);
                    bulk_copy_g2s(S.ring[s], from + size_t(v) * 16, bytes, &S.full[s]);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            gave_up(S, P, -1);
            // copies in flight land before the CTA may exit
            for (uint32_t j = chunk > kSlots ? chunk - kSlots : 0; j < chunk; ++j)
                wait(&S.full[j % kSlots], j / kSlots & 1u);
        }
    } else {
        uint32_t chunk = 0, joins = 0;
        const float grad_scale =
            kGrad && P.mode == kModePolicy ? scale_of_grad(P.policy.grad_scale, P.policy.grad_scale_dev) : 1.f;
        for (uint32_t n = 0;; ++n) {
            const uint32_t slot = n % kJobs;
            if (!wait(&S.job_full[slot], n / kJobs & 1u)) {
                gave_up(S, P, -1);
                break;
            }
            const RowJob job = S.jobs[slot];
            __syncwarp();
            if (lane == 0) arrive(&S.job_empty[slot]);
            if (job.row < 0) break;
            const int64_t r = job.row;
            const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
            T* g = kGrad ? static_cast<T*>(a.out_grad) + r * a.grad_stride : nullptr;
            const RowSpan span = row_span(x, a.vocab);
            const bool whole = kGrad && ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
            const int first = int(rank) * part_vecs, last = max(first, min(first + part_vecs, span.count));
            const bool closes = warp == 0;
            const bool writes = rank == 0 && warp == 0 && lane == 0;
            RowRecord rec;
            if (!job.live || job.bad_param) {
                if (closes) row_close(P, job, stats_empty(), 0.f, grad_scale, writes, rec);
                if (kGrad) fill(g, span, a.vocab, first, last, tid, whole, job.live != 0);
                continue;
            }
            const float x_t = closes ? load_logit(x + job.token) : 0.f;
            // pass 1
            Stats st = stats_empty();
            bool bad = false, ok = true;
            const int mine = last - first - tid;  // this thread has vectors first + tid + kChunkVecs * j
            const int chunks = (last - first + kChunkVecs - 1) / kChunkVecs;
            const int edge_lo = 0, edge_hi = span.count - 1;
            for (int j = 0; j < chunks; j += 2) {
                const uint32_t c0 = chunk + j, s0 = c0 % kSlots, c1 = c0 + 1, s1 = c1 % kSlots;
                const bool two = j + 1 < chunks;
                ok = ok && wait(&S.full[s0], c0 / kSlots & 1u);
                if (two) ok = ok && wait(&S.full[s1], c1 / kSlots & 1u);
                if (!ok) break;
                uint4 v[2];
                const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
                v[0] = v[1] = make_uint4(none, none, none, none);
                const int i0 = first + tid + kChunkVecs * j, i1 = i0 + kChunkVecs;
                if (mine > kChunkVecs * j) v[0] = reinterpret_cast<const uint4*>(S.ring[s0])[tid];
                if (mine > kChunkVecs * (j + 1)) v[1] = reinterpret_cast<const uint4*>(S.ring[s1])[tid];
                if (i0 == edge_lo || i0 == edge_hi || i1 == edge_hi) {
                    constexpr int kPer = Elems<T>::kPer;
                    const int hi = int(a.vocab) + span.head;
                    Elems<T>::mask(v[0], span.head - i0 * kPer, hi - i0 * kPer);
                    Elems<T>::mask(v[1], span.head - i1 * kPer, hi - i1 * kPer);
                }
                fold<T, kEntropy, 2>(st, bad, v, job.c_hi, job.c_lo);
                if (!kGrad) {
                    __syncwarp();
                    if (lane == 0) {
                        arrive(&S.empty[s0]);
                        if (two) arrive(&S.empty[s1]);
                    }
                }
            }
            if (!ok) {
                gave_up(S, P, r);
                break;
            }
            if (bad) st.s = quiet_nan();
            stats_warp(st, job.c);
            // join
            const uint32_t buf = joins & 1u;
            // a buffer is written again once every warp of the cluster has come to the join after its last
            // use (with a gradient, the wait for `closed` below has seen to that)
            if (!kGrad && joins > 0) ok = wait_cluster(&S.join[buf ^ 1u], (joins - 1u) >> 1 & 1u);
            if (ok && uint32_t(lane) < parts) {
                put_sums(dsmem_map(smem_addr(&S.sums[buf][rank * kWarps + warp]), lane), st.ref, st.s, st.t, x_t);
                arrive_cluster(dsmem_map(smem_addr(&S.join[buf]), lane));
            }
            if (ok && closes) {
                ok = wait_cluster(&S.join[buf], joins >> 1 & 1u);
                if (ok) {
                    st = stats_empty();
                    for (uint32_t i = lane; i < parts * kWarps; i += 32) {
                        const float4 p = S.sums[buf][i];
                        Stats o{p.x, p.y, p.z};
                        const float ref = fmaxf(st.ref, o.ref);
                        stats_move(st, ref, job.c);
                        stats_move(o, ref, job.c);
                        st.s += o.s;
                        st.t += o.t;
                    }
                    stats_warp(st, job.c);
                    row_close(P, job, st, x_t, grad_scale, writes, rec);
                    if (kGrad && lane == 0) {
                        S.rec[buf] = rec;
                        arrive(&S.closed[buf]);
                    }
                }
            }
            if (kGrad) ok = ok && wait(&S.closed[buf], joins >> 1 & 1u);
            if (!ok) {
                gave_up(S, P, r);
                break;
            }
            ++joins;
            if (kGrad) {
                rec = S.rec[buf];
                // pass 2
                const int tok = rec.token < kNoToken ? rec.token + span.head : -1;
                for (int j = 0; j < chunks; ++j) {
                    const uint32_t s = (chunk + j) % kSlots;
                    if (mine > kChunkVecs * j) {
                        const int64_t i = first + tid + kChunkVecs * j;
                        const uint4 v = reinterpret_cast<const uint4*>(S.ring[s])[tid];
                        put_vector(g, a.vocab, span.head, i, whole,
                                   gradient<T, kEntropy>(v, rec, tok - int(i) * Elems<T>::kPer));
                    }
                    __syncwarp();
                    if (lane == 0) arrive(&S.empty[s]);
                }
            }
            chunk += chunks;
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
            put_vector(g, a.vocab, span.head, i, whole,
                       zero ? v[k] : gradient<T, false>(v[k], rec, tok - i * Elems<T>::kPer));
    }
}

}  // namespace rows

namespace {

using RowsKernel = void (*)(const LossParams, int);

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
    int parts = 1;
    while (parts < rows::kMaxParts &&
           ((vecs + parts - 1) / parts > 8 * rows::kChunkVecs || p.rows.n_rows * parts * 2 <= sms))
        parts *= 2;
    const int part_vecs = int((vecs + parts - 1) / parts);
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(rows::kThreads);
    cfg.dynamicSmemBytes = sizeof(rows::Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {unsigned(parts), 1u, 1u};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int& resident = occ->clusters[es == 2][grad][entropy][parts == 1 ? 0 : parts == 2 ? 1 : parts == 4 ? 2 : parts == 8 ? 3 : 4];
    if (resident < 1) {  // once for each kernel and cluster size of a handle
        const void* k = reinterpret_cast<const void*>(kernel);
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(rows::Shared))) !=
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
    return cudaLaunchKernelEx(&cfg, kernel, p, part_vecs) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
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
