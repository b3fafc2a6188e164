// distill_kernel.cu -- distillation from a teacher's most likely tokens: the loss of
// rows of logits against lists of tokens with logprobs, and the logits' gradient.
//
// With S a row's list, q_j = exp(l_j) its masses, q_r the mass outside, W = sum q_j + q_r, h = token_coef
// and p_r = sum_{v not in S} p_v,
//     KL = sum_j q_j (l_j - ln p_j) + q_r (ln q_r - ln p_r),
//     T d loss / d x_v = (p_v / p_r) ((W + h) p_r - q_r)  outside the list,
//                        (W + h) p_j - q_j                inside,     and -h at the row's token.
// The two sides of the list are kept apart from the start: the sums of the tokens outside have their own reference, so
// that p_r is a sum and not a difference, however little it is, and an element outside is one exponential times one
// factor of the row. The list's own terms are taken one by one, with the accurate exponential, and added up as pairs
// of fp32: a divergence is a small difference of logprobs.
//
// As in the other losses (row_loss_kernel.cu) a cluster of C CTAs takes a row, each CTA a part of it in shared memory
// between the two passes, so that each logit is read once and each gradient written once. Here a part is one buffer,
// of which a CTA has two to four. Warp roles of a CTA:
//   producer   goes ahead over the cluster's rows and brings their parts in with bulk copies;
//   closers    (two, a row each in turn) mark the list's tokens of a part in a map of bits, a byte for each vector,
//              before pass 1; take their logits from the buffer and put their share of the list's sums into all CTAs of
//              the cluster; combine what all have put, work out the row's factors, write the row's outputs, and put the
//              list's own gradients into the buffer in their logits' place;
//   consumers  (sixteen, of short rows four) pass 1: the running reference and sum of what is not marked; pass 2: the
//              gradient, marked elements as they now are in the buffer. A row's pass 1 comes before the pass 2 of the row
//              before it, so that the join and the closer's work run under it.
//
// One CTA an SM (of short rows three). 4096 x 128000 bf16 with gradient, lists of 64, 0.9 of the rows counted: 378 us, 0.78
// of the copy rate over what has to move. Two CTAs of eight consumers an SM, with parts of half the size and twice as many: 475 us (twice
// the joins and closers' turns of a row). What bounds it now is the consumers' instructions, which take 0.68 of the issue
// slots: an exponential and packed arithmetic around it for each element in each pass.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "row_loss.cuh"
#include "row_queue.cuh"
#include "row_vectors.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace distill {

using namespace rows;

constexpr int kLongWarps = 16, kShortWarps = 4;  // consumers of a CTA, one or three on an SM
constexpr int kClosers = 2;                      // warps, of which each takes every other row
constexpr int kVecs = 4;                     // vectors that a consumer folds at once
constexpr int kMaxBuffers = 4;
constexpr int kMaxParts = 16;                // CTAs of a cluster
constexpr int kMaps = 3;                     // rows whose tokens are marked
constexpr int kSums = 4;                     // rows whose sums are in shared memory
constexpr int kHeld = SAMPLER_MAX_ALTERNATIVES / 32;  // of a list in each of the closer's lanes

// What follows from a CTA's number of consumer warps.
template <int kWarps>
struct Shape {
    static constexpr int kConsumers = kWarps * 32;
    static constexpr int kThreads = kConsumers + 32 + 32 * kClosers;
    static constexpr int kStep = kConsumers * kVecs;  // vectors that they take at once
    static constexpr int kResident = kWarps == kShortWarps ? 3 : 1;
    static constexpr int kSmem = (kResident == 1 ? 226 : 75) * 1024;
};
constexpr uint64_t kSettleNs = 100000;       // in which what is on its way to shared memory lands

// What a CTA's closer puts into all CTAs: sums of the list's tokens in its part.
struct ListSums {
    float ref, s;   // exponentials
    Pair a, q;      // q_j (l_j - (x_j - ref) / T) and q_j
    uint32_t flags, pad;
};
static_assert(sizeof(ListSums) == 32, "two stores of 16 bytes");
constexpr uint32_t kBadList = 1, kBadLogit = 2;

// A row's factors for pass 2.
struct Factor {
    float ref, c, k, at_token;
    int token;  // kNoToken: none
};

// A list's token that is in a CTA's part.
struct Entry {
    int at;     // element of the part's buffer
    float l, x, q;
};

struct Shared {
    Entry list[kClosers][SAMPLER_MAX_ALTERNATIVES];
    uint64_t full[kMaxBuffers], empty[kMaxBuffers];
    uint64_t unmarked[kMaps];
    uint64_t join[kSums], closed[kSums];
    RowQueue queue;
    Factor factor[kSums];
    double scratch[kLongWarps + 1 + kClosers];
    uint32_t flag, failed;  // failed: a wait of this cluster gave up
};

// The buffers, the consumers' sums [kSums][parts * kWarps], the closers' [kSums][parts], the maps [kMaps][part_vecs] and
// Shared.
template <int kWarps>
__host__ __device__ constexpr int map_bytes(int part_vecs)
{
    constexpr int kStep = Shape<kWarps>::kStep;
    return (part_vecs + kStep - 1) / kStep * kStep;
}

template <int kWarps>
constexpr int smem_of(int part_vecs, int buffers, int parts)
{
    return buffers * part_vecs * 16 + kSums * parts * (kWarps * 16 + int(sizeof(ListSums))) + kMaps * map_bytes<kWarps>(part_vecs) +
           int(sizeof(Shared));
}

__device__ __noinline__ void gave_up(Shared& S)
{
    const uint32_t cta = threadIdx.x & 31;
    if (cta < cluster_nctarank()) dsmem_st_u32(dsmem_map(smem_addr(&S.failed), cta), 1u);
}

__device__ __forceinline__ void write_row(const DistillParams& P, int64_t r, float kl, float logprob, int status, double term)
{
    if (P.distill.out_kl) P.distill.out_kl[r] = kl;
    if (P.rows.out_logprob) P.rows.out_logprob[r] = logprob;
    if (P.rows.out_status) P.rows.out_status[r] = status;
    P.ws.terms[r] = term;
}

// A wait of this cluster gave up. Which of its rows were done with is not known, so all of them are written again, by all
// CTAs after the last of them has come to its end: those that count as TIMEOUT with NaN, the others as ever.
template <typename T, bool kGrad, int kThreads>
__device__ __noinline__ void abandon(const DistillParams& P, uint32_t q, uint32_t n_clusters, uint32_t parts, uint32_t rank)
{
    // copies, and sums put into this CTA, that nobody has waited for land before it may exit
    const uint64_t until = now_ns() + kSettleNs;
    for (uint32_t i = 0; i < (1u << 20) && now_ns() < until; ++i) {
    }
    const sampler_rows_t& a = P.rows;
    RowDealer d;
    dealer_open(d, a, q);
    for (;;) {
        bool counts;
        const int64_t r = dealer_next(d, a, q, n_clusters, counts);
        if (r < 0) return;
        const float x = counts ? quiet_nan() : 0.f;
        if (rank == 0 && threadIdx.x == 0) write_row(P, r, x, x, counts ? SAMPLER_ROW_TIMEOUT : SAMPLER_ROW_OK, x);
        if (kGrad) {
            T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
            for (int64_t v = rank * kThreads + threadIdx.x; v < a.vocab; v += parts * kThreads) store_grad(g + v, x);
        }
    }
}

// A divergence is a small difference of logprobs: its terms are pairs, and so are their sums.
__device__ __forceinline__ Pair pair_add(const Pair& a, const Pair& b)
{
    const Pair s = two_sum(a.hi, b.hi);
    return Pair{s.hi, s.lo + (a.lo + b.lo)};
}

__device__ __forceinline__ Pair pair_times(float q, const Pair& a)
{
    const float p = q * a.hi;
    return Pair{p, fmaf(q, a.hi, -p) + q * a.lo};
}

// (x - ref) / T of a finite x
__device__ __forceinline__ Pair scaled(const RowJob& h, float x, float ref)
{
    const Pair d = two_sum(x, -ref);
    const float y = d.hi * h.inv_t;
    return Pair{y, fmaf(d.hi, h.inv_t, -y) + fmaf(d.hi, h.inv_t_lo, d.lo * h.inv_t)};
}

// The sum over a warp, in every lane.
__device__ __forceinline__ void pair_warp(Pair& a)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = pair_add(a, Pair{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
}

// Where the byte of a part's vector i is in a map: those of the vectors that a thread takes at once lie side by side.
template <int kWarps>
__device__ __forceinline__ int map_place(int i)
{
    constexpr int kStep = Shape<kWarps>::kStep, kConsumers = Shape<kWarps>::kConsumers;
    return (i & ~(kStep - 1)) | (i & (kConsumers - 1)) * kVecs | (i / kConsumers & (kVecs - 1));
}

// Marked elements of a vector become -inf, or those of `from`.
template <typename T>
__device__ __forceinline__ void blend(uint4& v, const uint4& from, uint32_t bits);
template <>
__device__ __forceinline__ void blend<float>(uint4& v, const uint4& from, uint32_t bits)
{
    if (bits & 1u) v.x = from.x;
    if (bits & 2u) v.y = from.y;
    if (bits & 4u) v.z = from.z;
    if (bits & 8u) v.w = from.w;
}
template <>
__device__ __forceinline__ void blend<uint16_t>(uint4& v, const uint4& from, uint32_t bits)
{
    auto word = [&](uint32_t& w, uint32_t f, uint32_t b) {
        const uint32_t m = (b & 1u ? 0xffffu : 0u) | (b & 2u ? 0xffff0000u : 0u);
        w = (w & ~m) | (f & m);
    };
    word(v.x, from.x, bits);
    word(v.y, from.y, bits >> 2);
    word(v.z, from.z, bits >> 4);
    word(v.w, from.w, bits >> 6);
}

// Whether some of the `step` vectors from `at` on of a row's span are partly beside the row.
__device__ __forceinline__ bool ragged(const RowSpan& span, int end, int at, int per, int step)
{
    return (at == 0 && span.head != 0) || (at + step >= span.count && end % per != 0);
}

template <typename T>
__device__ __forceinline__ uint4 nothing()
{
    const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

template <typename T, bool kGrad, int kWarps>
__global__ void __launch_bounds__(Shape<kWarps>::kThreads, Shape<kWarps>::kResident)
    distill_kernel(const __grid_constant__ DistillParams P)
{
    constexpr int kConsumers = Shape<kWarps>::kConsumers, kThreads = Shape<kWarps>::kThreads, kStep = Shape<kWarps>::kStep;
    constexpr int kProducer = kWarps, kCloser = kWarps + 1;
    constexpr int kPer = Elems<T>::kPer;
    extern __shared__ __align__(128) unsigned char smem[];
    const sampler_rows_t& a = P.rows;
    const sampler_distill_t& D = P.distill;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t parts = cluster_nctarank(), rank = cluster_ctarank();
    const uint32_t q = blockIdx.x / parts, n_clusters = gridDim.x / parts;
    const uint32_t buffers = uint32_t(P.buffers);
    const int buffer_bytes = P.part_vecs * 16;
    float4* sums = reinterpret_cast<float4*>(smem + buffers * buffer_bytes);
    ListSums* lists = reinterpret_cast<ListSums*>(sums + kSums * parts * kWarps);
    unsigned char* maps = reinterpret_cast<unsigned char*>(lists + kSums * parts);
    Shared& S = *reinterpret_cast<Shared*>(maps + kMaps * map_bytes<kWarps>(P.part_vecs));

    if (tid == 0) {
        for (int i = 0; i < kMaxBuffers; ++i) {
            mbar_init(&S.full[i], 2);  // its copy, and its row's marks
            mbar_init(&S.empty[i], kWarps + 1);
        }
        for (int i = 0; i < kMaps; ++i) {
            mbar_init(&S.unmarked[i], kWarps);
        }
        for (int i = 0; i < kSums; ++i) {
            mbar_init(&S.join[i], 1);
            mbar_init(&S.closed[i], 1);
        }
        queue_open(S.queue, kWarps + kClosers);
        S.failed = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < kMaps * map_bytes<kWarps>(P.part_vecs) / 4; i += kThreads) reinterpret_cast<uint32_t*>(maps)[i] = 0;
    cluster_sync();

    const int first_vec = int(rank) * P.part_vecs;
    if (warp == kProducer) {
        RingPlace buf{0, 0};
        uint32_t issued = 0;
        // (wait_ns 0: nothing begins, and every other wait of the cluster gives up)
        const bool ok = P.wait_ns != 0 && queue_fill<T>(S.queue, a, q, n_clusters, a.tokens != nullptr, P.wait_ns, [&](int64_t r) {
            const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
            const RowSpan span = row_span(x, a.vocab);
            const int n = min(first_vec + P.part_vecs, span.count) - first_vec;
            if (!wait(&S.empty[buf.at], buf.phase ^ 1u, P.wait_ns)) return false;
            if (elect_one()) {
                if (n > 0) {
                    mbar_arrive_expect_tx(&S.full[buf.at], uint32_t(n) * 16u);
                    bulk_copy_g2s(smem + buf.at * buffer_bytes,
                                  reinterpret_cast<const unsigned char*>(x - span.head) + size_t(first_vec) * 16, uint32_t(n) * 16u,
                                  &S.full[buf.at]);
                } else {
                    mbar_arrive(&S.full[buf.at]);  // the row ends before this part
                }
            }
            __syncwarp();
            buf.next(buffers);
            ++issued;
            return true;
        });
        if (!ok) {
            gave_up(S);
            // copies in flight land before the CTA may exit
            for (uint32_t j = issued > buffers ? issued - buffers : 0; j < issued; ++j)
                wait(&S.full[j % buffers], j / buffers & 1u, kSettleNs);
        }
    } else if (warp >= kCloser) {
        QueuePlace place{{0, 0}, 0};
        RingPlace buf{0, 0}, map{0, 0}, put{0, 0}, taken{0, 0};
        const float scale = kGrad ? scale_of_grad(D.grad_scale, D.grad_scale_dev) : 1.f;
        const int k = D.top_n;
        uint32_t writer = uint32_t(warp - kCloser);  // whose turn it is to write a row's outputs, modulo `parts`
        int before = warp - kCloser;                 // rows that the other closers take before this one's next
        // A row and its list, as they are read ahead.
        struct Fetched {
            RowItem item;
            int id[kHeld];
            float l[kHeld];
            float rest;  // the teacher's logprob outside the list
        };
        // A row whose list has been put, until it is closed. (Its tokens in this part are few of the list: they are moved
        // together first, so that the closers' work, which all CTAs of a cluster have, is one token in each lane.)
        struct Open {
            RowItem item;
            uint32_t buffer;
            int count;
            float rest;
        };
        Entry* list = S.list[warp - kCloser];
        // The next row that counts. 1: done; 0: no more rows; -1: a wait gave up.
        auto fetch = [&](Fetched& f) {
            for (;;) {
                if (!queue_next(S.queue, place, P.wait_ns, f.item)) return -1;
                if (f.item.row < 0) return 0;
                if (f.item.live && before-- == 0) break;
                if (!f.item.live && rank == 0 && lane == 0 && warp == kCloser) write_row(P, f.item.row, 0.f, 0.f, SAMPLER_ROW_OK, 0.0);
            }
            before = kClosers - 1;
            const int64_t r = f.item.row;
            f.rest = D.teacher_rest ? __ldg(D.teacher_rest + r) : -pos_inf();
#pragma unroll
            for (int e = 0; e < kHeld; ++e) {
                const int j = lane + 32 * e;
                f.id[e] = j < k ? __ldg(D.teacher_ids + r * k + j) : -1;
                f.l[e] = j < k ? __ldg(D.teacher_logprobs + r * k + j) : -pos_inf();
            }
            return 1;
        };
        // Marks a row's tokens, and puts its share of the sums; false where a wait gave up.
        auto open = [&](const Fetched& f, Open& o) {
            o.item = f.item;
            o.rest = f.rest;
            const int n = min(first_vec + P.part_vecs, o.item.count) - first_vec;  // vectors here
            const int head = o.item.head - first_vec * kPer;
            const RowJob h = job_of(o.item);
            uint32_t flags = o.rest < pos_inf() ? 0 : kBadList;
            o.count = 0;
#pragma unroll
            for (int e = 0; e < kHeld; ++e) {
                if (32 * e >= k) break;
                int id = f.id[e];
                if (id < -1 || int64_t(id) >= a.vocab || (id != -1 && !(f.l[e] < pos_inf()))) {
                    flags |= kBadList;
                    id = -1;
                }
                const int at = id + head;
                const bool here = id >= 0 && at >= 0 && at < n * kPer;
                const uint32_t lanes = __ballot_sync(0xffffffffu, here);
                if (here) {
                    Entry& t = list[o.count + __popc(lanes & ((1u << lane) - 1u))];
                    t.at = at;
                    t.l = f.l[e];
                }
                o.count += __popc(lanes);
            }
            __syncwarp();
            if (!wait(&S.unmarked[map.at], map.phase ^ 1u, P.wait_ns)) return false;
            unsigned char* bits = maps + map.at * map_bytes<kWarps>(P.part_vecs);
            for (int i = lane; i < o.count; i += 32) {
                const int at = list[i].at, byte = map_place<kWarps>(at / kPer);
                const uint32_t bit = 1u << (8 * (byte & 3) + at % kPer);
                if (atomicOr(reinterpret_cast<uint32_t*>(bits) + byte / 4, bit) & bit) flags |= kBadList;  // twice
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&S.full[buf.at]);
                mbar_arrive_expect_tx(&S.join[put.at], parts * uint32_t(kWarps * 16 + sizeof(ListSums)));
            }
            __syncwarp();
            if (!wait(&S.full[buf.at], buf.phase, P.wait_ns)) return false;
            o.buffer = buf.at;
            const T* in = reinterpret_cast<const T*>(smem + buf.at * buffer_bytes);
            float ref = -kFloatMax, s = 0.f;
            Pair sa{0.f, 0.f}, sq{0.f, 0.f};
            if (o.count) {
                for (int i = lane; i < o.count; i += 32) {
                    const float y = load_logit(in + list[i].at);
                    list[i].x = y;
                    if (!(y < pos_inf())) flags |= kBadLogit;
                    ref = fmaxf(ref, y);
                }
                ref = max_warp(ref);
                for (int i = lane; i < o.count; i += 32) {
                    const Entry t = list[i];
                    const float q = expf(t.l), d = t.x - ref;
                    list[i].q = q;
                    s += exp2f(fmaxf(fmaf(d, h.c_hi, d * h.c_lo), kLowest));
                    if (q > 0.f) {
                        sq = pair_add(sq, Pair{q, 0.f});
                        Pair z{pos_inf(), 0.f};
                        if (t.x > -pos_inf()) {
                            const Pair y = scaled(h, t.x, ref);
                            z = two_sum(t.l, -y.hi);
                            z.lo -= y.lo;
                        }
                        sa = pair_add(sa, pair_times(q, z));
                    }
                }
#pragma unroll
                for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
                pair_warp(sa);
                pair_warp(sq);
            }
            flags = __reduce_or_sync(0xffffffffu, flags);
            if (uint32_t(lane) < parts) {
                const uint32_t to = dsmem_map(smem_addr(lists + put.at * parts + rank), lane),
                               bar = dsmem_map(smem_addr(&S.join[put.at]), lane);
                put_sums(to, bar, ref, s, sa.hi, sa.lo);
                put_sums(to + 16, bar, sq.hi, sq.lo, __uint_as_float(flags), 0.f);
            }
            __syncwarp();
            if (!kGrad && lane == 0) mbar_arrive(&S.empty[buf.at]);
            return true;
        };
        // Closes a row; false where a wait gave up.
        auto close = [&](const Open& o) {
            if (!wait(&S.join[taken.at], taken.phase, P.wait_ns)) return false;
            const RowJob h = job_of(o.item);
            const Scale by{h.c_hi, h.c_lo};
            // outside the list, and inside
            const float4* in = sums + taken.at * parts * kWarps;
            Stats out = stats_empty();
            for (uint32_t i = lane; i < parts * kWarps; i += 32) out.ref = fmaxf(out.ref, in[i].x);
            out.ref = max_warp(out.ref);
            for (uint32_t i = lane; i < parts * kWarps; i += 32) {
                Stats p{in[i].x, in[i].y, 0.f};
                stats_move(p, out.ref, by);
                out.s += p.s;
            }
            ListSums mine{-kFloatMax, 0.f, {0.f, 0.f}, {0.f, 0.f}, 0, 0};
            if (uint32_t(lane) < parts) mine = lists[taken.at * parts + lane];
            Stats inside{mine.ref, mine.s, 0.f};
            stats_move(inside, max_warp(mine.ref), by);
            float q_list = mine.q.hi;
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) {
                out.s += __shfl_xor_sync(0xffffffffu, out.s, i);
                inside.s += __shfl_xor_sync(0xffffffffu, inside.s, i);
                q_list += __shfl_xor_sync(0xffffffffu, q_list, i);
            }
            const uint32_t flags = __reduce_or_sync(0xffffffffu, mine.flags);

            const float most = fmaxf(out.ref, inside.ref);
            auto lift = [&](float ref) {
                const float d = ref - most;
                return exp2f(fmaxf(fmaf(d, h.c_hi, d * h.c_lo), kLowest));
            };
            const float f_out = lift(out.ref);
            const float s = out.s * f_out + inside.s * lift(inside.ref);
            const int status = h.bad_param || (flags & kBadList)        ? SAMPLER_ROW_BAD_PARAM
                               : isnan(out.s) || (flags & kBadLogit) ? SAMPLER_ROW_NONFINITE
                               : s == 0.f                            ? SAMPLER_ROW_ALL_NEG_INF
                                                                     : SAMPLER_ROW_OK;
            const float inv_s = __fdiv_rn(1.f, s), p_out = out.s * f_out * inv_s;
            const float q_out = o.rest > -pos_inf() ? expf(o.rest) : 0.f;
            const float coef = a.tokens ? D.token_coef : 0.f;
            const float w = q_list + q_out + coef;
            const float g = o.item.weight * scale * h.inv_t;
            const bool fine = status == SAMPLER_ROW_OK;
            if (kGrad) {
                // the list's own gradients, in their logits' place
                T* to = reinterpret_cast<T*>(smem + o.buffer * buffer_bytes);
                const int head = o.item.head - first_vec * kPer;
                for (int i = lane; i < o.count; i += 32) {
                    const Entry t = list[i];
                    float y = fmaf(w, lift(t.x) * inv_s, -t.q);
                    if (a.tokens && t.at == o.item.token + head) y -= coef;
                    store_grad(to + t.at, fine ? y * g : quiet_nan());
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (lane == 0) {
                    Factor& f = S.factor[taken.at];
                    f.ref = fine ? out.ref : 0.f;
                    f.c = fine ? h.c : 0.f;
                    f.k = !fine ? quiet_nan() : out.s > 0.f ? __fdiv_rn(fmaf(w, p_out, -q_out), out.s) * g : 0.f;
                    f.at_token = -coef * g;
                    f.token = fine && coef != 0.f ? o.item.token : kNoToken;
                }
                __syncwarp();
            }
            if (lane == 0) {
                mbar_arrive(&S.closed[taken.at]);
                if (kGrad) mbar_arrive(&S.empty[o.buffer]);
            }
            // a row's outputs are the work of one of the cluster's closers in turn
            if (writer % parts == rank) {
                Pair ln_s = log_of(s);
                ln_s.lo = fmaf(kExp2Short, p_out, ln_s.lo);
                const Stats all{most, s, 0.f};
                // each part's tokens, from its reference to the row's: q_j (l_j - ln p_j) = q_j (l_j - (x_j - ref) / T)
                // + q_j (ln s + (most - ref) / T)
                Pair kl{0.f, 0.f};
                if (mine.q.hi > 0.f) {
                    const Pair y = scaled(h, most, mine.ref), z = pair_add(ln_s, y);
                    // (a part without a finite logit has its reference at the lowest float, and y may be infinite)
                    kl = mine.a.hi < pos_inf() && z.hi < pos_inf()
                             ? pair_add(mine.a, pair_add(pair_times(mine.q.hi, z), Pair{mine.q.lo * z.hi, 0.f}))
                             : Pair{pos_inf(), 0.f};
                }
                pair_warp(kl);
                if (q_out > 0.f) {
                    // ln p_out = (ref_out - most) / T - ln s + ln s_out
                    Pair z{pos_inf(), 0.f};
                    if (out.s > 0.f) {
                        Pair l = log_of(out.s);
                        l.lo += kExp2Short;
                        l = pair_add(l, logprob_of(h, all, out.ref, ln_s));
                        z = two_sum(o.rest, -l.hi);
                        z.lo -= l.lo;
                    }
                    kl = pair_add(kl, pair_times(q_out, z));
                }
                const Pair lp = logprob_of(h, all, o.item.x_t, ln_s);
                if (lane == 0) {
                    const double divergence = isinf(kl.hi) ? double(kl.hi) : double(kl.hi) + double(kl.lo);
                    double each = divergence;
                    if (coef != 0.f) each -= double(coef) * (double(lp.hi) + double(lp.lo));
                    write_row(P, o.item.row, fine ? float(divergence) : quiet_nan(), fine ? lp.hi : quiet_nan(), status,
                              fine ? double(o.item.weight) * each : double(quiet_nan()));
                }
            }
            writer += kClosers;
            return true;
        };
        auto skip = [&](int rows) {
            for (; rows > 0; --rows) {
                buf.next(buffers);
                map.next(kMaps);
                put.next(kSums);
                taken.next(kSums);
            }
        };
        skip(warp - kCloser);
        Fetched ahead;
        int more = fetch(ahead);  // whether `ahead` is a row
        bool ok = more >= 0;
        while (ok && more == 1) {
            Open now;
            ok = open(ahead, now);
            if (!ok) break;
            more = fetch(ahead);  // (on its way while the row is closed)
            ok = more >= 0 && close(now);
            skip(kClosers);
        }
        if (!ok) gave_up(S);
    } else {
        QueuePlace place{{0, 0}, 0};
        RingPlace buf1{0, 0}, buf2{0, 0}, map1{0, 0}, map2{0, 0}, put{0, 0}, closed{0, 0};
        const int vocab = int(a.vocab);
        // The next row that counts, and its pass 1. 1: done; 0: no more rows; -1: a wait gave up.
        auto pass1 = [&](RowItem& item) {
            for (;;) {
                if (!queue_next(S.queue, place, P.wait_ns, item)) return -1;
                if (item.row < 0) return 0;
                if (item.live) break;
                if (kGrad) {
                    T* g = static_cast<T*>(a.out_grad) + int64_t(item.row) * a.grad_stride;
                    const RowSpan span = row_span(g, a.vocab);
                    // (the gradient's own vectors, dealt to the cluster's CTAs)
                    for (int i = int(rank) * kConsumers + tid; i < span.count; i += int(parts) * kConsumers)
                        put_vector<T>(g, vocab, span.head, i, true, make_uint4(0u, 0u, 0u, 0u));
                }
            }
            const RowSpan span{item.head, item.count};
            const int n = min(first_vec + P.part_vecs, span.count) - first_vec;
            const int end = span.head + vocab;
            const Two c_hi = two(item.c_hi, item.c_hi), c_lo = two(item.c_lo, item.c_lo);
            const Scale by{item.c_hi, item.c_lo};
            if (!wait(&S.full[buf1.at], buf1.phase, P.wait_ns)) return -1;
            const uint4* in = reinterpret_cast<const uint4*>(smem + buf1.at * buffer_bytes);
            unsigned char* bits = maps + map1.at * map_bytes<kWarps>(P.part_vecs);
            Stats st = stats_empty();
            bool bad = false;
            for (int i0 = 0; i0 < n; i0 += kStep) {
                uint4 v[kVecs];
                uint32_t* marks = reinterpret_cast<uint32_t*>(bits + i0) + tid;  // (a byte for each of the four vectors)
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int i = i0 + k * kConsumers + tid;
                    v[k] = nothing<T>();
                    if (i < n) v[k] = in[i];
                }
                if (ragged(span, end, first_vec + i0, kPer, kStep))
#pragma unroll
                    for (int k = 0; k < kVecs; ++k) {
                        const int at = (first_vec + i0 + k * kConsumers + tid) * kPer;
                        if (at < span.head || at + kPer > end) Elems<T>::mask(v[k], span.head - at, end - at);
                    }
                if (const uint32_t b = *marks) {
#pragma unroll
                    for (int k = 0; k < kVecs; ++k)
                        if (b >> 8 * k & 0xffu) blend<T>(v[k], nothing<T>(), b >> 8 * k & 0xffu);
                    if (!kGrad) *marks = 0;
                }
                fold<T, false, kVecs>(st, bad, v, c_hi, c_lo, by);
            }
            if (bad) st.s = quiet_nan();
            stats_warp<false>(st, by);
            // (A buffer of sums is written again four rows later: by then every closer of the cluster is done with it, as
            // each puts a row's list sums after closing the row two before, and a warp puts a row's after that two before
            // is closed.)
            if (uint32_t(lane) < parts)
                put_sums(dsmem_map(smem_addr(sums + (put.at * parts + rank) * kWarps + warp), lane),
                         dsmem_map(smem_addr(&S.join[put.at]), lane), st.ref, st.s, 0.f, 0.f);
            __syncwarp();
            if (!kGrad && lane == 0) {
                mbar_arrive(&S.empty[buf1.at]);
                mbar_arrive(&S.unmarked[map1.at]);
            }
            buf1.next(buffers);
            map1.next(kMaps);
            put.next(kSums);
            return 1;
        };
        // Its pass 2, once it is closed; false where the wait gave up.
        auto pass2 = [&](const RowItem& item) {
            if (!wait(&S.closed[closed.at], closed.phase, P.wait_ns)) return false;
            if (kGrad) {
                const Factor f = S.factor[closed.at];
                const Factors fs{two(-f.ref, -f.ref), two(f.c, f.c), two(f.k, f.k), 0};
                const T* x = static_cast<const T*>(a.logits) + int64_t(item.row) * a.row_stride;
                T* g = static_cast<T*>(a.out_grad) + int64_t(item.row) * a.grad_stride;
                const RowSpan span{item.head, item.count};
                const int n = min(first_vec + P.part_vecs, span.count) - first_vec;
                const bool whole = ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
                const int token_vec = f.token == kNoToken ? -1 : (f.token + span.head) / kPer - first_vec;
                const uint4* in = reinterpret_cast<const uint4*>(smem + buf2.at * buffer_bytes);
                unsigned char* bits = maps + map2.at * map_bytes<kWarps>(P.part_vecs);
                const int end = span.head + vocab;
                for (int i0 = 0; i0 < n; i0 += kStep) {
                    uint32_t* marks = reinterpret_cast<uint32_t*>(bits + i0) + tid;
                    const uint32_t marked = *marks;
                    if (whole && !ragged(span, end, first_vec + i0, kPer, kStep) && !(token_vec >= i0 && token_vec < i0 + kStep)) {
                        uint4* to = reinterpret_cast<uint4*>(g - span.head) + first_vec + i0 + tid;
                        uint4 v[kVecs], y[kVecs];
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) v[k] = in[min(i0 + k * kConsumers + tid, n - 1)];
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) y[k] = gradient<T, false>(v[k], fs);
                        if (marked)
#pragma unroll
                            for (int k = 0; k < kVecs; ++k)
                                if (marked >> 8 * k & 0xffu) blend<T>(y[k], v[k], marked >> 8 * k & 0xffu);
#pragma unroll
                        for (int k = 0; k < kVecs; ++k)
                            if (i0 + k * kConsumers + tid < n) __stcs(to + k * kConsumers, y[k]);
                    } else {
#pragma unroll 1
                        for (int k = 0; k < kVecs; ++k) {
                            const int i = i0 + k * kConsumers + tid;
                            if (i >= n) break;
                            const uint4 v = in[i];
                            uint4 y = gradient_token<T, false>(v, fs, i == token_vec ? f.token + span.head - (first_vec + i) * kPer : -1,
                                                               f.at_token);
                            blend<T>(y, v, marked >> 8 * k & 0xffu);
                            put_vector<T>(g, vocab, span.head, first_vec + i, whole, y);
                        }
                    }
                    if (marked) *marks = 0;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&S.empty[buf2.at]);
                    mbar_arrive(&S.unmarked[map2.at]);
                }
                buf2.next(buffers);
                map2.next(kMaps);
            }
            closed.next(kSums);
            return true;
        };
        RowItem now, next;
        int more = pass1(now);
        while (more == 1) {
            more = pass1(next);
            if (more < 0 || !pass2(now)) {
                more = -1;
                break;
            }
            now = next;
        }
        if (more < 0) gave_up(S);
    }
    __syncwarp();
    cluster_sync();
    if (S.failed) abandon<T, kGrad, kThreads>(P, q, n_clusters, parts, rank);
    if (rank == 0 && last_block(P.ws.ticket, n_clusters, &S.flag)) {
        const double loss = sum_terms<kThreads>(P.ws.terms, a.n_rows, S.scratch);
        if (tid == 0) D.out_loss[0] = float(loss);
    }
}

}  // namespace distill

namespace distill {

// Clusters of `parts` CTAs that the device holds at once (asked once for each kernel of a handle); 0: an error.
template <int kWarps, typename Kernel>
int resident(Kernel kernel, cudaLaunchConfig_t cfg, int parts, int& known)
{
    if (known > 0) return known;
    const void* k = reinterpret_cast<const void*>(kernel);
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<kWarps>::kSmem) != cudaSuccess ||
        (parts > 8 && cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess))
        return 0;
    cudaLaunchAttribute attr = *cfg.attrs;
    attr.val.clusterDim = {unsigned(parts), 1u, 1u};
    cfg.attrs = &attr;
    cfg.gridDim = dim3(unsigned(parts));
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) return 0;
    return known = n;
}

// CTAs of a cluster: those for which the turns that the rows take on the clusters the device holds, each as long as a part
// takes, are the shortest; of equal ones the most. A turn is about 2.2 us for a part of one step of the consumers'
// (32 KB), 3.5 for two and 4.1 for a little more, and 7.5 where there is no room for three buffers (one is filled while two
// rows are in hand). Parts have 4 KB at least. Measured with gradient, us by parts:
//   1200 x 128000 bf16   3 (two buffers): 178   4: 127   5: 143   6: 169   8: 181
//   1200 x 151936 bf16   4 (two buffers): 216   5: 152   6: 170   8: 245
//   1200 x 65000 bf16    2: 75   3: 98   4: 95
//   800 x 100000 fp32    5 (two buffers): 157   6: 118   7: 141   8: 132
//   800 x 151936 fp32    8 (two buffers): 266   10: 168   16: 262
// Without gradient a row leaves its buffer after its first pass: two are enough, and a turn is about 1.6 us for one step of
// the consumers', 2.1 for two and 2.6 for three. Of 77 shapes (64 to 4096 rows of 20000 to 262144, both types, 1 to 16 parts,
// a cold L2) what that chooses is 0.2 % off the best on average and 6 at most; the turns with gradient were up to 65 % off.
// us by parts:
//   4096 x 40000 bf16    1 (two buffers): 90    2: 133   3: 166   4: 199
//   4096 x 200000 bf16   5 (two buffers): 377   6: 442   7: 569   8: 549
//   800 x 200000 fp32    9 (two buffers): 123   10: 133  11: 205  16: 203
//   1200 x 128000 fp32   6 (two buffers): 121   7: 168   8: 143   9: 147
//   64 x 151936 fp32     7: 25   9: 25   10: 23   16: 29
template <int kWarps, typename Kernel>
int parts_of(Kernel kernel, const cudaLaunchConfig_t& cfg, int64_t vecs, int64_t rows, bool grad, int (&known)[kMaxParts])
{
    using S = Shape<kWarps>;
    int best = 0;
    double least = 0.;
    for (int parts = 1; parts <= kMaxParts; ++parts) {
        const int part_vecs = int((vecs + parts - 1) / parts);
        if (smem_of<kWarps>(part_vecs, 2, parts) > S::kSmem || (parts > 1 && part_vecs < 256)) continue;
        const int clusters = resident<kWarps>(kernel, cfg, parts, known[parts - 1]);
        if (clusters < 1) continue;
        const int steps = part_vecs <= S::kStep ? 1 : part_vecs <= 2 * S::kStep ? 2 : 3;
        const double turn = !grad                                             ? steps == 1 ? 1.6 : steps == 2 ? 2.1 : 2.6
                            : smem_of<kWarps>(part_vecs, 3, parts) > S::kSmem ? 7.5
                            : steps == 1                                      ? 2.2
                            : steps == 2                                      ? 3.5
                                                                              : 4.1;
        const double time = turn * double((rows + clusters - 1) / clusters);
        if (best == 0 || time <= least) {
            best = parts;
            least = time;
        }
    }
    return best;
}

template <int kWarps>
int launch(DistillParams& p, int sms, DistillOccupancy* occ, cudaStream_t stream)
{
    using S = Shape<kWarps>;
    const bool bf16 = p.rows.dtype == SAMPLER_DTYPE_BF16, grad = p.rows.out_grad != nullptr;
    const int per = bf16 ? 8 : 4;
    const int64_t vecs = (p.rows.vocab + 2 * per - 2) / per;  // the most that a row touches, wherever it starts
    const auto kernel = bf16 ? grad ? distill_kernel<uint16_t, true, kWarps> : distill_kernel<uint16_t, false, kWarps>
                             : grad ? distill_kernel<float, true, kWarps> : distill_kernel<float, false, kWarps>;
    int(&known)[kMaxParts] = occ->clusters[kWarps == kShortWarps][bf16][grad];
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = size_t(S::kSmem);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int parts = 1;
    if (kWarps == kShortWarps) {
        // short rows: one, or as many as give each SM a part where rows are few
        while (parts < kMaxParts && p.rows.n_rows * parts < sms && vecs / (2 * parts) >= 256) parts *= 2;
    } else {
        parts = parts_of<kWarps>(kernel, cfg, vecs, p.rows.n_rows, grad, known);
    }
    if (parts < 1) return SAMPLER_ERR_CUDA;
    const int clusters = resident<kWarps>(kernel, cfg, parts, known[parts - 1]);
    if (clusters < 1) return SAMPLER_ERR_CUDA;
    p.part_vecs = int((vecs + parts - 1) / parts);
    p.buffers = 2;
    if (smem_of<kWarps>(p.part_vecs, p.buffers, parts) > S::kSmem) return SAMPLER_ERR_TOO_LARGE;  // (no vocabulary of a handle's)
    while (p.buffers < kMaxBuffers && smem_of<kWarps>(p.part_vecs, p.buffers + 1, parts) <= S::kSmem) ++p.buffers;
    attr.val.clusterDim = {unsigned(parts), 1u, 1u};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(p.rows.n_rows, clusters) * parts));
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace distill

int distill_launch(const DistillParams& params, int sms, DistillOccupancy* occ, cudaStream_t stream)
{
    using namespace distill;
    DistillParams p = params;
    // Rows of which the shared memory of a small CTA has room for two (32 KB at most) go to CTAs of four consumer warps, of
    // which an SM holds three: a row's fixed work, the chain from
    // its sums to its factors, is then under way for three times as many rows. With gradient, bf16, us by four and by sixteen
    // warps: 4096 x 1000 52 and 84, 4096 x 8000 74 and 94, 4096 x 16000 99 and 104, 4096 x 24000 138 and 131; fp32:
    // 4 x 1024 8.7 and 10.2, 4096 x 8000 80 and 90.
    const int per = p.rows.dtype == SAMPLER_DTYPE_BF16 ? 8 : 4;
    const int64_t vecs = (p.rows.vocab + 2 * per - 2) / per;
    const bool small = vecs <= 2049 && smem_of<kShortWarps>(int(vecs), 2, 1) <= Shape<kShortWarps>::kSmem;
    return small ? launch<kShortWarps>(p, sms, occ, stream) : launch<kLongWarps>(p, sms, occ, stream);
}

}  // namespace dst
