// row_loss_kernel.cu -- scoring and the losses over logits rows: logprob,
// entropy, the clipped policy loss, the preference loss, and the logits'
// gradients.
//
// A row's gradient needs the row's sums, so a row is wanted twice, and is read
// from memory once: a cluster of C CTAs takes a row, each CTA a part of it in
// shared memory, where the second pass finds it. Warp roles of a CTA:
//   producer   goes ahead over the cluster's rows: it reads their parameters and
//              brings their parts in with bulk copies, through a ring of 16 KB chunks;
//   consumers  (eight) pass 1, four vectors of each chunk in every thread: the
//              running reference and the sums of exponentials, which each warp puts
//              into every CTA of the cluster (distributed shared memory);
//   closer     combines the cluster's sums, works out the gradient's factors and
//              writes the row's outputs;
//   consumers  pass 2, with a gradient: the same vectors again from the ring,
//              16-byte stores, and each chunk's slot goes back to the producer.
// Before pass 2 of a row the consumers take pass 1 of the next as far as the ring
// holds it, so that the join and the closer's work (about 2 us a row, most of it
// latency) run under it.
// Measured, policy loss with its gradient in bf16: 2048 x 128000 in 176 us, 5.9 TB/s
// of logits and gradients (88 % of the copy rate); 2048 x 151936 in 210 us; one row
// of 151936 in 8.6 us, which is launch, one part's way through memory and the join.
// At 1024 x 128000 the DRAM is 62 % busy from cold caches and 58 % of the issue
// slots are taken: the arithmetic of the two passes and the memory's latency share
// the time. (fp32 rows, with half the elements to a byte, take 322 us at 2048 x
// 128000, 6.5 TB/s, 96 % of the copy rate.)
// The rows that count are dealt to the clusters evenly whatever rows are left
// out: each producer counts them, 32 weights at a time.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "row_loss.cuh"
#include "row_queue.cuh"
#include "row_vectors.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace rows {

constexpr int kWarps = 8;                        // consumers: few, with much in hand (see below)
constexpr int kConsumers = kWarps * 32;
constexpr int kProducer = kWarps, kCloser = kWarps + 1;
constexpr int kThreads = kConsumers + 64;
constexpr int kVecs = 4;                         // 16-byte vectors of a chunk in each consumer
constexpr int kChunkVecs = kConsumers * kVecs;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kMaxSlots = 6;
constexpr int kPartChunks = 6;                   // of a row in a CTA, where the row allows it
constexpr int kMaxParts = 16;                    // CTAs of a cluster
constexpr int kBatch = 8;                        // rows whose parameters are fetched together
constexpr int kFirstBatch = 2;                   // the first time, when all wait for them
constexpr int kSums = 4;                         // rows whose sums are in shared memory
constexpr int kSmemMax = 113 * 1024;             // of a CTA: two on an SM
constexpr uint64_t kSettleNs = 100000;           // in which what is on its way to shared memory lands

// The ring (slots * kChunkBytes), the sums [kSums][parts * kWarps] and this.
struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t job_full[2], job_empty[2];
    uint64_t join[kSums], closed[kSums];
    RowJob jobs[2][kBatch];
    RowRecord rec[kSums];
    double scratch[kThreads / 32];
    uint32_t flag, failed;  // failed: a wait of this cluster gave up
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
};

constexpr int kPut = 0x7fffffff;  // in the place of the next vector: the row's sums have been put

using Place = RingPlace;

// The two kernels after the rows' are launched as programmatic dependents: their
// blocks come up while the grid before ends, and wait for it here.
__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependent_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A wait of this warp gave up: every CTA of the cluster is told, and abandons the
// cluster's rows once all have come to their end.
__device__ __noinline__ void gave_up(Shared& S)
{
    const uint32_t cta = threadIdx.x & 31;
    if (cta < cluster_nctarank()) dsmem_st_u32(dsmem_map(smem_addr(&S.failed), cta), 1u);
}

// ---------------------------------------------------------------- the kernel
// A wait of this cluster gave up. Which of its rows were done with is not known,
// so all of them are written again, by all CTAs after the last of them has come to
// its end: those that count as TIMEOUT with NaN, the others as ever. Otherwise a
// loss, or the pairs' kernel after this one, would go on with what an earlier call
// has left in the workspace.
template <typename T, bool kGrad>
__device__ __noinline__ void abandon(const LossParams& P, uint32_t q, uint32_t n_clusters, uint32_t parts, uint32_t rank)
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
        if (rank == 0 && threadIdx.x == 0) row_give_up(P, r, counts);
        if (kGrad) {
            T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
            for (int64_t v = rank * kThreads + threadIdx.x; v < a.vocab; v += parts * kThreads)
                store_grad(g + v, counts ? quiet_nan() : 0.f);
        }
    }
}

// What a row needs besides its logits and its weight, one row in each lane.
__device__ __forceinline__ void job_load(RowJob& j, float& temperature, const LossParams& P, int64_t r)
{
    const sampler_rows_t& a = P.rows;
    j.token = a.tokens[r];
    j.weight = a.weight ? a.weight[r] : 1.f;
    temperature = a.temperature ? a.temperature[r] : 1.f;
    j.in0 = j.in1 = j.in2 = 0.f;
    if (P.mode == kModeScoreGrad) {
        j.in0 = P.grad_logprob[r];
        if (P.grad_entropy) j.in1 = P.grad_entropy[r];
    } else if (P.mode == kModePolicy) {
        j.in0 = P.policy.advantage[r];
        j.in1 = P.policy.old_logprob[r];
        if (P.policy.ref_logprob) j.in2 = P.policy.ref_logprob[r];
    }
}

// Its token's logit. It is read before the row is taken up, and so before any
// CTA can write the row's gradient in the logits' place.
template <typename T>
__device__ __forceinline__ void job_token(RowJob& j, const sampler_rows_t& a, int64_t r, bool live)
{
    j.x_t = 0.f;
    if (live && j.token >= 0 && int64_t(j.token) < a.vocab)
        j.x_t = load_logit(static_cast<const T*>(a.logits) + r * a.row_stride + j.token);
}

// A CTA's part of row r, worked out once by the producer.
template <typename T>
__device__ __forceinline__ RowPart row_part(const sampler_rows_t& a, int64_t r, uint32_t rank, const RowPlan& plan)
{
    const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
    const RowSpan span = row_span(x, a.vocab);
    RowPart p;
    p.head = span.head;
    p.count = span.count;
    p.first = int(rank) * plan.part_vecs;
    p.last = max(p.first, min(p.first + plan.part_vecs, span.count));
    p.inner_first = span.head ? 1 : 0;
    p.inner_last = min(p.last, int((span.head + a.vocab) / (16 / int(sizeof(T))))) - kChunkVecs;
    T* g = a.out_grad ? static_cast<T*>(a.out_grad) + r * a.grad_stride : nullptr;
    p.whole = ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
    p.grad = g;
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

    if (P.mode == kModePairs) dependent_launch();
    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
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
        Place slot{0, 0}, batch{0, 0};
        uint32_t issued = 0;
        bool ok = P.wait_ns != 0, end = false;  // 0: nothing begins, and every other wait of the cluster gives up
        auto copy_in = [&](int64_t row) {
            const RowPart part = row_part<T>(a, row, rank, plan);
            const unsigned char* from = reinterpret_cast<const unsigned char*>(static_cast<const T*>(a.logits) +
                                                                               row * a.row_stride - part.head);
            for (int v = part.first; ok && v < part.last; v += kChunkVecs) {
                ok = wait(&S.empty[slot.at], slot.phase ^ 1u, P.wait_ns);
                if (!ok) break;
                const uint32_t bytes = uint32_t(min(kChunkVecs, part.last - v)) * 16u;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&S.full[slot.at], bytes);
                    bulk_copy_g2s(ring + slot.at * kChunkBytes, from + size_t(v) * 16, bytes, &S.full[slot.at]);
                }
                __syncwarp();
                slot.next(slots);
                ++issued;
            }
        };
        // The next `most` rows at most, the k-th in lane k (row -1: the end); which of them count. Their number.
        auto deal = [&](int most, int64_t& mine, uint32_t& live) {
            int count = 0;
            mine = -1;
            live = 0;
            while (count < most && !end) {
                bool counts;
                const int64_t r = dealer_next(d, a, q, n_clusters, counts);
                if (lane == count) mine = r;
                if (r < 0)
                    end = true;
                else if (counts)
                    live |= 1u << count;
                ++count;
            }
            return count;
        };
        auto publish = [&](RowJob& job, float temperature, int count, int64_t mine, uint32_t live) {
            ok = ok && wait(&S.job_empty[batch.at], batch.phase ^ 1u, P.wait_ns);
            if (!ok) return;
            if (lane < count) {
                job.row = int32_t(mine);
                job.live = live >> lane & 1u;
                job.last = lane == count - 1;
                if (mine >= 0) {
                    row_scale(job, a, temperature);
                    job.part = row_part<T>(a, mine, rank, plan);
                }
                S.jobs[batch.at][lane] = job;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.job_full[batch.at]);
            batch.next(2);
        };
        int64_t mine;
        uint32_t live;
        int count = deal(kFirstBatch, mine, live);
        {
            RowJob job;
            float temperature;
            if (mine >= 0) job_load(job, temperature, P, mine);
            if (live & 1u) copy_in(__shfl_sync(0xffffffffu, mine, 0));
            if (mine >= 0) job_token<T>(job, a, mine, live >> lane & 1u);
            publish(job, temperature, count, mine, live);
        }
        // a batch's copies, and on their way the parameters of the next
        for (int k0 = 1; ok; k0 = 0) {
            int64_t mine_next;
            uint32_t live_next;
            const int count_next = deal(kBatch, mine_next, live_next);
            RowJob job;
            float temperature;
            if (mine_next >= 0) job_load(job, temperature, P, mine_next);
            for (int k = k0; ok && k < count; ++k) {
                if (live >> k & 1u) copy_in(__shfl_sync(0xffffffffu, mine, k));
                if (k == k0 && mine_next >= 0) job_token<T>(job, a, mine_next, live_next >> lane & 1u);
            }
            if (k0 >= count && mine_next >= 0) job_token<T>(job, a, mine_next, live_next >> lane & 1u);
            if (count_next == 0) break;
            publish(job, temperature, count_next, mine_next, live_next);
            mine = mine_next;
            live = live_next;
            count = count_next;
        }
        if (!ok) {
            gave_up(S);
            // copies in flight land before the CTA may exit
            for (uint32_t j = issued > slots ? issued - slots : 0; j < issued; ++j)
                wait(&S.full[j % slots], j / slots & 1u, kWaitNs);
        }
    } else if (warp == kCloser) {
        const float grad_scale =
            kGrad && P.mode == kModePolicy ? scale_of_grad(P.policy.grad_scale, P.policy.grad_scale_dev) : 1.f;
        Place batch{0, 0}, sp{0, 0};
        for (int k = 0;; ++k) {
            if (k == 0 && !wait(&S.job_full[batch.at], batch.phase, P.wait_ns)) {
                gave_up(S);
                break;
            }
            const RowJob job = S.jobs[batch.at][k];
            if (job.row < 0) break;
            Stats st = stats_empty();
            if (job.live) {
                if (lane == 0) mbar_arrive_expect_tx(&S.join[sp.at], kWarps * parts * 16u);
                __syncwarp();
                if (!wait(&S.join[sp.at], sp.phase, P.wait_ns)) {
                    gave_up(S);
                    break;
                }
                const float4* in = sums + sp.at * parts * kWarps;
                float ref = -kFloatMax;
                for (uint32_t i = lane; i < parts * kWarps; i += 32) ref = fmaxf(ref, in[i].x);
                st.ref = max_warp(ref);
                for (uint32_t i = lane; i < parts * kWarps; i += 32) {
                    const float4 p = in[i];
                    Stats o{p.x, p.y, p.z};
                    stats_move(o, st.ref, job.c);
                    st.s += o.s;
                    st.t += o.t;
                }
                sum_warp<kEntropy>(st);
            }
            RowRecord rec;
            RowOut out;
            row_close(P, job, st, grad_scale, rec, out);
            if (job.live) {
                if (lane == 0) {
                    if (kGrad) S.rec[sp.at] = rec;
                    mbar_arrive(&S.closed[sp.at]);
                }
                sp.next(kSums);
            }
            if (rank == 0 && lane == 0) row_write(P, job.row, rec, out);
            __syncwarp();
            if (job.last) {
                if (lane == 0) mbar_arrive(&S.job_empty[batch.at]);
                batch.next(2);
                k = -1;
            }
        }
    } else {
        constexpr int kPer = Elems<T>::kPer;
        const int vocab = int(a.vocab);
        Place batch{0, 0}, slot1{0, 0}, slot2{0, 0}, sp{0, 0}, cp{0, 0};
        uint32_t behind = 0;  // rows put into the join whose closing has not been waited for
        int at = 0;           // of the batch
        bool ok = true;
        // The next job; its row is -1 at the end.
        auto next_job = [&]() -> const RowJob* {
            if (at < 0) {
                batch.next(2);
                at = 0;
            }
            if (at == 0 && !wait(&S.job_full[batch.at], batch.phase, P.wait_ns)) {
                gave_up(S);
                ok = false;
                return nullptr;
            }
            const RowJob* job = &S.jobs[batch.at][at];
            at = job->last ? -1 : at + 1;
            return job;
        };
        // a job that has been done with gives its batch back if it is the batch's last
        auto leave = [&](const RowJob* job) {
            __syncwarp();
            if (job->last && lane == 0) mbar_arrive(&S.job_empty[(job - S.jobs[0]) / kBatch]);
        };
        // pass 1 of a row, as far as it has come
        Stats st;
        bool bad;
        int i1;
        auto open1 = [&](const RowJob* job) {
            st = stats_empty();
            bad = false;
            i1 = job->part.first;
        };
        // goes on for `most` chunks at most; at the row's end puts the sums into the cluster's join
        auto pass1 = [&](const RowJob* job, int most) {
            const RowPart part = job->part;
            const Two c_hi = two(job->c_hi, job->c_hi), c_lo = two(job->c_lo, job->c_lo);
            const float c = job->c;
            for (; i1 < part.last && most > 0; i1 += kChunkVecs, --most) {
                ok = wait(&S.full[slot1.at], slot1.phase, P.wait_ns);
                if (!ok) break;
                const uint4* in = reinterpret_cast<const uint4*>(ring + slot1.at * kChunkBytes) + tid;
                // whole chunks at the row's ends, too: 2048 x 50257 bf16 scored in 43 us (47 without), 100001 fp32 126 (137),
                // 128000 bf16 91 (90); with a gradient that gains nothing
                if (kGrad ? part.inner(i1) : i1 + kChunkVecs <= part.last) {
                    uint4 v[kVecs];
#pragma unroll
                    for (int k = 0; k < kVecs; ++k) v[k] = in[k * kConsumers];
                    if (!kGrad && !part.inner(i1)) {
                        const int hi = vocab + part.head;
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) {
                            const int ik = i1 + tid + k * kConsumers;
                            if (ik == 0 || ik == part.count - 1)
                                Elems<T>::mask(v[k], part.head - ik * kPer, hi - ik * kPer);
                        }
                    }
                    fold<T, kEntropy, kVecs>(st, bad, v, c_hi, c_lo, c);
                } else {
                    const int hi = vocab + part.head;
#pragma unroll 1
                    for (int ik = i1 + tid, k = 0; k < kVecs && ik < part.last; ++k, ik += kConsumers) {
                        uint4 v[1] = {in[k * kConsumers]};
                        if (ik == 0 || ik == part.count - 1)
                            Elems<T>::mask(v[0], part.head - ik * kPer, hi - ik * kPer);
                        fold<T, kEntropy, 1>(st, bad, v, c_hi, c_lo, c);
                    }
                }
                if (!kGrad) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.empty[slot1.at]);
                }
                slot1.next(slots);
            }
            if (!ok || i1 < part.last || i1 == kPut) return;
            i1 = kPut;
            if (bad) st.s = quiet_nan();
            stats_warp<kEntropy>(st, c);
            // A buffer of sums is written again four rows later. By then this CTA has closed the row two before
            // this one, so every warp of the cluster had come to that row's join, and each had seen the row two
            // before that closed in its own CTA: all closers are done with the buffer. (With a gradient, pass 2
            // has waited for it.)
            if (!kGrad) {
                if (behind == 2) {
                    ok = wait(&S.closed[cp.at], cp.phase, P.wait_ns);
                    if (!ok) return;
                    cp.next(kSums);
                } else {
                    ++behind;
                }
            }
            if (uint32_t(lane) < parts)
                put_sums(dsmem_map(smem_addr(sums + (sp.at * parts + rank) * kWarps + warp), lane),
                         dsmem_map(smem_addr(&S.join[sp.at]), lane), st.ref, st.s, st.t, 0.f);
            sp.next(kSums);
        };
        auto pass2 = [&](const RowJob* job) {
            const RowPart part = job->part;
            T* g = static_cast<T*>(part.grad);
            ok = wait(&S.closed[cp.at], cp.phase, P.wait_ns);
            if (!ok) return;
            const RowRecord rec = S.rec[cp.at];
            cp.next(kSums);
            const Factors f = factors(rec);
            const int tok = rec.token < kNoToken ? rec.token + part.head : -1;
            for (int i0 = part.first; i0 < part.last; i0 += kChunkVecs) {
                const uint4* in = reinterpret_cast<const uint4*>(ring + slot2.at * kChunkBytes) + tid;
                const int i = i0 + tid;
                if (part.whole && part.inner(i0) && unsigned(tok - i0 * kPer) >= unsigned(kChunkVecs * kPer)) {
                    uint4* out = reinterpret_cast<uint4*>(g + (i * kPer - part.head));
#pragma unroll
                    for (int k = 0; k < kVecs; ++k)
                        __stcs(out + k * kConsumers, gradient<T, kEntropy>(in[k * kConsumers], f));
                } else {
#pragma unroll 1
                    for (int ik = i, k = 0; k < kVecs && ik < part.last; ++k, ik += kConsumers) {
                        const uint4 v = in[k * kConsumers];
                        put_vector(g, vocab, part.head, ik, part.whole,
                                   gradient_token<T, kEntropy>(v, f, tok - ik * kPer, rec.at_token));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.empty[slot2.at]);
                slot2.next(slots);
            }
        };
        const RowJob* job = next_job();
        if (ok) open1(job);
        while (ok && job->row >= 0) {
            const RowJob* next = nullptr;
            if (job->live) {
                pass1(job, kMaxSlots);
                if (ok && kGrad) {
                    // pass 1 of the next row as far as the ring holds it beside this one
                    next = next_job();
                    if (ok) open1(next);
                    if (ok && next->row >= 0 && next->live)
                        pass1(next, int(slots) - (job->part.last - job->part.first + kChunkVecs - 1) / kChunkVecs);
                    if (ok) pass2(job);
                }
                if (!ok) gave_up(S);
            } else if (kGrad) {
                const RowPart part = job->part;
                for (int i = part.first + tid; i < part.last; i += kConsumers)
                    put_vector(static_cast<T*>(part.grad), vocab, part.head, i, part.whole, make_uint4(0u, 0u, 0u, 0u));
            }
            if (!ok) break;
            leave(job);
            if (!next) {
                next = next_job();
                if (!ok) break;
                open1(next);
            }
            job = next;
        }
    }
    // no CTA leaves while another may still write to its shared memory
    __syncwarp();
    cluster_sync();
    if (S.failed) abandon<T, kGrad>(P, q, n_clusters, parts, rank);
    if (P.mode == kModePolicy && rank == 0 &&  // the first CTAs have written the rows' shares
        last_block(P.ws.ticket, n_clusters, &S.flag)) {
        const double loss = sum_terms<kThreads>(P.ws.terms, a.n_rows, S.scratch);
        if (tid == 0) *P.policy.out_loss = float(loss);
    }
}

// ---------------------------------------------------------------- small rows
// Rows of up to kSmallVecs vectors for each thread of kGroup warps stay in
// registers from pass 1 to pass 2, and a row is a group's whole work: what such
// rows cost is latency, and with no roles and no ring many of them are under way
// on an SM at once, or few are done with sooner. (Clusters of such blocks, for few
// longer rows, gained nothing with a gradient, and without one took 12 us against
// the ring's 7.8 for 32 x 151936 bf16.)
constexpr int kSmallVecs = 8;
constexpr int kSmallBlock = 4;  // rows of one warp that share a block

constexpr int small_threads(int group) { return 32 * (group == 1 ? kSmallBlock : group); }
constexpr int kSmallResident = 896;  // threads of an SM, with a gradient (1024: registers spill, 4096 x 4000 fp32 30 / 29 us)

template <typename T, bool kGrad, bool kEntropy, int kGroup>
__global__ void __launch_bounds__(small_threads(kGroup), kGrad ? kSmallResident / small_threads(kGroup) : 0)
    small_rows_kernel(const __grid_constant__ LossParams P)
{
    constexpr int kPer = Elems<T>::kPer, kStep = 32 * kGroup;
    __shared__ float4 sums[kGroup];
    __shared__ RowRecord shared_rec;
    __shared__ double scratch[kGroup == 1 ? kSmallBlock : kGroup];
    __shared__ uint32_t flag;
    const sampler_rows_t& a = P.rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tid = kGroup == 1 ? lane : int(threadIdx.x);
    const int64_t r = kGroup == 1 ? int64_t(blockIdx.x) * kSmallBlock + warp : int64_t(blockIdx.x);
    if (P.mode == kModePairs) dependent_launch();
    if (kGroup > 1 || r < a.n_rows) {
        RowJob job;
        float temperature;
        job.row = int32_t(r);
        job_load(job, temperature, P, r);
        job.live = job.weight != 0.f;
        const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
        const RowSpan span = row_span(x, a.vocab);
        const uint4* from = reinterpret_cast<const uint4*>(x - span.head);
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
        const int vocab = int(a.vocab), hi = vocab + span.head;
        uint4 v[kSmallVecs];
#pragma unroll
        for (int k = 0; k < kSmallVecs; ++k) {
            const int i = tid + k * kStep;
            v[k] = make_uint4(none, none, none, none);
            if (job.live && i < span.count) v[k] = __ldcs(from + i);
        }
        job_token<T>(job, a, r, job.live);
        row_scale(job, a, temperature);
#pragma unroll
        for (int k = 0; k < kSmallVecs; ++k) {
            const int i = tid + k * kStep;
            if (i == 0 || i == span.count - 1) Elems<T>::mask(v[k], span.head - i * kPer, hi - i * kPer);
        }
        Stats st = stats_empty();
        bool bad = false;
        fold<T, kEntropy, kSmallVecs>(st, bad, v, two(job.c_hi, job.c_hi), two(job.c_lo, job.c_lo), job.c);
        if (bad) st.s = quiet_nan();
        stats_warp<kEntropy>(st, job.c);
        if (kGroup > 1) {
            if (lane == 0) sums[warp] = make_float4(st.ref, st.s, st.t, 0.f);
            __syncthreads();
            if (warp == 0) {
                st = stats_empty();
                if (lane < kGroup) st = Stats{sums[lane].x, sums[lane].y, sums[lane].z};
                stats_warp<kEntropy>(st, job.c);
            }
        }
        RowRecord rec;
        if (kGroup == 1 || warp == 0) {
            RowOut out;
            row_close(P, job, st,
                      kGrad && P.mode == kModePolicy ? scale_of_grad(P.policy.grad_scale, P.policy.grad_scale_dev) : 1.f,
                      rec, out);
            if (kGroup > 1 && lane == 0) shared_rec = rec;
            if (lane == 0) row_write(P, r, rec, out);
        }
        if (kGrad) {
            if (kGroup > 1) {
                __syncthreads();
                rec = shared_rec;
            }
            T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
            const bool whole = ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
            const Factors f = factors(rec);
            const int tok = rec.token >= 0 && rec.token < kNoToken ? rec.token + span.head : -kPer;
#pragma unroll
            for (int k = 0; k < kSmallVecs; ++k) {
                const int i = tid + k * kStep;
                // the vector is widened again: pass 1's wide values, kept till here, take half of the registers (16384 x
                // 8000 bf16 145 us, so 106)
                asm volatile("" : "+r"(v[k].x), "+r"(v[k].y), "+r"(v[k].z), "+r"(v[k].w));
                if (i < span.count)
                    put_vector(g, vocab, span.head, i, whole,
                               rec.token < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                             : gradient_token<T, kEntropy>(v[k], f, tok - i * kPer, rec.at_token));
            }
        }
    }
    if (P.mode == kModePolicy && last_block(P.ws.ticket, gridDim.x, &flag)) {
        const double loss = sum_terms<kGroup == 1 ? 32 * kSmallBlock : kStep>(P.ws.terms, a.n_rows, scratch);
        if (threadIdx.x == 0) *P.policy.out_loss = float(loss);
    }
}

// ---------------------------------------------------------------- pairs
constexpr int kPairThreads = 256;

// One block for a pair, a half of it for an answer: the answer's sums, the
// pair's share of the loss, and the gradient's factors of the rows. The sums are
// in double (a reward is a small difference of long sums); what follows from the
// margin is in fp32, in forms that lose nothing where a sigmoid is near 0 or 1.
// The host cannot look at the offsets, and where they decrease a row may lie in
// several answers: each counts itself in the row's record, the first to come
// there alone writes the factors, and a row with a count above one gets NaN in
// the next kernel, whichever came first.
__global__ void __launch_bounds__(kPairThreads) pairs_kernel(const sampler_rows_t a, const sampler_preference_t q,
                                                             const RowWorkspace ws)
{
    constexpr int kHalf = kPairThreads / 2, kWarpsHalf = kHalf / 32;
    __shared__ double part[2][2 * kWarpsHalf];
    __shared__ double scratch[kPairThreads / 32];
    __shared__ double rewards[2];
    __shared__ uint32_t flag;
    const int64_t i = blockIdx.x;
    const int k = threadIdx.x / kHalf, t = threadIdx.x % kHalf;
    const int64_t b = q.seq_offsets[2 * i + k], e = q.seq_offsets[2 * i + k + 1];
    const bool ok = b >= 0 && b <= e && e <= a.n_rows;
    const int64_t begin = ok ? b : 0, end = ok ? e : 0;
    dependent_wait();
    dependent_launch();  // not before: the gradient's blocks would take the rows' kernel's place on the SMs
    double s = 0.0, n = 0.0;
    for (int64_t r = begin + t; r < end; r += kHalf) {
        const float w = a.weight ? a.weight[r] : 1.f;
        if (w == 0.f) continue;
        s += double(w) * (ws.terms[r] - (q.ref_logprob ? double(q.ref_logprob[r]) : 0.0));
        n += double(w);
    }
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if ((t & 31) == 0) {
        part[k][t >> 5] = s;
        part[k][kWarpsHalf + (t >> 5)] = n;
    }
    __syncthreads();
    s = n = 0.0;
    for (int w = 0; w < kWarpsHalf; ++w) {
        s += part[k][w];
        n += part[k][kWarpsHalf + w];
    }
    const double share = !q.mean_over_tokens ? 1.0 : n != 0.0 ? 1.0 / n : 0.0;
    const double reward = ok ? double(q.beta) * (s * share) : double(quiet_nan());
    if (t == 0) {
        rewards[k] = reward;
        if (q.out_reward) q.out_reward[2 * i + k] = float(reward);
    }
    __syncthreads();
    const float z = float(rewards[0] - rewards[1] - double(q.margin));
    const float eps = q.label_smoothing, small = expf(-fabsf(z));  // exp of the negative magnitude
    if (threadIdx.x == 0) {
        // -ln sigmoid(z) = max(-z, 0) + ln(1 + exp(-|z|)); a share of 0 takes no part, even of an infinity
        const float tail = log1pf(small);
        const float chosen = eps != 1.f ? (1.f - eps) * (fmaxf(-z, 0.f) + tail) : 0.f;
        const float other = eps != 0.f ? eps * (fmaxf(z, 0.f) + tail) : 0.f;
        ws.pair_terms[i] = double(isnan(z) ? z : chosen + other);
    }
    if (a.out_grad) {
        // d loss / d z = eps - sigmoid(-z)
        const float by_z = eps - __fdiv_rn(z > 0.f ? small : 1.f, 1.f + small);
        const float by_sum =
            float(double(k ? -by_z : by_z) * (double(q.beta) * share / double(q.n_pairs))) *
            scale_of_grad(q.grad_scale, q.grad_scale_dev);
        for (int64_t r = begin + t; r < end; r += kHalf) {
            RowRecord& to = ws.records[r];
            const uint32_t before = atomicAdd(&to.answers, 1u);
            RowRecord rec = to;
            if (rec.token < 0 || before != 0u) continue;
            set_factors(rec, (a.weight ? a.weight[r] : 1.f) * by_sum, 0.f, 0.f, 0.f);
            to.k0 = rec.k0;
            to.at_token = rec.at_token;
        }
    }
    if (last_block(ws.ticket, gridDim.x, &flag)) {
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
    dependent_wait();
    RowRecord rec = ws.records[r];
    if (rec.answers > 1u) rec.k0 = rec.at_token = quiet_nan();
    const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
    T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
    const RowSpan span = row_span(x, a.vocab);
    const bool whole = ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
    const uint4* from = reinterpret_cast<const uint4*>(x - span.head);
    const int first = int(blockIdx.x) * kGradThreads * kGradVecs + threadIdx.x;
    const Factors f = factors(rec);
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
            put_vector(g, int(a.vocab), span.head, i, whole,
                       zero ? v[k] : gradient_token<T, false>(v[k], f, tok - i * Elems<T>::kPer, rec.at_token));
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

using SmallKernel = void (*)(const LossParams);

template <typename T, int kGroup>
SmallKernel small_kernel_for(bool grad, bool entropy)
{
    return grad ? entropy ? rows::small_rows_kernel<T, true, true, kGroup> : rows::small_rows_kernel<T, true, false, kGroup>
           : entropy ? rows::small_rows_kernel<T, false, true, kGroup>
                     : rows::small_rows_kernel<T, false, false, kGroup>;
}

template <typename T>
SmallKernel small_kernel(int group, bool grad, bool entropy)
{
    return group == 1   ? small_kernel_for<T, 1>(grad, entropy)
           : group == 2 ? small_kernel_for<T, 2>(grad, entropy)
           : group == 4 ? small_kernel_for<T, 4>(grad, entropy)
           : group == 8 ? small_kernel_for<T, 8>(grad, entropy)
                        : small_kernel_for<T, 16>(grad, entropy);
}

// Warps whose registers a row stays in; 0 for the kernel with a ring. Rows of up to 16 KB (four warps) always do
// (policy with its gradient, against the ring: 4096 x 2000 bf16 13.5 / 29 us, 4096 x 4000 fp32 29 / 38, 4096 x 8000
// bf16 32 / 43, 16 x 1024 fp32 5.2 / 7.4). Larger groups are too few on an SM for the way from a row's loads to its
// stores, so they are taken where rows are few, or without a gradient: eight warps with a gradient 400 x 16000 bf16
// 10.3 / 12.8 us, 600 x 16000 15.8 / 15.7, 4096 x 16000 61 / 58; without 64 x 8000 fp32 3.1 / 5.3, 4096 x 16000 26 / 34;
// sixteen with 150 x 32000 bf16 8.6 / 11.4, 300 x 32000 17 / 16; without 64 x 32000 3.8 / 6.0, 600 x 32000 11 / 14,
// 4096 x 32000 53 / 50.
int small_group(int64_t vecs, int64_t n_rows, int sms, bool grad)
{
    int group = 1;
    while (group <= 16 && vecs > group * 32 * rows::kSmallVecs) group *= 2;
    const int64_t most = group <= 4 ? INT64_MAX : group == 8 ? (grad ? 3 * sms : INT64_MAX) : grad ? sms : 4 * sms;
    return group <= 16 && n_rows <= most ? group : 0;
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
    const int group = small_group(vecs, p.rows.n_rows, sms, grad);
    if (group) {
        const SmallKernel small = es == 2 ? small_kernel<uint16_t>(group, grad, entropy) : small_kernel<float>(group, grad, entropy);
        const int64_t blocks = group == 1 ? (p.rows.n_rows + rows::kSmallBlock - 1) / rows::kSmallBlock : p.rows.n_rows;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(blocks));
        cfg.blockDim = dim3(unsigned(rows::small_threads(group)));
        cfg.stream = stream;
        return cudaLaunchKernelEx(&cfg, small, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
    }
    // parts of at most kPartChunks chunks; smaller ones while few rows leave the device unfilled (policy with its
    // gradient, against parts of kPartChunks: 1 x 151936 bf16 8.9 / 11.0 us, 8 x 128000 8.9 / 10.7, 32 x 32000 8.8 / 11)
    int parts = 1;
    while (parts < rows::kMaxParts && ((vecs + parts - 1) / parts > rows::kPartChunks * rows::kChunkVecs ||
                                       p.rows.n_rows * parts * 2 <= sms))
        parts *= 2;
    rows::RowPlan plan;
    // whole vectors for every consumer, and whole chunks where that makes the largest part little larger (2048 x 151936
    // bf16, 5 % larger: 210 us against 214.5; 127 x 50257 fp32, 23 % larger: 18.3 against 17.6)
    const int64_t part = (vecs + parts - 1) / parts;
    const int64_t even = (part + rows::kConsumers - 1) / rows::kConsumers * rows::kConsumers;
    const int64_t chunks = (part + rows::kChunkVecs - 1) / rows::kChunkVecs * rows::kChunkVecs;
    plan.part_vecs = int(chunks * 16 <= even * 17 ? chunks : even);
    plan.slots = rows::slots_for(parts);
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

namespace {

// As the programmatic dependent of the kernel enqueued before, or (not first)
// after it.
template <typename... Args>
bool launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, bool dependent, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

}  // namespace

int pairs_launch(const sampler_rows_t& rows, const sampler_preference_t& pref, const RowWorkspace& ws,
                 cudaStream_t stream)
{
    // (with no rows there is no kernel of this call before it)
    return launch_dependent(rows::pairs_kernel, dim3(unsigned(pref.n_pairs)), rows::kPairThreads, rows.n_rows > 0,
                            stream, rows, pref, ws)
               ? SAMPLER_OK
               : SAMPLER_ERR_CUDA;
}

int pairs_grad_launch(const sampler_rows_t& rows, const RowWorkspace& ws, bool dependent, cudaStream_t stream)
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
        const bool ok = es == 2 ? launch_dependent(rows::pairs_grad_kernel<uint16_t>, grid, rows::kGradThreads,
                                                   dependent && done == 0, stream, some, at)
                                : launch_dependent(rows::pairs_grad_kernel<float>, grid, rows::kGradThreads,
                                                   dependent && done == 0, stream, some, at);
        if (!ok) return SAMPLER_ERR_CUDA;
    }
    return SAMPLER_OK;
}

}  // namespace dst
