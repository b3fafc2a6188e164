// row_queue.cuh -- which rows a cluster of CTAs takes, and how the warp that brings
// them in hands them to the others.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "row_vectors.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace rows {

// The rows of cluster `q` of `n_clusters`, in order: every n_clusters-th of those
// that count, and every n_clusters-th of those that are left out. One warp.
struct RowDealer {
    int64_t base;            // first row of the 32 in `mine`; without weights: the next row
    uint32_t mine;           // those of them that are this cluster's and have not been given out
    uint32_t is_live;        // those that count
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
    d.mine = d.is_live = d.live = d.dead = d.counts = 0;
    d.group = 3;
    if (a.weight) dealer_load(d, a, 0);
}

// The next row, -1 at the end; whether it counts.
__device__ __forceinline__ int64_t dealer_next(RowDealer& d, const sampler_rows_t& a, uint32_t q, uint32_t n_clusters,
                                               bool& counting)
{
    if (!a.weight) {
        counting = true;
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
        d.is_live = live;
        const uint32_t before = (1u << lane) - 1u;
        uint32_t rank = counts ? d.live + __popc(live & before) : d.dead + __popc(dead & before);
        rank %= n_clusters;
        d.mine = __ballot_sync(0xffffffffu, in && rank == q);
        d.live = (d.live + __popc(live)) % n_clusters;
        d.dead = (d.dead + __popc(dead)) % n_clusters;
    }
    const int bit = __ffs(d.mine) - 1;
    d.mine &= d.mine - 1u;
    counting = d.is_live >> bit & 1u;
    return d.base + bit;
}

// A row as it is handed over: what it needs besides its logits, read ahead, and what follows from that.
struct RowItem {
    int32_t row;   // -1: no more rows
    int32_t live;  // 0: left out
    int32_t last;  // of its batch
    int32_t token, bad_param;
    float weight, temperature;
    float x_t;     // the token's logit (0 without one)
    float c;                               // the float nearest to c_hi + c_lo
    float c_hi, c_lo, inv_t, inv_t_lo;     // as in RowJob
    int32_t head, count;                   // of its span of vectors
};

// What the functions of row_loss.cuh read of a row.
__device__ __forceinline__ RowJob job_of(const RowItem& i)
{
    RowJob h;
    h.token = i.token;
    h.bad_param = i.bad_param;
    h.x_t = i.x_t;
    h.c = i.c;
    h.c_hi = i.c_hi;
    h.c_lo = i.c_lo;
    h.inv_t = i.inv_t;
    h.inv_t_lo = i.inv_t_lo;
    return h;
}

constexpr int kQueueBatch = 8;  // rows whose parameters are fetched together
constexpr int kQueueFirst = 2;  // the first time, when all wait for them

struct RowQueue {
    uint64_t full[2], empty[2];
    RowItem items[2][kQueueBatch];
};

__device__ __forceinline__ void queue_open(RowQueue& S, int readers)
{
    for (int i = 0; i < 2; ++i) {
        mbar_init(&S.full[i], 1);
        mbar_init(&S.empty[i], uint32_t(readers));
    }
}

// The producer warp: deals out the rows of cluster `q`, hands each over and has copy_in(row, batch item) bring it in,
// where it counts; copy_in says whether it could. Ends with false where a wait gave up. want_token: x_t is read.
template <typename T, typename F>
__device__ __forceinline__ bool queue_fill(RowQueue& S, const sampler_rows_t& a, uint32_t q, uint32_t n_clusters,
                                           bool want_token, uint64_t wait_ns, F copy_in)
{
    const int lane = threadIdx.x & 31;
    RowDealer d;
    dealer_open(d, a, q);
    RingPlace batch{0, 0};
    bool end = false;
    for (int most = kQueueFirst; !end; most = kQueueBatch) {
        int count = 0;
        int64_t mine = -1;
        uint32_t live = 0;
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
        RowItem item;
        item.row = int32_t(mine);
        item.live = int32_t(live >> lane & 1u);
        item.last = lane == count - 1;
        item.token = 0;
        item.temperature = item.weight = 1.f;
        item.x_t = 0.f;
        if (mine >= 0) {
            if (a.tokens) item.token = a.tokens[mine];
            if (a.temperature) item.temperature = a.temperature[mine];
            if (a.weight) item.weight = a.weight[mine];
            const T* x = static_cast<const T*>(a.logits) + mine * a.row_stride;
            if (want_token && a.tokens && item.live && item.token >= 0 && int64_t(item.token) < a.vocab)
                item.x_t = load_logit(x + item.token);
            RowJob h;
            h.token = item.token;
            row_scale(h, a, item.temperature);
            item.bad_param = h.bad_param;
            item.c = Scale{h.c_hi, h.c_lo}.nearest();
            item.c_hi = h.c_hi;
            item.c_lo = h.c_lo;
            item.inv_t = h.inv_t;
            item.inv_t_lo = h.inv_t_lo;
            const RowSpan span = row_span(x, a.vocab);
            item.head = span.head;
            item.count = span.count;
        }
        if (!wait(&S.empty[batch.at], batch.phase ^ 1u, wait_ns)) return false;
        if (lane < count) S.items[batch.at][lane] = item;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.full[batch.at]);
        batch.next(2);
        for (int k = 0; k < count; ++k)
            if (live >> k & 1u)
                if (!copy_in(__shfl_sync(0xffffffffu, mine, k))) return false;
    }
    return true;
}

// Where a reading warp is in the queue.
struct QueuePlace {
    RingPlace batch;
    int k;
};

// The next row (row -1: the end), the same for all warps; false where the wait gave up.
__device__ __forceinline__ bool queue_next(RowQueue& S, QueuePlace& p, uint64_t wait_ns, RowItem& item)
{
    if (p.k == 0 && !wait(&S.full[p.batch.at], p.batch.phase, wait_ns)) return false;
    item = S.items[p.batch.at][p.k++];
    __syncwarp();
    if (item.last) {
        if ((threadIdx.x & 31) == 0) mbar_arrive(&S.empty[p.batch.at]);
        p.batch.next(2);
        p.k = 0;
    }
    return true;
}

}  // namespace rows
}  // namespace dst
