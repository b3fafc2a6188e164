// row_loss_kernel.cu -- scoring and the losses over logits rows: logprob,
// entropy, the clipped policy loss, the preference loss, and the logits'
// gradients.
//
// One block takes one row at a time: a pass over the row for the running
// reference and the sums, one thread's work on them (row_close), and a second
// pass that writes the gradient.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "row_loss.cuh"

namespace dst {
namespace rows {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ void row_zero(T* g, int64_t vocab)
{
    for (int64_t v = threadIdx.x; v < vocab; v += kThreads) store_grad(g + v, 0.f);
}

template <typename T>
__device__ __forceinline__ void row_write(const T* x, T* g, int64_t vocab, const RowRecord& rec)
{
    for (int64_t v = threadIdx.x; v < vocab; v += kThreads) {
        const float u = fmaxf((load_logit(x + v) - rec.ref) * rec.c, kLowest);
        float y = exp2_fast(u) * fmaf(rec.k1, u, rec.k0);
        if (v == rec.token) y += rec.at_token;
        store_grad(g + v, y);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ LossParams P)
{
    __shared__ Stats part[kWarps];
    __shared__ RowRecord rec;
    __shared__ double scratch[kWarps];
    __shared__ uint32_t flag;
    const sampler_rows_t& a = P.rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
        const RowHead h = row_open(a, r);
        const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
        T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
        const bool read = h.live && !h.bad_param;
        Stats st = stats_empty();
        if (read) {
            for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) {
                const float xv = load_logit(x + v);
                if (!(xv < pos_inf())) st.bad = 1u;
                if (xv == neg_inf() || st.bad) continue;
                if (xv > st.ref) st = stats_join(st, Stats{xv, 0.f, 0.f, 0u}, h.c);
                const float u = (xv - st.ref) * h.c, e = exp2_fast(u);
                st.s += e;
                st.t = fmaf(e, fmaxf(u, kLowest), st.t);
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            Stats q;
            q.ref = __shfl_xor_sync(0xffffffffu, st.ref, o);
            q.s = __shfl_xor_sync(0xffffffffu, st.s, o);
            q.t = __shfl_xor_sync(0xffffffffu, st.t, o);
            q.bad = __shfl_xor_sync(0xffffffffu, st.bad, o);
            st = stats_join(st, q, h.c);
        }
        if (lane == 0) part[warp] = st;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWarps; ++w) st = stats_join(st, part[w], h.c);
            RowRecord mine;
            row_close(P, r, h, st, read ? load_logit(x + h.token) : 0.f, true, mine);
            rec = mine;
        }
        __syncthreads();
        if (a.out_grad && P.mode != kModePairs) {
            if (rec.token < 0)
                row_zero(g, a.vocab);
            else
                row_write(x, g, a.vocab, rec);
        }
        __syncthreads();
    }
    if (P.mode == kModePolicy && last_block(P.ws.ticket, gridDim.x, &flag)) {
        const double loss = sum_terms<kThreads>(P.ws.terms, a.n_rows, scratch);
        if (threadIdx.x == 0) *P.policy.out_loss = float(loss);
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
    if (last_block(ws.ticket, gridDim.x, &flag)) {
        const double loss = sum_terms<kPairThreads>(ws.pair_terms, q.n_pairs, scratch);
        if (threadIdx.x == 0) *q.out_loss = float(loss / double(q.n_pairs));
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pairs_grad_kernel(const sampler_rows_t a, const RowWorkspace ws)
{
    for (int64_t r = blockIdx.x; r < a.n_rows; r += gridDim.x) {
        const RowRecord rec = ws.records[r];
        const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
        T* g = static_cast<T*>(a.out_grad) + r * a.grad_stride;
        if (rec.token < 0 || (rec.k0 == 0.f && rec.at_token == 0.f))
            row_zero(g, a.vocab);
        else
            row_write(x, g, a.vocab, rec);
    }
}

}  // namespace rows

int rows_launch(const LossParams& p, int sms, cudaStream_t stream)
{
    const unsigned grid = unsigned(std::min<int64_t>(p.rows.n_rows, int64_t(sms) * 4));
    if (p.rows.dtype == SAMPLER_DTYPE_BF16)
        rows::rows_kernel<uint16_t><<<grid, rows::kThreads, 0, stream>>>(p);
    else
        rows::rows_kernel<float><<<grid, rows::kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

int pairs_launch(const sampler_rows_t& rows, const sampler_preference_t& pref, const RowWorkspace& ws,
                 cudaStream_t stream)
{
    rows::pairs_kernel<<<unsigned(pref.n_pairs), rows::kPairThreads, 0, stream>>>(rows, pref, ws);
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

int pairs_grad_launch(const sampler_rows_t& rows, const RowWorkspace& ws, int sms, cudaStream_t stream)
{
    const unsigned grid = unsigned(std::min<int64_t>(rows.n_rows, int64_t(sms) * 4));
    if (rows.dtype == SAMPLER_DTYPE_BF16)
        rows::pairs_grad_kernel<uint16_t><<<grid, rows::kThreads, 0, stream>>>(rows, ws);
    else
        rows::pairs_grad_kernel<float><<<grid, rows::kThreads, 0, stream>>>(rows, ws);
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
