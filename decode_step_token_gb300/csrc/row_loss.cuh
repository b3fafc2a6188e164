// row_loss.cuh -- what one logits row contributes to a score, a loss and their
// gradients, given the statistics of the row.
//
// Exponents are kept in base 2: with c = log2(e) / T, element v of a row has
//     u_v = (x_v - ref) * c,    e_v = 2^u_v,    s = sum e_v,    t = sum e_v u_v,
// where ref is the row's largest element. The difference is taken before the
// product: a product less the rounded product of the largest element would be
// one operation, but where x_v c passes 2^24 (a row of the type's lowest value,
// a T near 1e-5) it would leave the rounding of that product in every exponent.
// Then
//     p_v = e_v / s,   ln p_t = (x_t - ref) / T - ln s,   entropy = ln s - ln2 * t / s,
// and a loss with gradient a by the logprob and b by the entropy has
//     d loss / d x_v = (a (1[v = t] - p_v) - b p_v (ln p_v + entropy)) / T
//                    = e_v (k0 + k1 u_v) + 1[v = t] a / T,
//     k0 = -(a + b (entropy - ln s)) / (s T),    k1 = -b ln2 / (s T).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "launch.h"

namespace dst {
namespace rows {

constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;  // log2(e) as a pair
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGreedyT = 1e-5f;  // below it a row is greedy and its outputs use T = 1
constexpr int32_t kNoToken = 0x7fffffff;  // of a row with an error status: matches no element
constexpr float kLowest = -3e4f;   // exponents are not taken below this where they are multiplied by 2^u (= 0)
// ex2.approx is on average this much too small, of its value (means of -2.5e-8 to -5.0e-8 over ranges of length 0.5
// to 20 below 0; at most 1.5e-7). A row's sum is, too, but for the exact 1 of its largest element, and so would be
// all logprobs of a sequence the same way. The mean error of 2048 logprobs against 64 bits, without and with this:
// 4.4e-8 and 1.0e-8 (128000 bf16), 4.7e-8 and 0.8e-8 (1024 fp32), 7.5e-8 and 4.0e-8 (151936 fp32).
constexpr float kExp2Short = 4e-8f;
constexpr float kFloatMax = 3.402823466e38f;

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }
__device__ __forceinline__ float pos_inf() { return __int_as_float(0x7f800000); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Sums of a part of a row relative to a reference of its own, which is at least
// the lowest float: a -inf logit is then infinitely far below it and adds
// nothing. A part with a NaN or +inf logit has s = NaN, an empty one s = 0.
struct Stats {
    float ref, s, t;
};

__device__ __forceinline__ Stats stats_empty() { return Stats{-kFloatMax, 0.f, 0.f}; }

// `a` relative to a reference that is at least its own.
__device__ __forceinline__ void stats_move(Stats& a, float ref, float c)
{
    const float d = fmaxf((a.ref - ref) * c, kLowest), f = exp2_fast(d);
    a.t = f * fmaf(a.s, d, a.t);
    a.s *= f;
    a.ref = ref;
}

// log2(e) / T as a pair (of RowJob), and as the float that is nearest to it.
struct Scale {
    float c_hi, c_lo;
    __device__ __forceinline__ float nearest() const { return __fadd_rn(c_hi, c_lo); }
};

// The same by the pair. (What moves is all that was added up before: an error in its exponent is one of all of that, the
// same way each time, and RowJob's c is up to 1.9 units of 2^-24 off.)
__device__ __forceinline__ void stats_move(Stats& a, float ref, const Scale& q)
{
    const float x = a.ref - ref, d = fmaxf(fmaf(x, q.c_hi, x * q.c_lo), kLowest), f = exp2_fast(d);
    a.t = f * fmaf(a.s, d, a.t);
    a.s *= f;
    a.ref = ref;
}

// The largest of all lanes' values, in every lane.
__device__ __forceinline__ float max_warp(float x)
{
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

template <bool kEntropy>
__device__ __forceinline__ void sum_warp(Stats& a)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        if (kEntropy) a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
    }
}

// The statistics of all lanes' parts, in every lane (t where kEntropy).
template <bool kEntropy, typename C>
__device__ __forceinline__ void stats_warp(Stats& a, const C& c)
{
    stats_move(a, max_warp(a.ref), c);
    sum_warp<kEntropy>(a);
}

// A CTA's part of a row: vectors first .. last of the `count` 16-byte vectors that
// cover it, the first of which begins `head` elements before the row.
struct RowPart {
    int32_t head, count, first, last;
    int32_t inner_first, inner_last;  // first vectors of the chunks that are whole and lie wholly inside the row
    int32_t whole;   // the gradient's vectors lie as the logits' do
    void* grad;      // the row's gradient
    // whether the chunk from vector i on is whole and lies wholly inside the row
    __device__ __forceinline__ bool inner(int i) const { return i >= inner_first && i <= inner_last; }
};

// A row as the kernels take it up: its parameters and what its mode reads of it.
struct RowJob {
    RowPart part;
    int32_t row;      // -1: no more rows
    int32_t token;
    int32_t live;     // 0: left out
    int32_t bad_param;
    int32_t last;     // of its batch
    float weight;
    float x_t;        // the token's logit
    float c, c_hi, c_lo;    // log2(e) / T, rounded, and as a pair: c_lo > 0
    float inv_t, inv_t_lo;  // 1 / T as a pair
    float in0, in1, in2;    // kModeScoreGrad: the gradients by logprob and entropy; kModePolicy: advantage,
                            // old_logprob, ref_logprob
};

// Sums and products of two floats without rounding, as pairs (Dekker, Knuth).
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
    return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}

// What follows of a row from its temperature. The pair c_hi + c_lo matters where
// sums are taken: c alone is off by up to 2^-24 of itself in every exponent the
// same way, which is an error of the logprob of that times the row's mean depth,
// and does not average out over a sequence. c_lo > 0 keeps -inf * c_lo = -inf.
__device__ __forceinline__ void row_scale(RowJob& h, const sampler_rows_t& a, float T)
{
    h.bad_param = !(T >= 0.f) || isinf(T) || h.token < 0 || int64_t(h.token) >= a.vocab;
    const float Te = T >= kGreedyT ? T : 1.f;  // a NaN or a negative T: the row is not used
    h.inv_t = __fdiv_rn(1.f, Te);
    h.inv_t_lo = fmaf(-Te, h.inv_t, 1.f) * h.inv_t;
    h.c = kLog2e * h.inv_t;
    const float rest = fmaf(kLog2e, h.inv_t, -h.c) + fmaf(kLog2e, h.inv_t_lo, kLog2eRest * h.inv_t);
    // `rest` is above -1.8 units of c's last place (half of one, one by inv_t's rounding, and kLog2eRest's): four
    // steps down, which are two of them just above a power of two
    h.c_hi = __int_as_float(__float_as_int(h.c) - 4);
    h.c_lo = (h.c - h.c_hi) + rest;
}

// ln s, off by about 3e-8: the exponent's part exactly (ln 2 = 355/512 less a
// small rest, after Cody and Waite), the mantissa's (within [1/sqrt 2, sqrt 2],
// so of magnitude below 0.35) by logf.
__device__ __forceinline__ Pair log_of(float s)
{
    int e;
    float f = frexpf(s, &e);  // [0.5, 1)
    if (f < 0.70710678f) {
        f *= 2.f;
        --e;
    }
    const float n = float(e);
    const Pair p = two_sum(n * 0.693359375f, logf(f));
    return two_sum(p.hi, p.lo - n * 2.1219444005469058e-4f);
}

// ln p of the token with logit x_t.
__device__ __forceinline__ Pair logprob_of(const RowJob& h, const Stats& st, float x_t, const Pair& ln_s)
{
    const Pair d = two_sum(x_t, -st.ref);
    const float y = d.hi * h.inv_t;
    if (!(y >= -kFloatMax)) return Pair{y, 0.f};  // no mass
    const float rest = fmaf(d.hi, h.inv_t, -y) + fmaf(d.hi, h.inv_t_lo, d.lo * h.inv_t);
    const Pair p = two_sum(y, -ln_s.hi);
    const Pair q = two_sum(p.hi, p.lo + (rest - ln_s.lo));
    return q;
}

// exp(d) - d - 1 and exp(d) - 1, given exp(d). Near 0 the former is its Taylor
// series (to d^9: the next term is below 1e-8 of the sum at |d| = 0.5), where the
// differences would lose digits.
__device__ __forceinline__ float exp_less_linear(float d, float exp_d, float& expm1_d)
{
    if (fabsf(d) < 0.5f) {
        float p = 1.f / 362880.f;
        p = fmaf(p, d, 1.f / 40320.f);
        p = fmaf(p, d, 1.f / 5040.f);
        p = fmaf(p, d, 1.f / 720.f);
        p = fmaf(p, d, 1.f / 120.f);
        p = fmaf(p, d, 1.f / 24.f);
        p = fmaf(p, d, 1.f / 6.f);
        p = fmaf(p, d, 0.5f);
        const float k = d * d * p;
        expm1_d = d + k;
        return k;
    }
    expm1_d = exp_d - 1.f;
    return isinf(d) ? pos_inf() : expm1_d - d;
}

__device__ __forceinline__ float scale_of_grad(float scale, const float* dev) { return dev ? scale * *dev : scale; }

// The factors of a row's gradient from those by its logprob (a) and entropy (b).
__device__ __forceinline__ void set_factors(RowRecord& rec, float a, float b, float entropy, float ln_s)
{
    const float q = rec.inv_s * rec.inv_t;
    rec.k0 = -(b != 0.f ? fmaf(b, entropy - ln_s, a) : a) * q;
    rec.k1 = -b * kLn2 * q;
    rec.at_token = a * rec.inv_t;
}

// A row's outputs and its share of the loss.
struct RowOut {
    Pair lp;
    float entropy, ratio, kl;
    double term;
    int status;
};

// What becomes of a row once its statistics are known (grad_scale: the whole
// factor of the gradient). A whole warp works on one row: where two exponentials
// are wanted, its halves take one each.
__device__ __forceinline__ void row_close(const LossParams& P, const RowJob& h, const Stats& st, float grad_scale,
                                          RowRecord& rec, RowOut& out)
{
    const sampler_rows_t& a = P.rows;
    rec.c = h.c;
    rec.ref = st.ref;
    rec.token = h.token;
    rec.inv_s = rec.inv_t = rec.k0 = rec.k1 = rec.at_token = 0.f;
    Pair lp = {0.f, 0.f};
    float entropy = 0.f, ratio = 0.f, kl = 0.f, term = 0.f;
    int status = SAMPLER_ROW_OK;
    if (!h.live) {
        rec.token = -1;
    } else {
        status = h.bad_param   ? SAMPLER_ROW_BAD_PARAM
                 : isnan(st.s) ? SAMPLER_ROW_NONFINITE
                 : st.s == 0.f ? SAMPLER_ROW_ALL_NEG_INF
                               : SAMPLER_ROW_OK;
        if (status != SAMPLER_ROW_OK) {
            // every value of the gradient becomes a multiple of NaN
            rec.c = rec.ref = 0.f;
            rec.token = kNoToken;
            rec.inv_s = rec.k0 = rec.at_token = quiet_nan();
            lp.hi = entropy = ratio = kl = term = quiet_nan();
        } else {
            rec.inv_s = __fdiv_rn(1.f, st.s);
            rec.inv_t = h.inv_t;
            Pair ln_s = log_of(st.s);
            ln_s.lo = fmaf(kExp2Short, 1.f - rec.inv_s, ln_s.lo);
            lp = logprob_of(h, st, h.x_t, ln_s);
            entropy = ln_s.hi + fmaf(-kLn2, st.t * rec.inv_s, ln_s.lo);
            if (P.mode == kModeScoreGrad) {
                set_factors(rec, h.in0, h.in1, entropy, ln_s.hi);
            } else if (P.mode == kModePolicy) {
                const sampler_policy_t& q = P.policy;
                const float A = h.in0;
                // the exponential of lp - old in the warp's lower half, of ref - lp in its upper
                const bool upper = threadIdx.x & 16;
                const Pair d = upper ? two_sum(h.in2, -lp.hi) : two_sum(lp.hi, -h.in1);
                const float e = isinf(d.hi) ? d.hi : d.hi + (upper ? d.lo - lp.lo : d.lo + lp.lo);
                const float E = expf(e);
                ratio = __shfl_sync(0xffffffffu, E, 0);
                const float lo = 1.f - q.clip_low, hi = 1.f + q.clip_high;
                const float plain = ratio * A;
                const float cut = fminf(fmaxf(ratio, lo), hi) * A;
                const float gain = plain < cut ? plain : plain >= cut ? cut : quiet_nan();
                const bool decided = (A > 0.f && ratio > hi) || (A < 0.f && ratio < lo);  // by the clip
                float by_lp = decided ? 0.f : -plain;
                term = -gain;
                if (q.ref_logprob) {
                    float em;
                    kl = exp_less_linear(__shfl_sync(0xffffffffu, e, 16), __shfl_sync(0xffffffffu, E, 16), em);
                    if (q.kl_coef != 0.f) {
                        term = fmaf(q.kl_coef, kl, term);
                        by_lp = fmaf(-q.kl_coef, em, by_lp);
                    }
                }
                if (q.entropy_coef != 0.f) term = fmaf(-q.entropy_coef, entropy, term);
                if (a.out_grad) {
                    const float g = h.weight * grad_scale;
                    set_factors(rec, g * by_lp, -g * q.entropy_coef, entropy, ln_s.hi);
                }
            }
        }
    }
    out.lp = lp;
    out.entropy = entropy;
    out.ratio = ratio;
    out.kl = kl;
    out.term = h.live ? double(h.weight) * double(term) : 0.0;
    out.status = status;
}

__device__ __forceinline__ void row_write(const LossParams& P, int64_t r, const RowRecord& rec, const RowOut& out)
{
    const sampler_rows_t& a = P.rows;
    if (a.out_logprob) a.out_logprob[r] = out.lp.hi;
    if (a.out_entropy) a.out_entropy[r] = out.entropy;
    if (a.out_status) a.out_status[r] = out.status;
    if (P.mode == kModePolicy) {
        if (P.policy.out_ratio) P.policy.out_ratio[r] = out.ratio;
        if (P.policy.out_kl) P.policy.out_kl[r] = out.kl;
        P.ws.terms[r] = out.term;
    }
    if (P.mode == kModePairs) {
        // the pairs' kernel takes the logprob from here and puts the gradient's factors in
        P.ws.terms[r] = double(out.lp.hi) + double(out.lp.lo);
        P.ws.records[r] = rec;
    }
}

// What is written of a row whose cluster gave up (see abandon): nothing of it is
// known, so its outputs, its share of the loss and all of its gradient are NaN.
// A row that is left out has its zeros as ever.
__device__ __forceinline__ void row_give_up(const LossParams& P, int64_t r, bool counts)
{
    const float x = counts ? quiet_nan() : 0.f;
    const RowRecord rec{0.f, 0.f, x, 0.f, x, counts ? kNoToken : -1, x, 0.f};
    const RowOut out{Pair{x, 0.f}, x, x, x, double(x), counts ? SAMPLER_ROW_TIMEOUT : SAMPLER_ROW_OK};
    row_write(P, r, rec, out);
}

// True in the last of `blocks` blocks to get here; what the others wrote before
// is then visible. Clears the ticket for the next launch. Called by every thread
// of a block; `flag` is a word of its shared memory.
__device__ __forceinline__ bool last_block(uint32_t* ticket, uint32_t blocks, uint32_t* flag)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const uint32_t got = atomicAdd(ticket, 1u);
        *flag = 0u;
        if (got + 1u == blocks) {
            *flag = 1u;
            *ticket = 0u;
            __threadfence();
        }
    }
    __syncthreads();
    return *flag != 0u;
}

// Sum of terms[0 .. n) in double by one block of kThreads threads, in an order
// that depends on n alone; the result is valid in thread 0.
template <int kThreads>
__device__ __forceinline__ double sum_terms(const double* terms, int64_t n, double* scratch)
{
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) v += __ldcg(terms + i);
    for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kThreads / 32; ++w) v += scratch[w];
    return v;
}

}  // namespace rows
}  // namespace dst
