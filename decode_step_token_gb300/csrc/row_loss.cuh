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

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;
constexpr float kGreedyT = 1e-5f;  // below it a row is greedy and its outputs use T = 1
constexpr int32_t kNoToken = 0x7fffffff;  // of a row with an error status: matches no element
constexpr float kLowest = -3e4f;   // exponents are not taken below this where they are multiplied by 2^u (= 0)

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }
__device__ __forceinline__ float pos_inf() { return __int_as_float(0x7f800000); }
__device__ __forceinline__ float neg_inf() { return __int_as_float(int(0xff800000u)); }

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

// Sum of exponentials relative to a reference of its own. ref = -inf: nothing
// has been added (s = t = 0). bad: a NaN or +inf was met.
struct Stats {
    float ref, s, t;
    uint32_t bad;
};

__device__ __forceinline__ Stats stats_empty() { return Stats{neg_inf(), 0.f, 0.f, 0u}; }

// a and b, relative to the larger reference.
__device__ __forceinline__ Stats stats_join(const Stats& a, const Stats& b, float c)
{
    const float ref = fmaxf(a.ref, b.ref);
    Stats r;
    r.ref = ref;
    r.bad = a.bad | b.bad;
    if (ref == neg_inf()) {
        r.s = r.t = 0.f;
        return r;
    }
    const float da = fmaxf((a.ref - ref) * c, kLowest), db = fmaxf((b.ref - ref) * c, kLowest);
    const float fa = exp2_fast(da), fb = exp2_fast(db);
    r.s = a.s * fa + b.s * fb;
    r.t = fa * fmaf(a.s, da, a.t) + fb * fmaf(b.s, db, b.t);
    return r;
}

// A row's parameters.
struct RowHead {
    float c, inv_t;
    float weight;
    int32_t token;
    bool live;       // false: left out
    bool bad_param;
};

__device__ __forceinline__ RowHead row_open(const sampler_rows_t& a, int64_t r)
{
    RowHead h;
    h.weight = a.weight ? a.weight[r] : 1.f;
    h.live = h.weight != 0.f;
    h.token = a.tokens[r];
    const float T = a.temperature ? a.temperature[r] : 1.f;
    h.bad_param = !(T >= 0.f) || isinf(T) || h.token < 0 || int64_t(h.token) >= a.vocab;
    const float Te = T < kGreedyT ? 1.f : T;
    h.inv_t = __fdiv_rn(1.f, Te);
    h.c = __fdiv_rn(kLog2e, Te);
    return h;
}

// ln s to about 3e-8: the exponent's part in double, the mantissa's (within
// [1/sqrt 2, sqrt 2], so of magnitude below 0.35) by logf.
__device__ __forceinline__ double log_of(float s)
{
    int e;
    float f = frexpf(s, &e);  // [0.5, 1)
    if (f < 0.70710678f) {
        f *= 2.f;
        --e;
    }
    return double(e) * kLn2 + double(logf(f));
}

// exp(d) - d - 1. Near 0 its Taylor series (to d^9: the next term is below 1e-8
// of the sum at |d| = 0.5), where the difference would lose digits.
__device__ __forceinline__ float exp_less_linear(float d)
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
        return d * d * p;
    }
    return expm1f(d) - d;
}

__device__ __forceinline__ float scale_of_grad(float scale, const float* dev) { return dev ? scale * *dev : scale; }

// The factors of a row's gradient from those by its logprob (a) and entropy (b).
__device__ __forceinline__ void set_factors(RowRecord& rec, float a, float b, float entropy, float ln_s)
{
    const float q = rec.inv_s * rec.inv_t;
    rec.k0 = -(b != 0.f ? fmaf(b, entropy - ln_s, a) : a) * q;
    rec.k1 = -b * float(kLn2) * q;
    rec.at_token = a * rec.inv_t;
}

// One thread's work once a row's statistics are known (x_t: the token's logit):
// the row's outputs (where `write`), its share of the loss, and its record.
__device__ __forceinline__ void row_close(const LossParams& P, int64_t r, const RowHead& h, const Stats& st, float x_t,
                                          bool write, RowRecord& rec)
{
    const sampler_rows_t& a = P.rows;
    rec.c = h.c;
    rec.ref = st.ref;
    rec.token = h.token;
    rec.inv_s = rec.inv_t = rec.k0 = rec.k1 = rec.at_token = 0.f;
    float logprob = 0.f, entropy = 0.f, ratio = 0.f, kl = 0.f;
    double term = 0.0;
    int status = SAMPLER_ROW_OK;
    if (!h.live) {
        rec.token = -1;
    } else {
        status = h.bad_param ? SAMPLER_ROW_BAD_PARAM
                 : st.bad    ? SAMPLER_ROW_NONFINITE
                 : st.ref == neg_inf() ? SAMPLER_ROW_ALL_NEG_INF
                                       : SAMPLER_ROW_OK;
        if (status != SAMPLER_ROW_OK) {
            // every value of the gradient becomes a multiple of NaN
            rec.c = rec.ref = 0.f;
            rec.token = kNoToken;
            rec.inv_s = rec.k0 = rec.at_token = quiet_nan();
            logprob = entropy = ratio = kl = quiet_nan();
            term = double(quiet_nan());
        } else {
            rec.inv_s = __fdiv_rn(1.f, st.s);
            rec.inv_t = h.inv_t;
            const double ln_s = log_of(st.s);
            const double lp = (double(x_t) - double(st.ref)) * double(h.inv_t) - ln_s;
            logprob = float(lp);
            entropy = float(ln_s - kLn2 * double(__fdiv_rn(st.t, st.s)));
            if (P.mode == kModeScoreGrad) {
                set_factors(rec, P.grad_logprob[r], P.grad_entropy ? P.grad_entropy[r] : 0.f, entropy, float(ln_s));
            } else if (P.mode == kModePolicy) {
                const sampler_policy_t& q = P.policy;
                const float A = q.advantage[r];
                ratio = expf(float(lp - double(q.old_logprob[r])));
                const float lo = 1.f - q.clip_low, hi = 1.f + q.clip_high;
                const float plain = ratio * A;
                const float cut = fminf(fmaxf(ratio, lo), hi) * A;
                const float gain = plain < cut ? plain : plain >= cut ? cut : quiet_nan();
                const bool decided = (A > 0.f && ratio > hi) || (A < 0.f && ratio < lo);  // by the clip
                float by_lp = decided ? 0.f : -plain;
                term = -double(gain);
                if (q.ref_logprob) {
                    const float d = float(double(q.ref_logprob[r]) - lp);
                    kl = exp_less_linear(d);
                    if (q.kl_coef != 0.f) {
                        term += double(q.kl_coef) * double(kl);
                        by_lp = fmaf(-q.kl_coef, expm1f(d), by_lp);
                    }
                }
                if (q.entropy_coef != 0.f) term -= double(q.entropy_coef) * double(entropy);
                term *= double(h.weight);
                if (a.out_grad) {
                    const float g = h.weight * scale_of_grad(q.grad_scale, q.grad_scale_dev);
                    set_factors(rec, g * by_lp, -g * q.entropy_coef, entropy, float(ln_s));
                }
            }
        }
    }
    if (!write) return;
    if (a.out_logprob) a.out_logprob[r] = logprob;
    if (a.out_entropy) a.out_entropy[r] = entropy;
    if (a.out_status) a.out_status[r] = status;
    if (P.mode == kModePolicy) {
        if (P.policy.out_ratio) P.policy.out_ratio[r] = ratio;
        if (P.policy.out_kl) P.policy.out_kl[r] = kl;
        P.ws.terms[r] = term;
    }
    if (P.mode == kModePairs) {
        // the pairs' kernel takes the logprob from here and puts the gradient's factors in
        P.ws.terms[r] = double(logprob);
        P.ws.records[r] = rec;
    }
}

// Whether this block is the last of the launch to get here; what the others
// wrote before is then visible. Clears the ticket for the next launch. Called by
// every thread of a block; `flag` is a word of its shared memory.
__device__ __forceinline__ bool last_block(uint32_t* ticket, uint32_t blocks, uint32_t* flag)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const uint32_t got = atomicAdd(ticket, 1u);
        *flag = got + 1u == blocks;
        if (*flag) {
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
