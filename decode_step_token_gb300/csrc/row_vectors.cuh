// row_vectors.cuh -- rows as 16-byte vectors, for the kernels over logits rows: which
// vectors cover a row, packed fp32 operations, the elements of a vector, and the two
// passes over vectors.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "row_loss.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace rows {

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

// Two fp32 values in a register pair, and two operations in one instruction:
// both passes are bound by the number of instructions before they are by memory.
// (The pairs are kept as 64-bit values: put together for each operation they
// cost as many moves as the operations save.)
using Two = unsigned long long;

__device__ __forceinline__ Two two(float a, float b)
{
    Two y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ void split(Two x, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}

__device__ __forceinline__ Two add2(Two a, Two b)
{
    Two y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

__device__ __forceinline__ Two mul2(Two a, Two b)
{
    Two y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}

__device__ __forceinline__ Two exp2_two(Two u)
{
    float a, b;
    split(u, a, b);
    return two(exp2_fast(a), exp2_fast(b));
}

__device__ __forceinline__ Two clamp2(Two u)
{
    float a, b;
    split(u, a, b);
    return two(fmaxf(a, kLowest), fmaxf(b, kLowest));
}

template <typename T>
struct Elems;
template <>
struct Elems<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ void widen(const uint4& v, Two (&x)[2])
    {
        x[0] = two(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = two(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ float largest(const uint4& v)  // NaN where there is one
    {
        float a, b;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w)));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(b));
        return a;
    }
    static __device__ __forceinline__ uint4 round(const Two (&y)[2])
    {
        return make_uint4(uint32_t(y[0]), uint32_t(y[0] >> 32), uint32_t(y[1]), uint32_t(y[1] >> 32));
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
    static __device__ __forceinline__ void widen(const uint4& v, Two (&x)[4])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = two(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
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
    static __device__ __forceinline__ uint4 round(const Two (&y)[4])
    {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            split(y[j], a, b);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(b), "f"(a));
        }
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

// Pass 1 over N vectors. The reference moves only when one holds a larger
// element, which is rare after the first few; c is what stats_move takes.
template <typename T, bool kEntropy, int N, typename C>
__device__ __forceinline__ void fold(Stats& st, bool& bad, const uint4 (&v)[N], Two c_hi, Two c_lo, const C& c)
{
    constexpr int kPer = Elems<T>::kPer;
    float m = Elems<T>::largest(v[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) m = max_nan(m, Elems<T>::largest(v[k]));
    if (!(m <= st.ref)) {
        if (m < pos_inf())
            stats_move(st, m, c);
        else
            bad = true;
    }
    const Two ref = two(-st.ref, -st.ref);
    Two s = two(st.s, 0.f), t = two(st.t, 0.f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        Two x[kPer / 2];
        Elems<T>::widen(v[k], x);
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
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

// A row's record as pass 2 uses it.
struct Factors {
    Two ref, c, k0, k1;
};

__device__ __forceinline__ Factors factors(const RowRecord& rec)
{
    return Factors{two(-rec.ref, -rec.ref), two(rec.c, rec.c), two(rec.k0, rec.k0), two(rec.k1, rec.k1)};
}

// Pass 2 of one vector.
template <typename T, bool kEntropy>
__device__ __forceinline__ void gradient(const uint4& v, const Factors& f, Two (&y)[Elems<T>::kPer / 2])
{
    Elems<T>::widen(v, y);
#pragma unroll
    for (int j = 0; j < Elems<T>::kPer / 2; ++j) {
        Two u = mul2(add2(y[j], f.ref), f.c);
        if (kEntropy) {
            u = clamp2(u);
            y[j] = mul2(exp2_two(u), fma2(f.k1, u, f.k0));
        } else {
            y[j] = mul2(exp2_two(u), f.k0);
        }
    }
}

template <typename T, bool kEntropy>
__device__ __forceinline__ uint4 gradient(const uint4& v, const Factors& f)
{
    Two y[Elems<T>::kPer / 2];
    gradient<T, kEntropy>(v, f, y);
    return Elems<T>::round(y);
}

// The same with the token at place `at` of the vector (kPer or more, or below 0: not in it).
template <typename T, bool kEntropy>
__device__ __forceinline__ uint4 gradient_token(const uint4& v, const Factors& f, int at, float at_token)
{
    Two y[Elems<T>::kPer / 2];
    gradient<T, kEntropy>(v, f, y);
#pragma unroll
    for (int j = 0; j < Elems<T>::kPer / 2; ++j) {
        float a, b;
        split(y[j], a, b);
        y[j] = two(2 * j == at ? a + at_token : a, 2 * j + 1 == at ? b + at_token : b);
    }
    return Elems<T>::round(y);
}

// Store vector `i` of a row's span to the gradient: as one where it lies wholly
// inside the row and the gradient's vectors lie as the logits' do (`whole`), else
// by element.
template <typename T>
__device__ __forceinline__ void put_vector(T* g, int vocab, int head, int i, bool whole, const uint4& y)
{
    constexpr int kPer = Elems<T>::kPer;
    const int first = i * kPer - head;
    if (whole && first >= 0 && first + kPer <= vocab) {
        __stcs(reinterpret_cast<uint4*>(g + first), y);
    } else {
        const T* e = reinterpret_cast<const T*>(&y);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (first + j >= 0 && first + j < vocab) g[first + j] = e[j];
    }
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

// A whole warp waits for the phase of `bar` with the given parity, for `ns` at
// most; all of its lanes get the same answer.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, uint64_t ns)
{
    return mbar_wait_warp(bar, parity, now_ns() + ns);
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint64_t ns)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_slow(bar, parity, ns);
}

}  // namespace rows
}  // namespace dst
