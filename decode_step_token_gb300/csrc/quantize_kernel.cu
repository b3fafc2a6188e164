// quantize_kernel.cu -- rows to e4m3 with one fp32 scale for each block of
// 128 columns by 1 or 128 rows: scale = m / 448 and value = e4m3(x * (448 / m))
// for the block's largest magnitude m.
//
// A block's values have to be known before any of them can be rounded, so they
// are kept in registers between the two: one pass over memory. 256 threads take
// 128 columns, a row in 16 (bf16) or 32 (fp32) neighbouring lanes with one
// 16-byte load each; a thread has up to kPasses rows. Blocks of one row need a
// shuffle among those lanes, blocks of 128 rows the whole thread block.
// Magnitudes are compared as the integers of their bits, in which an infinity
// and a NaN are the largest.
// Measured: a weight of 128000 x 4096 bf16 in blocks of 128 x 128 in 226 us, 6.9
// TB/s (the copy rate); 64 hidden rows of 4096 in 1.9 us, which is the launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"

namespace dst {
namespace quant {

constexpr float kMost = 448.f;               // the largest e4m3 value
constexpr float kLeast = 7.888609052e-31f;   // 2^-100: keeps 448 / m finite and m / 448 normal
constexpr int kThreads = 256;

// Two values to two e4m3 codes, rounded to nearest even.
__device__ __forceinline__ uint32_t codes2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

struct Scale {
    float inv, scale;
    uint32_t keep;  // mask of the codes: 0 where the block has a NaN or an infinity
};

template <typename T>
struct Elems;
template <>
struct Elems<uint16_t> {
    static constexpr int kPer = 8;
    // the largest magnitude of a vector, as fp32 bits
    static __device__ __forceinline__ uint32_t largest(const uint4& v)
    {
        uint32_t a, b;
        const uint32_t k = 0x7fff7fffu;
        asm("max.u16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x & k), "r"(v.y & k));
        asm("max.u16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z & k), "r"(v.w & k));
        asm("max.u16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return max(a & 0xffff0000u, a << 16);
    }
    static __device__ __forceinline__ void put(uint8_t* to, const uint4& v, const Scale& s, int count, bool whole)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q[j] = codes2(__uint_as_float(w[j] << 16) * s.inv, __uint_as_float(w[j] & 0xffff0000u) * s.inv) & s.keep;
        if (whole)
            __stcs(reinterpret_cast<uint2*>(to), make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16));
        else
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < count) to[j] = uint8_t(q[j / 2] >> 8 * (j & 1));
    }
};
template <>
struct Elems<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ uint32_t largest(const uint4& v)
    {
        const uint32_t k = 0x7fffffffu;
        return max(max(v.x & k, v.y & k), max(v.z & k, v.w & k));
    }
    static __device__ __forceinline__ void put(uint8_t* to, const uint4& v, const Scale& s, int count, bool whole)
    {
        const uint32_t q = (codes2(__uint_as_float(v.x) * s.inv, __uint_as_float(v.y) * s.inv) |
                            codes2(__uint_as_float(v.z) * s.inv, __uint_as_float(v.w) * s.inv) << 16) &
                           s.keep;
        if (whole)
            __stcs(reinterpret_cast<uint32_t*>(to), q);
        else
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < count) to[j] = uint8_t(q >> 8 * j);
    }
};

// From the bits of a block's largest magnitude.
__device__ __forceinline__ Scale scale_of(uint32_t most)
{
    Scale s;
    if (most >= 0x7f800000u) {
        s.inv = 0.f;
        s.scale = __int_as_float(0x7fc00000);
        s.keep = 0u;
    } else {
        const float m = fmaxf(__uint_as_float(most), kLeast);
        s.inv = __fdiv_rn(kMost, m);
        s.scale = __fdiv_rn(m, kMost);
        s.keep = 0xffffffffu;
    }
    return s;
}

// kSquare: blocks of 128 x 128, one to a thread block; else blocks of 1 x 128.
// vec_in, vec_out: the rows of either matrix lie so that whole vectors can be
// moved.
template <typename T, int kPasses, bool kSquare>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const sampler_quantize_t q, bool vec_in, bool vec_out)
{
    constexpr int kPer = Elems<T>::kPer;
    constexpr int kLanes = 128 / kPer;           // of a row
    constexpr int kRows = kThreads / kLanes;     // of a pass
    const int lane = threadIdx.x & 31;
    const int64_t row0 = int64_t(blockIdx.y) * (kRows * kPasses) + threadIdx.x / kLanes;
    const int64_t col = int64_t(blockIdx.x) * 128 + threadIdx.x % kLanes * kPer;
    const int count = int(max(int64_t(0), min(int64_t(kPer), q.cols - col)));  // of this thread's vector
    const T* src = static_cast<const T*>(q.src) + row0 * q.src_stride + col;
    uint4 v[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (row0 + k * kRows < q.rows) {
            const T* p = src + int64_t(k) * kRows * q.src_stride;
            if (vec_in && count == kPer) {
                v[k] = __ldcs(reinterpret_cast<const uint4*>(p));
            } else {
                T* e = reinterpret_cast<T*>(&v[k]);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j < count) e[j] = p[j];
            }
        }
    }
    uint32_t most[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) most[k] = Elems<T>::largest(v[k]);
    uint8_t* to = static_cast<uint8_t*>(q.values) + row0 * q.values_stride + col;
    const bool whole = vec_out && count == kPer;
    if (kSquare) {
        __shared__ uint32_t part[kThreads / 32];
        uint32_t m = most[0];
#pragma unroll
        for (int k = 1; k < kPasses; ++k) m = max(m, most[k]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, part[w]);
        const Scale s = scale_of(m);
        if (threadIdx.x == 0) q.scales[int64_t(blockIdx.y) * q.scale_stride + blockIdx.x] = s.scale;
#pragma unroll
        for (int k = 0; k < kPasses; ++k)
            if (row0 + k * kRows < q.rows)
                Elems<T>::put(to + int64_t(k) * kRows * q.values_stride, v[k], s, count, whole);
    } else {
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) most[k] = max(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
            const Scale s = scale_of(most[k]);
            const int64_t row = row0 + k * kRows;
            if (row < q.rows) {
                Elems<T>::put(to + int64_t(k) * kRows * q.values_stride, v[k], s, count, whole);
                if (threadIdx.x % kLanes == 0) q.scales[row * q.scale_stride + blockIdx.x] = s.scale;
            }
        }
    }
}

template <typename T>
bool launch(sampler_quantize_t q, int sms, cudaStream_t stream)
{
    constexpr int kRows = kThreads * Elems<T>::kPer / 128;
    constexpr int kMany = 64 / kRows;  // passes of blocks of one row where there are many: 64 rows
    constexpr int kAll = 128 / kRows;
    const bool vec_in = reinterpret_cast<uintptr_t>(q.src) % 16 == 0 && q.src_stride * int64_t(sizeof(T)) % 16 == 0;
    const bool vec_out = reinterpret_cast<uintptr_t>(q.values) % Elems<T>::kPer == 0 && q.values_stride % Elems<T>::kPer == 0;
    const int64_t across = (q.cols + 127) / 128;
    const bool square = q.block_rows == 128;
    // one row a thread up to so many blocks of threads for each SM, for its latency; else several loads in flight. One
    // row / several, from inputs not in L2: bf16 x 4096 64 rows 2.5 / 3.4 us, 600 3.7 / 4.7, 1200 5.5 / 5.9, 2400 9.2 /
    // 9.2 (4800 blocks, 32 an SM), 3600 12.8 / 11.9, 8192 25.6 / 23.3; x 16384 300 rows 5.6 / 6.2, 600 9.2 / 9.2 (4864),
    // 1200 15.9 / 14.7; fp32 x 4096 600 rows 5.1 / 6.3, 2400 13.9 / 15.1, 3600 19.9 / 20.3 (14400 blocks, 95 an SM),
    // 4800 25.4 / 24.9; x 16384 900 rows 19.9 / 20.7 (14464), 1800 36.6 / 34.5
    constexpr int kFewBlocks = sizeof(T) == 2 ? 32 : 96;
    const bool few = !square && (q.rows + kRows - 1) / kRows * across <= int64_t(sms) * kFewBlocks;
    const int rows = square ? 128 : few ? kRows : 64;
    // the grid's second dimension is limited: taller matrices go in several launches
    const int64_t most = 65535LL * rows;
    const char* src = static_cast<const char*>(q.src);
    uint8_t* values = static_cast<uint8_t*>(q.values);
    float* scales = q.scales;
    const int64_t all = q.rows;
    for (int64_t done = 0; done < all; done += most) {
        q.rows = std::min(all - done, most);
        q.src = src + done * q.src_stride * int64_t(sizeof(T));
        q.values = values + done * q.values_stride;
        q.scales = scales + done / q.block_rows * q.scale_stride;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(across), unsigned((q.rows + rows - 1) / rows));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        const auto kernel = square ? quantize_kernel<T, kAll, true>
                            : few  ? quantize_kernel<T, 1, false>
                                   : quantize_kernel<T, kMany, false>;
        // (the launch's own status: cudaGetLastError would also report what an earlier call has left)
        if (cudaLaunchKernelEx(&cfg, kernel, q, vec_in, vec_out) != cudaSuccess) return false;
    }
    return true;
}

}  // namespace quant

int quantize_launch(const sampler_quantize_t& q, int sms, cudaStream_t stream)
{
    const bool ok = q.dtype == SAMPLER_DTYPE_BF16 ? quant::launch<uint16_t>(q, sms, stream) : quant::launch<float>(q, sms, stream);
    return ok ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
