// quantize_kernel.cu -- rows to e4m3 with one fp32 scale for each block of
// 128 columns by 1 or 128 rows: scale = m / 448 and value = e4m3(x * (448 / m))
// for the block's largest magnitude m.
//
// One block of 128 threads takes one block of values, a thread a column: a pass
// for the largest magnitude, a pass that rounds.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"

namespace dst {
namespace quant {

constexpr float kMost = 448.f;               // the largest e4m3 value
constexpr float kLeast = 7.888609052e-31f;   // 2^-100: keeps 448 / m finite and m / 448 normal

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }

template <typename T>
__global__ void __launch_bounds__(128) quantize_kernel(const sampler_quantize_t q, int64_t blocks, int across)
{
    __shared__ float part[4];
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t br = b / across, bc = b % across;
        const int64_t r0 = br * q.block_rows, r1 = min(r0 + q.block_rows, q.rows);
        const int64_t c = bc * 128 + threadIdx.x;
        float m = 0.f;
        if (c < q.cols)
            for (int64_t r = r0; r < r1; ++r) {
                const float v = fabsf(load(static_cast<const T*>(q.src) + r * q.src_stride + c));
                m = v <= m ? m : v;  // a NaN is taken over ...
                if (!(v <= 3.402823466e38f)) m = __int_as_float(0x7f800000);  // ... as an infinity
            }
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
        const bool bad = isinf(m);
        m = fmaxf(m, kLeast);
        const float inv = bad ? 0.f : __fdiv_rn(kMost, m);
        if (c < q.cols)
            for (int64_t r = r0; r < r1; ++r) {
                const float v = load(static_cast<const T*>(q.src) + r * q.src_stride + c);
                static_cast<uint8_t*>(q.values)[r * q.values_stride + c] =
                    bad ? uint8_t(0) : __nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
            }
        if (threadIdx.x == 0)
            q.scales[br * q.scale_stride + bc] = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(m, kMost);
    }
}

}  // namespace quant

int quantize_launch(const sampler_quantize_t& q, int sms, cudaStream_t stream)
{
    const int across = int((q.cols + 127) / 128);
    const int64_t blocks = (q.rows + q.block_rows - 1) / q.block_rows * across;
    const unsigned grid = unsigned(std::min<int64_t>(blocks, int64_t(sms) * 16));
    if (q.dtype == SAMPLER_DTYPE_BF16)
        quant::quantize_kernel<uint16_t><<<grid, 128, 0, stream>>>(q, blocks, across);
    else
        quant::quantize_kernel<float><<<grid, 128, 0, stream>>>(q, blocks, across);
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
