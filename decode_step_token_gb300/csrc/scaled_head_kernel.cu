// scaled_head_kernel.cu -- the LM head in 8 bits: logits[i, v] = sum over blocks
// b of 128 of hidden_scale[i, b] * weight_scale[v / 128, b] * the block's product
// of e4m3 values, in fp32.
//
// One block of 256 threads takes a tile of 64 rows by 64 tokens, a thread 4 x 4
// of it, with the block's values widened to fp32 in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "launch.h"

namespace dst {
namespace scaled {

constexpr int kTile = 64;
constexpr int kStep = 32;

__device__ __forceinline__ float widen(uint8_t v)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <typename T>
__global__ void __launch_bounds__(256) head_kernel(const sampler_scaled_head_t g, T* logits, int64_t ldl, int64_t rows,
                                                   int64_t vocab)
{
    __shared__ float h[kStep][kTile + 1], w[kStep][kTile + 1];
    const int64_t row0 = int64_t(blockIdx.y) * kTile, v0 = int64_t(blockIdx.x) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float sum[4][4] = {}, part[4][4] = {};
    for (int64_t k0 = 0; k0 < g.hidden_dim; k0 += kStep) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int k = i % kStep, r = i / kStep;
            const bool in = k0 + k < g.hidden_dim;
            h[k][r] = in && row0 + r < rows
                          ? widen(static_cast<const uint8_t*>(g.hidden)[(row0 + r) * g.hidden_stride + k0 + k])
                          : 0.f;
            w[k][r] = in && v0 + r < vocab
                          ? widen(static_cast<const uint8_t*>(g.weight)[(v0 + r) * g.weight_stride + k0 + k])
                          : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(h[k][ty * 4 + i], w[k][tx + 16 * j], part[i][j]);
        if (k0 % 128 == 128 - kStep || k0 + kStep >= g.hidden_dim) {
            const int64_t b = k0 / 128;
            for (int i = 0; i < 4; ++i) {
                const int64_t r = row0 + ty * 4 + i;
                const float sh = r < rows ? g.hidden_scale[r * g.hidden_scale_stride + b] : 0.f;
                for (int j = 0; j < 4; ++j) {
                    const int64_t v = v0 + tx + 16 * j;
                    const float sw = v < vocab ? g.weight_scale[v / 128 * g.weight_scale_stride + b] : 0.f;
                    sum[i][j] = fmaf(part[i][j], sh * sw, sum[i][j]);
                    part[i][j] = 0.f;
                }
            }
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = row0 + ty * 4 + i, v = v0 + tx + 16 * j;
            if (r < rows && v < vocab) put(logits + r * ldl + v, sum[i][j]);
        }
}

}  // namespace scaled

int scaled_head_launch(const sampler_scaled_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows,
                       int64_t vocab, int, unsigned long long*, cudaStream_t stream)
{
    const int64_t up = (rows + scaled::kTile - 1) / scaled::kTile;
    if (up > 65535) return SAMPLER_ERR_TOO_LARGE;
    const dim3 grid(unsigned((vocab + scaled::kTile - 1) / scaled::kTile), unsigned(up));
    if (dtype == SAMPLER_DTYPE_BF16)
        scaled::head_kernel<<<grid, 256, 0, stream>>>(g, static_cast<uint16_t*>(logits), ldl, rows, vocab);
    else
        scaled::head_kernel<<<grid, 256, 0, stream>>>(g, static_cast<float*>(logits), ldl, rows, vocab);
    return cudaGetLastError() == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
