// tensor_core.cuh -- what the LM heads in 8 and 4 bits share: TMA loads and stores of
// tiles, tensor memory, the operands' descriptors, and the encoder of tensor maps. (The
// bf16 head has its own. The stores of a warp's logits are the 4-bit head's: the 8-bit
// one writes the same steps out, as calling them spills registers of its fp32 form.)
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "ptx.cuh"
#include "sampler.h"

namespace dst {

// K-major tile in the 128-byte swizzled layout that the TMA engine writes: 8-row
// atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr)
{
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 consecutive columns of this thread's tensor-memory lane; complete after tmem_wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Passes 16 loaded registers through, after tmem_wait: what uses them is not moved ahead of it.
__device__ __forceinline__ void tmem_take16(uint32_t* r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

constexpr uint32_t kBoxBytes = 32 * 128;  // a box of logits: 32 rows of 128 bytes, swizzled

// A warp stores its part of a tile of logits: a row from `row` on in each lane, kCols columns from v on, by way of its
// box in shared memory to the TMA engine where that can write them (P.tma_stores), else from the box by element. P: a
// kernel's parameters, which have to and tma_stores, logits, ldl, rows and V.
template <typename T, int kCols, typename Params>
__device__ __forceinline__ void store_logits(const Params& P, unsigned char* out, int row, int v,
                                             const float2 (&sum)[kCols / 2])
{
    constexpr int kBoxCols = 128 / int(sizeof(T));
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c0 = 0; c0 < kCols; c0 += kBoxCols) {
        if (P.tma_stores) {  // the box before has left the buffer
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // 16 bytes each, at their swizzled place in the lane's row
            const float2* x = sum + (c0 + i * kBoxCols / 8) / 2;
            const uint4 w = sizeof(T) == 2 ? make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y),
                                                        pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y))
                                           : make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y),
                                                        __float_as_uint(x[1].x), __float_as_uint(x[1].y));
            *reinterpret_cast<uint4*>(out + lane * 128 + (i ^ (lane & 7)) * 16) = w;
        }
        // the TMA engine ends a row at a multiple of 16 bytes: the last tile may have to be stored otherwise
        if (P.tma_stores && (v + kCols <= P.V || P.V % (kBoxCols / 8) == 0)) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                if (row < P.rows && v + c0 < P.V) tma_store_2d(&P.to, v + c0, row, smem_addr(out));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        } else {
            __syncwarp();
            // eight rows' elements under way at once (one: 333 x 20011 x 1000 fp32 26.1 us, so 18.7
            // from inputs in L2, 20.2 from others; two bf16 columns a lane on their 4-byte boundaries: 28 us
            // where this takes 16.6, for the branches)
            const int n = min(32, P.rows - row), cols = min(kBoxCols, P.V - v - c0);
            T* g = static_cast<T*>(P.logits) + int64_t(row) * P.ldl + v + c0;
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
#pragma unroll
                for (int c = lane; c < kBoxCols; c += 32)
                    if (k < n && c < cols)
                        g[c] = *reinterpret_cast<const T*>(out + k * 128 + (c * int(sizeof(T)) ^ (k & 7) * 16));
                g += P.ldl;
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- host side
inline PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Tensor map of the logits: boxes of 128 bytes x 32 rows, a warp's part of a tile.
inline bool encode_logits(CUtensorMap* map, void* base, int dtype, int64_t rows, int64_t cols, int64_t ld)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return false;
    const bool bf16 = dtype == SAMPLER_DTYPE_BF16;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * (bf16 ? 2u : 4u)};
    const cuuint32_t box[2] = {bf16 ? 64u : 32u, 32u};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over rows x cols bytes, box 128 x box_rows; bytes outside read as zero.
inline bool encode_bytes(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld)};
    const cuuint32_t box[2] = {128u, cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dst
