// scaled_head_kernel.cu -- the LM head in 8 bits on the fifth-generation tensor
// cores: logits[i, v] = sum over blocks b of 128 of hidden_scale[i, b] *
// weight_scale[v / 128, b] * (the block's product of e4m3 values).
//
// A scale belongs to one block of K, so the products of a block are summed by
// the tensor cores (fp32, in tensor memory) and the blocks by the epilogue's
// threads, in fp32 registers: sum += scale * product. One block of K is one
// stage of the operand ring (128 bytes: one swizzled row) and one accumulator
// of tensor memory; there are two accumulators, so that the tensor cores fill
// one while the threads empty the other.
//
// The product is taken transposed: a tile is 128 weight rows (M: one block of
// the weight's scales, so that scale is one number for a tile and block) by NT
// hidden rows (N, at most 256). It suits a decode step of a few rows, where the
// weight's bytes are all the time, and a prompt, and its lanes are neighbouring
// tokens of the vocabulary, so that the logits are stored as they lie.
//
// Persistent, one CTA an SM; warp roles:
//   warps 0-7  the epilogue: two groups of four warps, each a half of the tile's
//              columns (hidden rows), a warp 32 of its lanes (weight rows);
//   warp 8     one thread issues the TMA loads of the operand ring;
//   warp 9     owns the tensor memory, and one thread issues the MMAs.
// Warps 10 and 11 fill up the third warpgroup, which gives its registers to the
// epilogue's (a thread there holds up to 128 sums).
// Every wait is bounded in time; a CTA whose wait gives up counts itself in the
// handle's statistics and leaves its logits unwritten.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "launch.h"
#include "ptx.cuh"

namespace dst {
namespace scaled {

constexpr int kBM = 128;                       // weight rows of a tile: MMA M, and a block of scales
constexpr int kBK = 128;                       // K of a stage: a block of scales, one 128-byte swizzled row
constexpr int kUK = 32;                        // K of one tcgen05.mma of 8-bit operands
constexpr int kThreads = 384;
constexpr int kFewRegs = 40, kManyRegs = 224;  // 128 * 40 + 256 * 224 <= 384 * 168
constexpr int kGroupThreads = 128;             // of one half of the columns
constexpr int kMaxStages = 8;
constexpr int kMaxRows = 256;                  // hidden rows of a tile: MMA N
constexpr int kScaleBlocks = 4;                // blocks of K whose scales are fetched together
constexpr uint32_t kABytes = kBM * kBK;        // 16 KB a stage
constexpr uint64_t kWaitNs = 2000000000ull;    // a wait gives up after 2 s
constexpr size_t kScaleBytes = 2 * kScaleBlocks * kMaxRows * 4;  // two buffers of scales for every column
constexpr size_t kBarBytes = 256;
constexpr size_t kSmemMax = 227 * 1024;

struct Params {
    CUtensorMap tw;      // weight [V, K]: box 128 x 128, 128-byte swizzle
    CUtensorMap th;      // hidden [rows, K]: box 128 x NT
    const float* hidden_scale;
    const float* weight_scale;
    int64_t hidden_scale_stride, weight_scale_stride;
    void* logits;
    int64_t ldl;
    int rows, V, NT;
    int row_tiles, tiles;  // tiles of hidden rows; of both
    int blocks;            // of K
    int stages;
    uint32_t tmem_cols;    // a power of two >= 2 * NT
    int wide_scales;       // the hidden scales can be read four at a time
    unsigned long long* timeouts;
};

// K-major tile in the 128-byte swizzled layout that the TMA engine writes: 8-row
// atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr)
{
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// kind::f8f6f4, fp32 accumulator, e4m3 A and B (type 0 each), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
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

// The registers of the loads before it are passed through, so that nothing that
// uses them is moved ahead of the wait.
__device__ __forceinline__ void tmem_wait(uint32_t* r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// (a, b) += (x, y) * (p, q), two fp32 operations in one.
__device__ __forceinline__ void fma2(float2& a, uint32_t x, uint32_t y, float p, float q)
{
    asm("{\n\t.reg .b64 s, t, u;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%4, %5};\n\t"
        "fma.rn.f32x2 s, t, u, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "r"(x), "r"(y), "f"(p), "f"(q));
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase of `bar` with the given parity, for kWaitNs at most.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity)
{
    uint64_t until = 0;
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u) {
            const uint64_t now = now_ns();
            if (until == 0) until = now + kWaitNs;
            if (now > until) return false;
        }
    }
    return false;
}

__device__ __forceinline__ void arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void group_sync(int group)
{
    if (group == 0)
        asm volatile("bar.sync 1, %0;" ::"n"(kGroupThreads) : "memory");
    else
        asm volatile("bar.sync 2, %0;" ::"n"(kGroupThreads) : "memory");
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// kCols: columns of a tile that a thread of the epilogue holds, at least NT / 2.
template <typename T, int kCols>
__global__ void __launch_bounds__(kThreads, 1) head_kernel(const __grid_constant__ Params P)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int S = P.stages;
    const uint32_t b_bytes = uint32_t(P.NT) * kBK;
    unsigned char* sa = smem;
    unsigned char* sb = smem + size_t(S) * kABytes;
    float* scales = reinterpret_cast<float*>(sb + size_t(S) * b_bytes);  // [2][kScaleBlocks][kMaxRows]
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + 2 * kScaleBlocks * kMaxRows);
    uint64_t* empty = full + kMaxStages;
    uint64_t* tfull = empty + kMaxStages;  // [2] an accumulator is complete
    uint64_t* tempty = tfull + 2;          // [2] an accumulator has been read
    uint64_t* drained = tempty + 2;        // every MMA of the CTA has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    int* gave_up = reinterpret_cast<int*>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 8);
        }
        mbar_init(drained, 1);
        *gave_up = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tw)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.th)) : "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(P.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int G = int(gridDim.x), first = int(blockIdx.x);

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 8) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; ok && t < P.tiles; t += G) {
                const int v0 = t / P.row_tiles * kBM, r0 = t % P.row_tiles * P.NT;
                for (int b = 0; b < P.blocks; ++b, ++it) {
                    const uint32_t s = it % S;
                    ok = wait(&empty[s], (it / S & 1u) ^ 1u);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&full[s], kABytes + b_bytes);
                    tma_load_2d(smem_addr(sa + s * kABytes), &P.tw, b * kBK, v0, smem_addr(&full[s]));
                    tma_load_2d(smem_addr(sb + s * b_bytes), &P.th, b * kBK, r0, smem_addr(&full[s]));
                }
            }
            if (!ok) *gave_up = 1;
            // the last copies issued land before the CTA may exit
            for (uint32_t j = it > uint32_t(S) ? it - S : 0; j < it; ++j) wait(&full[j % S], j / S & 1u);
        }
    } else if (warp == 9) {
        if (lane == 0) {
            const uint32_t idesc = idesc_e4m3(kBM, P.NT);
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; ok && t < P.tiles; t += G) {
                for (int b = 0; b < P.blocks; ++b, ++it) {
                    const uint32_t s = it % S, acc = it & 1u;
                    ok = wait(&tempty[acc], (it >> 1 & 1u) ^ 1u) && wait(&full[s], it / S & 1u);
                    if (!ok) break;
                    fence_after_sync();
                    const uint32_t d = tmem + acc * uint32_t(P.NT);
                    const uint64_t da = desc_sw128(smem_addr(sa + s * kABytes));
                    const uint64_t db = desc_sw128(smem_addr(sb + s * b_bytes));
#pragma unroll
                    for (int k = 0; k < kBK / kUK; ++k)  // +32 bytes inside the 128-byte rows
                        mma_e4m3(d, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc, uint32_t(k));
                    mma_commit(&empty[s]);
                    mma_commit(&tfull[acc]);
                }
            }
            if (!ok) *gave_up = 1;
            mma_commit(drained);
            wait(drained, 0);
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int group = warp >> 2, quarter = warp & 3;  // quarter: the tensor-memory lanes a warp may read
        const int j = quarter * 32 + lane;                      // thread of the group: its column's scales
        const int half = ((P.NT >> 1) + 15) & ~15;
        const int c0 = group * half, cols = max(0, min(half, P.NT - c0));
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(c0);
        uint32_t it = 0, fetched = 0;
        bool ok = true;
        for (int t = first; t < P.tiles; t += G) {  // to the end even where a wait gave up: its group's barriers count on it
            const int vb = t / P.row_tiles, v = vb * kBM + quarter * 32 + lane, r0 = t % P.row_tiles * P.NT;
            const float* sw = P.weight_scale + vb * P.weight_scale_stride;
            const bool has = j < cols && r0 + c0 + j < P.rows;
            const float* sh = P.hidden_scale + int64_t(r0 + c0 + j) * P.hidden_scale_stride;
            // the scales of blocks b .. b + 3 of this thread's column, times the weight's
            float next[kScaleBlocks];
            auto fetch = [&](int b) {
                if (has && P.wide_scales && b + kScaleBlocks <= P.blocks) {
                    const float4 q = *reinterpret_cast<const float4*>(sh + b);
                    next[0] = q.x * sw[b];
                    next[1] = q.y * sw[b + 1];
                    next[2] = q.z * sw[b + 2];
                    next[3] = q.w * sw[b + 3];
                } else {
#pragma unroll
                    for (int i = 0; i < kScaleBlocks; ++i) next[i] = has && b + i < P.blocks ? sh[b + i] * sw[b + i] : 0.f;
                }
            };
            fetch(0);
            float2 sum[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = make_float2(0.f, 0.f);
            for (int b = 0; b < P.blocks; ++b, ++it) {
                float* row = scales + (fetched & 1u) * (kScaleBlocks * kMaxRows) + group * (kMaxRows / 2);
                if (b % kScaleBlocks == 0) {
                    // the other buffer of scales is free: all have come to this barrier after their last use of it
                    ++fetched;
                    row = scales + (fetched & 1u) * (kScaleBlocks * kMaxRows) + group * (kMaxRows / 2);
#pragma unroll
                    for (int i = 0; i < kScaleBlocks; ++i) row[i * kMaxRows + j] = next[i];
                    group_sync(group);
                    if (b + kScaleBlocks < P.blocks) fetch(b + kScaleBlocks);
                }
                row += b % kScaleBlocks * kMaxRows;
                const uint32_t acc = it & 1u;
                ok = ok && wait(&tfull[acc], it >> 1 & 1u);
                if (ok) {
                    fence_after_sync();
                    const uint32_t at = lanes + acc * uint32_t(P.NT);
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
                        uint32_t r[32];
                        if (c < cols) {
                            tmem_ld16(at + c, r);
                            if (kCols > 16 && c + 16 < cols) tmem_ld16(at + c + 16, r + 16);
                            tmem_wait(r);
#pragma unroll
                            for (int i = 0; i < 32 && i < kCols; i += 4) {
                                const float4 s = *reinterpret_cast<const float4*>(row + c + i);
                                fma2(sum[(c + i) / 2], r[i], r[i + 1], s.x, s.y);
                                fma2(sum[(c + i) / 2 + 1], r[i + 2], r[i + 3], s.z, s.w);
                            }
                        }
                    }
                    fence_before_sync();
                }
                __syncwarp();
                if (ok && lane == 0) arrive(&tempty[acc]);
            }
            if (ok && v < P.V) {
                T* out = static_cast<T*>(P.logits) + int64_t(r0 + c0) * P.ldl + v;
                const int n = min(cols, P.rows - r0 - c0);
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if (c < n) put(out + int64_t(c) * P.ldl, c & 1 ? sum[c / 2].y : sum[c / 2].x);
            }
        }
        if (!ok && lane == 0) *gave_up = 1;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
    if (tid == 0 && *gave_up && P.timeouts) atomicAdd(P.timeouts, 1ull);
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder()
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

// Tensor map over rows x cols bytes, box 128 x box_rows; bytes outside read as zero.
bool encode(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld)};
    const cuuint32_t box[2] = {cuuint32_t(kBK), cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Kernel = void (*)(const Params);

template <typename T>
Kernel kernel_for(int NT)
{
    return NT <= 32 ? head_kernel<T, 16> : NT <= 64 ? head_kernel<T, 32> : NT <= 128 ? head_kernel<T, 64> : head_kernel<T, 128>;
}

}  // namespace scaled

int scaled_head_launch(const sampler_scaled_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows,
                       int64_t vocab, int sms, unsigned long long* timeouts, cudaStream_t stream)
{
    using namespace scaled;
    Params p;
    std::memset(&p, 0, sizeof p);
    const int64_t row_tiles = (rows + kMaxRows - 1) / kMaxRows;
    p.row_tiles = int(row_tiles);
    p.NT = int(((rows + row_tiles - 1) / row_tiles + 15) / 16 * 16);
    const int64_t tiles = (vocab + kBM - 1) / kBM * row_tiles;
    if (tiles > INT32_MAX - 65536) return SAMPLER_ERR_TOO_LARGE;
    p.tiles = int(tiles);
    p.blocks = int((g.hidden_dim + kBK - 1) / kBK);
    const size_t stage = kABytes + size_t(p.NT) * kBK;
    p.stages = int(std::min<size_t>(kMaxStages, (kSmemMax - 1024 - kBarBytes - kScaleBytes) / stage));
    p.tmem_cols = 32;
    while (p.tmem_cols < uint32_t(2 * p.NT)) p.tmem_cols <<= 1;
    if (!encode(&p.tw, g.weight, vocab, g.hidden_dim, g.weight_stride, kBM) ||
        !encode(&p.th, g.hidden, rows, g.hidden_dim, g.hidden_stride, p.NT))
        return SAMPLER_ERR_CUDA;
    p.hidden_scale = g.hidden_scale;
    p.weight_scale = g.weight_scale;
    p.hidden_scale_stride = g.hidden_scale_stride;
    p.weight_scale_stride = g.weight_scale_stride;
    p.wide_scales = g.hidden_scale_stride % 4 == 0 && reinterpret_cast<uintptr_t>(g.hidden_scale) % 16 == 0;
    p.logits = logits;
    p.ldl = ldl;
    p.rows = int(rows);
    p.V = int(vocab);
    p.timeouts = timeouts;
    const Kernel kernel = dtype == SAMPLER_DTYPE_BF16 ? kernel_for<uint16_t>(p.NT) : kernel_for<float>(p.NT);
    const size_t smem = 1024 + size_t(p.stages) * stage + kScaleBytes + kBarBytes;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(smem)) != cudaSuccess)
        return SAMPLER_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min(sms, p.tiles)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
