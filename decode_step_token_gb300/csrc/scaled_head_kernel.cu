// scaled_head_kernel.cu -- the LM head in 8 bits on the fifth-generation tensor
// cores: logits[i, v] = sum over blocks b of 128 of hidden_scale[i, b] *
// weight_scale[v / 128, b] * (the block's product of e4m3 values).
//
// A scale belongs to one block of K, so the products of a block are summed by
// the tensor cores (fp32, in tensor memory) and the blocks by the epilogue's
// threads, in fp32 registers: sum += scale * product. One block of K is one
// stage of the operand ring (128 bytes: one swizzled row) and one accumulator
// of tensor memory; there are two accumulators or more, so that the tensor cores
// fill one while the threads empty another.
//
// Few rows (a decode step; up to kFewRows) are taken transposed: a tile is 128
// weight rows (M: one block of the weight's scales, so that scale is one number
// for a tile and block) by all hidden rows (N). The weight's bytes are all the
// time then. A column's scale is the same for all lanes and comes from shared
// memory; the accumulators are up to eight, and the lanes are neighbouring
// tokens of the vocabulary, so that the logits are stored as they lie.
//
// Many rows (a prompt) are taken as they are, by pairs of CTAs: a tile is 256
// hidden rows (M, 128 in each CTA) by 256 weight rows (N, 128 of them in each
// CTA's shared memory, which the pair's tensor cores read both of). So a block of
// a tile costs a CTA 32 KB of loads; alone it would cost 48 KB, and the loads
// from L2 and not the tensor cores would be the time (measured at 4096 x 64000 x
// 4096: 15 to 17 TB/s with 48 KB, whatever else was left out). The tensor cores
// take 512 cycles for a block, in which its 32768 products of each CTA have to be
// scaled: a lane is a hidden row here, so its scale is one register, two products
// are one instruction, and nothing is read from shared memory. The logits go
// through shared memory once, to be stored by row.
//
// Persistent, one CTA an SM; warp roles:
//   warps 0-7  the epilogue: two groups of four warps, each a half of the tile's
//              columns, a warp 32 of its lanes;
//   warp 8     issues the TMA loads of the operand ring;
//   warp 9     owns the tensor memory and issues the MMAs (of a pair: the first
//              CTA's).
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

constexpr int kBM = 128;                       // MMA M, and a block of the weight's scales
constexpr int kBK = 128;                       // K of a stage: a block of scales, one 128-byte swizzled row
constexpr int kUK = 32;                        // K of one tcgen05.mma of 8-bit operands
constexpr int kThreads = 384;
constexpr int kFewRegs = 40, kManyRegs = 224;  // 128 * 40 + 256 * 224 <= 384 * 168
constexpr int kGroupThreads = 128;             // of one half of the columns
constexpr int kMaxStages = 8;
constexpr int kMaxAccs = 8;
constexpr int kTmemCols = 512;
constexpr int kFewRows = 128;                  // the most that are taken transposed
constexpr int kWideN = 256;                    // weight rows of a tile of many hidden rows
constexpr int kScaleBlocks = 4;                // blocks of K whose scales are fetched together
constexpr uint32_t kABytes = kBM * kBK;        // 16 KB a stage
constexpr uint64_t kWaitNs = 2000000000ull;    // a wait gives up after 2 s
constexpr size_t kScaleBytes = 2 * kScaleBlocks * kFewRows * 4;  // transposed: two buffers of every column's scales
constexpr int kRowBytes = 64, kRowPitch = 80;  // many rows: a piece of a row on its way out; 80: no bank conflicts
constexpr size_t kOutBytes = 8 * 32 * kRowPitch;
constexpr size_t kBarBytes = 512;
constexpr size_t kSmemMax = 227 * 1024;

struct Params {
    CUtensorMap tm, tn;  // the operands of M and N [rows, K], 128-byte swizzle: boxes of 128 bytes by 128 and NT
                         // rows (of a pair: 128 and 128)
    const float* hidden_scale;
    const float* weight_scale;
    int64_t hidden_scale_stride, weight_scale_stride;
    void* logits;
    int64_t ldl;
    int rows, V, NT;
    int row_tiles, tiles;  // tiles of hidden rows (many rows); of both
    int blocks;            // of K
    int stages, accs;
    uint32_t tmem_cols;    // a power of two >= accs * NT
    int wide_scales;       // the hidden scales can be read four at a time
    int wide_stores;       // the logits can be written 16 bytes at a time
    unsigned long long* timeouts;
};

// A ring's place and the parity of its phase.
struct Ring {
    uint32_t at, phase;
    __device__ __forceinline__ void next(uint32_t n)
    {
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
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

// The same for a pair of CTAs: the loads' barrier may be the other CTA's, the
// MMA's operands and accumulator are halves in each, and the arrivals go to the
// barrier of both.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit_pair(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
}

// Arrive on a barrier of the pair. What it tells is that tensor memory has been
// read, which tcgen05.fence orders; a release would wait for this thread's other
// accesses as well, on the way of every block.
__device__ __forceinline__ void arrive_pair(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 or 32 consecutive columns of this thread's tensor-memory lane; complete after tmem_wait.
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

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
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

// (a, b) += (x, y) * (p, q), two fp32 operations in one.
__device__ __forceinline__ void fma2(float2& a, uint32_t x, uint32_t y, float p, float q)
{
    asm("{\n\t.reg .b64 s, t, u;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%4, %5};\n\t"
        "fma.rn.f32x2 s, t, u, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "+f"(a.x), "+f"(a.y)
        : "r"(x), "r"(y), "f"(p), "f"(q));
}

// True in one lane of a warp whose lanes are together. The warps that issue TMA
// loads and MMAs run as a whole, with this around the issuing instructions: their
// operands are then known to be the same for all lanes, which those instructions
// need. (Inside `if (lane == 0)` an MMA took about 65 cycles to issue and a commit
// about 100, together more than the tensor cores took for a block.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
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

// What both kernels have in shared memory after the operand ring and their own.
struct Control {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t tfull[kMaxAccs], tempty[kMaxAccs];  // an accumulator is complete; has been read
    uint64_t drained;                            // every MMA of the CTA has completed
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(Control) <= kBarBytes, "");

template <bool kPair>
__device__ __forceinline__ void begin(const Params& P, Control& C)
{
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&C.full[s], 1);
            mbar_init(&C.empty[s], 1);
        }
        for (int a = 0; a < kMaxAccs; ++a) {
            mbar_init(&C.tfull[a], 1);
            mbar_init(&C.tempty[a], kPair ? 16 : 8);
        }
        mbar_init(&C.drained, 1);
        C.gave_up = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tm)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tn)) : "memory");
    }
    if (warp == 9) {
        if (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&C.tmem)),
                         "r"(P.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&C.tmem)),
                         "r"(P.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    fence_before_sync();
    __syncthreads();
    if (kPair) cluster_sync();
    fence_after_sync();
}

template <bool kPair>
__device__ __forceinline__ void end(const Params& P, Control& C, uint32_t tmem)
{
    fence_before_sync();
    __syncthreads();
    if (kPair) {
        // every MMA has completed, and the last of their arrivals has come; then the other CTA is done with this
        // one's shared and tensor memory, too
        if (threadIdx.x == 0 && !wait(&C.drained, 0)) C.gave_up = 1;
        __syncthreads();
        cluster_sync();
    }
    fence_after_sync();
    if (threadIdx.x >> 5 == 9) {
        if (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols)
                         : "memory");
    }
    if (threadIdx.x == 0 && C.gave_up && P.timeouts) atomicAdd(P.timeouts, 1ull);
}

// The TMA warp of a CTA that works alone.
__device__ __forceinline__ void produce(const Params& P, Control& C, unsigned char* sa, unsigned char* sb)
{
    const uint32_t S = uint32_t(P.stages), b_bytes = uint32_t(P.NT) * kBK;
    Ring s{0, 0};
    uint32_t issued = 0;
    bool ok = true;
    for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
        for (int b = 0; b < P.blocks; ++b) {
            ok = wait(&C.empty[s.at], s.phase ^ 1u);
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&C.full[s.at], kABytes + b_bytes);
                tma_load_2d(smem_addr(sa + s.at * kABytes), &P.tm, b * kBK, t * kBM, smem_addr(&C.full[s.at]));
                tma_load_2d(smem_addr(sb + s.at * b_bytes), &P.tn, b * kBK, 0, smem_addr(&C.full[s.at]));
            }
            __syncwarp();
            s.next(S);
            ++issued;
        }
    }
    if (!ok) C.gave_up = 1;
    // the last copies issued land before the CTA may exit
    for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j) wait(&C.full[j % S], j / S & 1u);
}

// The MMA warp: each block of K into the next accumulator.
__device__ __forceinline__ void multiply(const Params& P, Control& C, unsigned char* sa, unsigned char* sb,
                                         uint32_t tmem)
{
    const uint32_t idesc = idesc_e4m3(kBM, P.NT), b_bytes = uint32_t(P.NT) * kBK;
    Ring s{0, 0}, acc{0, 0};
    bool ok = true;
    for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
        for (int b = 0; b < P.blocks; ++b) {
            ok = wait(&C.full[s.at], s.phase) && wait(&C.tempty[acc.at], acc.phase ^ 1u);
            if (!ok) break;
            fence_after_sync();
            const uint32_t d = tmem + acc.at * uint32_t(P.NT);
            const uint64_t da = desc_sw128(smem_addr(sa + s.at * kABytes));
            const uint64_t db = desc_sw128(smem_addr(sb + s.at * b_bytes));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBK / kUK; ++k)  // +32 bytes inside the 128-byte rows
                    mma_e4m3(d, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc, uint32_t(k));
                mma_commit(&C.tfull[acc.at]);
                mma_commit(&C.empty[s.at]);
            }
            __syncwarp();
            s.next(uint32_t(P.stages));
            acc.next(uint32_t(P.accs));
        }
    }
    if (!ok) C.gave_up = 1;
    if (elect_one()) mma_commit(&C.drained);
    __syncwarp();
    wait(&C.drained, 0);
}

// Scales of blocks b .. b + 3 from one row of them; 0 past the row's end and where there is none.
__device__ __forceinline__ void fetch_scales(float (&q)[kScaleBlocks], const float* row, int b, int blocks, bool has,
                                             bool wide)
{
    if (has && wide && b + kScaleBlocks <= blocks) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + b));
        q[0] = v.x;
        q[1] = v.y;
        q[2] = v.z;
        q[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < kScaleBlocks; ++i) q[i] = has && b + i < blocks ? __ldg(row + b + i) : 0.f;
    }
}

// Few rows: the weight is M, the hidden rows N = NT <= 2 * kCols.
template <typename T, int kCols>
__global__ void __launch_bounds__(kThreads, 1) few_rows_kernel(const __grid_constant__ Params P)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sa = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char* sb = sa + size_t(P.stages) * kABytes;
    float* scales = reinterpret_cast<float*>(sb + size_t(P.stages) * P.NT * kBK);  // [2][kScaleBlocks][kFewRows]
    Control& C = *reinterpret_cast<Control*>(reinterpret_cast<unsigned char*>(scales) + kScaleBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    begin<false>(P, C);
    const uint32_t tmem = C.tmem;

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 8) {
        produce(P, C, sa, sb);
    } else if (warp == 9) {
        multiply(P, C, sa, sb, tmem);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int group = warp >> 2, quarter = warp & 3;  // quarter: the tensor-memory lanes a warp may read
        const int j = quarter * 32 + lane;                // thread of the group: it fetches column j's scales
        const int half = ((P.NT >> 1) + 15) & ~15;
        const int c0 = group * half, cols = max(0, min(half, P.NT - c0));
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(c0);
        const bool has = j < cols && c0 + j < P.rows;
        const float* sh = P.hidden_scale + int64_t(c0 + j) * P.hidden_scale_stride;
        float* mine = scales + group * (kFewRows / 2);
        Ring acc{0, 0};
        uint32_t buffer = 0;
        bool ok = true;
        // raw scales of the next four blocks: they are fetched four blocks ahead and multiplied when those come
        float qh[kScaleBlocks], qw[kScaleBlocks];
        if (int(blockIdx.x) < P.tiles) {
            fetch_scales(qh, sh, 0, P.blocks, has, P.wide_scales);
            fetch_scales(qw, P.weight_scale + blockIdx.x * P.weight_scale_stride, 0, P.blocks, true, false);
        }
        for (int t = int(blockIdx.x); t < P.tiles; t += int(gridDim.x)) {  // to the end even where a wait gave up:
                                                                           // its group's barriers count on it
            float2 sum[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = make_float2(0.f, 0.f);
            for (int b = 0; b < P.blocks; ++b) {
                if (b % kScaleBlocks == 0) {
                    // the other buffer is free: all have come to the barrier before this one after its last use
                    buffer ^= 1u;
                    float* row = mine + buffer * (kScaleBlocks * kFewRows);
                    if (j < kFewRows / 2)
#pragma unroll
                        for (int i = 0; i < kScaleBlocks; ++i) row[i * kFewRows + j] = qh[i] * qw[i];
                    group_sync(group);
                    const bool more = b + kScaleBlocks < P.blocks;
                    const int nt = more ? t : t + int(gridDim.x), nb = more ? b + kScaleBlocks : 0;
                    if (nt < P.tiles) {
                        fetch_scales(qh, sh, nb, P.blocks, has, P.wide_scales);
                        fetch_scales(qw, P.weight_scale + nt * P.weight_scale_stride, nb, P.blocks, true, false);
                    }
                }
                const float* row = mine + buffer * (kScaleBlocks * kFewRows) + b % kScaleBlocks * kFewRows;
                ok = ok && wait(&C.tfull[acc.at], acc.phase);
                if (ok) {
                    fence_after_sync();
                    const uint32_t at = lanes + acc.at * uint32_t(P.NT);
                    uint32_t r[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; c += 16)
                        if (c < cols) tmem_ld16(at + c, r + c);
                    tmem_wait();
                    fence_before_sync();
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        tmem_take16(r + c);
                        if (c < cols)
#pragma unroll
                            for (int i = c; i < c + 16; i += 4) {
                                const float4 s = *reinterpret_cast<const float4*>(row + i);
                                fma2(sum[i / 2], r[i], r[i + 1], s.x, s.y);
                                fma2(sum[i / 2 + 1], r[i + 2], r[i + 3], s.z, s.w);
                            }
                    }
                }
                __syncwarp();
                if (ok && lane == 0) arrive(&C.tempty[acc.at]);
                acc.next(uint32_t(P.accs));
            }
            const int v = t * kBM + quarter * 32 + lane;
            if (ok && v < P.V) {
                T* out = static_cast<T*>(P.logits) + int64_t(c0) * P.ldl + v;
                const int n = min(cols, P.rows - c0);
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if (c < n) put(out + int64_t(c) * P.ldl, c & 1 ? sum[c / 2].y : sum[c / 2].x);
            }
        }
        if (!ok && lane == 0) C.gave_up = 1;
    }
    end<false>(P, C, tmem);
}

// Store 16-byte pieces, or single elements where they do not lie on 16 bytes: a
// warp's 32 rows of kRowBytes from its buffer, columns from v0 on.
template <typename T>
__device__ __forceinline__ void store_rows(const Params& P, const unsigned char* buf, int row0, int v0, int lane)
{
    constexpr int kPer = kRowBytes / int(sizeof(T));
    if (P.wide_stores && v0 + kPer <= P.V) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + (lane >> 2), piece = lane & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(buf + row * kRowPitch + piece * 16);
            if (row0 + row < P.rows)
                __stcs(reinterpret_cast<uint4*>(static_cast<T*>(P.logits) + int64_t(row0 + row) * P.ldl + v0) + piece, v);
        }
    } else {
        const int col = lane % kPer;
        for (int row = lane / kPer; row < 32; row += 32 / kPer) {
            const T v = reinterpret_cast<const T*>(buf + row * kRowPitch)[col];
            if (row0 + row < P.rows && v0 + col < P.V)
                (static_cast<T*>(P.logits) + int64_t(row0 + row) * P.ldl + v0)[col] = v;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// A pair's tile t: its first hidden and weight rows.
__device__ __forceinline__ void pair_tile(const Params& P, int t, int& m, int& n)
{
    m = t % P.row_tiles * (2 * kBM);
    n = t / P.row_tiles * kWideN;
}

// The same barrier of the pair's first CTA, in the cluster's shared memory.
__device__ __forceinline__ uint32_t of_first(uint64_t* bar) { return dsmem_map(smem_addr(bar), 0); }

// The TMA warp of each CTA of a pair: its half of both operands. The first
// CTA's barrier counts the bytes of both.
__device__ __forceinline__ void pair_produce(const Params& P, Control& C, unsigned char* sa, unsigned char* sb,
                                             uint32_t rank, int first, int step)
{
    const uint32_t S = uint32_t(P.stages);
    Ring s{0, 0};
    uint32_t issued = 0;
    bool ok = true;
    for (int t = first; ok && t < P.tiles; t += step) {
        int m, n;
        pair_tile(P, t, m, n);
        m += int(rank) * kBM;
        n += int(rank) * kBM;
        for (int b = 0; b < P.blocks; ++b) {
            ok = wait(&C.empty[s.at], s.phase ^ 1u);
            if (!ok) break;
            const uint32_t bar = of_first(&C.full[s.at]);
            if (elect_one()) {
                if (rank == 0) mbar_arrive_expect_tx(&C.full[s.at], 4 * kABytes);
                tma_load_2d_pair(smem_addr(sa + s.at * kABytes), &P.tm, b * kBK, m, bar);
                tma_load_2d_pair(smem_addr(sb + s.at * kABytes), &P.tn, b * kBK, n, bar);
            }
            __syncwarp();
            s.next(S);
            ++issued;
        }
    }
    if (!ok) C.gave_up = 1;
    // the last copies of both CTAs land before either may exit (the other waits for this one at the end)
    if (rank == 0)
        for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j) wait(&C.full[j % S], j / S & 1u);
}

// The MMA warp of the pair.
__device__ __forceinline__ void pair_multiply(const Params& P, Control& C, unsigned char* sa, unsigned char* sb,
                                              uint32_t tmem, int first, int step)
{
    const uint32_t idesc = idesc_e4m3(2 * kBM, kWideN);
    Ring s{0, 0}, acc{0, 0};
    bool ok = true;
    for (int t = first; ok && t < P.tiles; t += step) {
        for (int b = 0; b < P.blocks; ++b) {
            ok = wait(&C.full[s.at], s.phase) && wait(&C.tempty[acc.at], acc.phase ^ 1u);
            if (!ok) break;
            fence_after_sync();
            const uint32_t d = tmem + acc.at * uint32_t(kWideN);
            const uint64_t da = desc_sw128(smem_addr(sa + s.at * kABytes));
            const uint64_t db = desc_sw128(smem_addr(sb + s.at * kABytes));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBK / kUK; ++k)  // +32 bytes inside the 128-byte rows
                    mma_e4m3_pair(d, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc, uint32_t(k));
                mma_commit_pair(&C.tfull[acc.at]);
                mma_commit_pair(&C.empty[s.at]);
            }
            __syncwarp();
            s.next(uint32_t(P.stages));
            acc.next(uint32_t(P.accs));
        }
    }
    if (!ok) C.gave_up = 1;
    if (elect_one()) mma_commit_pair(&C.drained);
    __syncwarp();
}

// Many rows: the hidden rows are M, the weight N = 256, of a pair of CTAs.
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    many_rows_kernel(const __grid_constant__ Params P)
{
    constexpr int kCols = kWideN / 2;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sa = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char* sb = sa + size_t(P.stages) * kABytes;
    unsigned char* outs = sb + size_t(P.stages) * kABytes;
    Control& C = *reinterpret_cast<Control*>(outs + kOutBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int first = int(blockIdx.x >> 1), step = int(gridDim.x >> 1);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    begin<true>(P, C);
    const uint32_t tmem = C.tmem;

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 8) {
        pair_produce(P, C, sa, sb, rank, first, step);
    } else if (warp == 9) {
        if (rank == 0) pair_multiply(P, C, sa, sb, tmem, first, step);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int group = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(group * kCols);
        unsigned char* buf = outs + warp * (32 * kRowPitch);
        Ring acc{0, 0};
        bool ok = true;
        // a lane's hidden row and the group's block of weight rows: their scales, fetched four blocks ahead
        float qh[kScaleBlocks], qw[kScaleBlocks];
        auto fetch = [&](int t, int b) {
            int m, n;
            pair_tile(P, t, m, n);
            const int row = m + int(rank) * kBM + quarter * 32 + lane, vb = n / kBM + group;
            fetch_scales(qh, P.hidden_scale + int64_t(row) * P.hidden_scale_stride, b, P.blocks, row < P.rows,
                         P.wide_scales);
            fetch_scales(qw, P.weight_scale + int64_t(vb) * P.weight_scale_stride, b, P.blocks, vb * kBM < P.V, false);
        };
        if (first < P.tiles) fetch(first, 0);
        for (int t = first; ok && t < P.tiles; t += step) {
            float2 sum[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = make_float2(0.f, 0.f);
            for (int b0 = 0; ok && b0 < P.blocks; b0 += kScaleBlocks) {
                float q[kScaleBlocks];
#pragma unroll
                for (int i = 0; i < kScaleBlocks; ++i) q[i] = qh[i] * qw[i];
                const bool more = b0 + kScaleBlocks < P.blocks;
                if (more || t + step < P.tiles) fetch(more ? t : t + step, more ? b0 + kScaleBlocks : 0);
#pragma unroll
                for (int i = 0; i < kScaleBlocks; ++i) {
                    if (b0 + i >= P.blocks) break;
                    ok = wait(&C.tfull[acc.at], acc.phase);
                    if (!ok) break;
                    fence_after_sync();
                    const uint32_t at = lanes + acc.at * uint32_t(kWideN);
                    uint32_t r[2][16];
                    tmem_ld16(at, r[0]);
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        uint32_t* now = r[c / 16 & 1];
                        tmem_wait();
                        tmem_take16(now);
                        if (c + 16 < kCols) {  // the next columns come while these are added
                            tmem_ld16(at + c + 16, r[c / 16 + 1 & 1]);
                        } else {               // all of the accumulator has been read
                            fence_before_sync();
                            __syncwarp();
                            if (lane == 0) arrive_pair(of_first(&C.tempty[acc.at]));
                        }
#pragma unroll
                        for (int k = 0; k < 16; k += 2) fma2(sum[(c + k) / 2], now[k], now[k + 1], q[i], q[i]);
                    }
                    acc.next(uint32_t(P.accs));
                }
            }
            if (!ok) break;
            int row0, v0;
            pair_tile(P, t, row0, v0);
            row0 += int(rank) * kBM + quarter * 32;
            v0 += group * kCols;
            constexpr int kPer = kRowBytes / int(sizeof(T));
#pragma unroll
            for (int c = 0; c < kCols; c += kPer) {
                uint4* to = reinterpret_cast<uint4*>(buf + lane * kRowPitch);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (sizeof(T) == 2) {
                        const float2* s = sum + c / 2 + 4 * i;
                        to[i] = make_uint4(pack_bf16(s[0].x, s[0].y), pack_bf16(s[1].x, s[1].y),
                                           pack_bf16(s[2].x, s[2].y), pack_bf16(s[3].x, s[3].y));
                    } else {
                        const float2* s = sum + c / 2 + 2 * i;
                        to[i] = make_uint4(__float_as_uint(s[0].x), __float_as_uint(s[0].y), __float_as_uint(s[1].x),
                                           __float_as_uint(s[1].y));
                    }
                }
                __syncwarp();
                store_rows<T>(P, buf, row0, v0 + c, lane);
                __syncwarp();
            }
        }
        if (!ok && lane == 0) C.gave_up = 1;
    }
    end<true>(P, C, tmem);
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
Kernel kernel_for(bool few, int NT)
{
    return !few       ? many_rows_kernel<T>
           : NT <= 32 ? few_rows_kernel<T, 16>
           : NT <= 64 ? few_rows_kernel<T, 32>
                      : few_rows_kernel<T, 64>;
}

}  // namespace scaled

int scaled_head_launch(const sampler_scaled_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows,
                       int64_t vocab, int sms, unsigned long long* timeouts, cudaStream_t stream)
{
    using namespace scaled;
    Params p;
    std::memset(&p, 0, sizeof p);
    const bool few = rows <= kFewRows;
    p.row_tiles = few ? 1 : int((rows + 2 * kBM - 1) / (2 * kBM));
    p.NT = few ? int((rows + 15) / 16 * 16) : kWideN;
    const int64_t tiles = (vocab + (few ? kBM : kWideN) - 1) / (few ? kBM : kWideN) * p.row_tiles;
    if (tiles > INT32_MAX - 65536) return SAMPLER_ERR_TOO_LARGE;
    p.tiles = int(tiles);
    p.blocks = int((g.hidden_dim + kBK - 1) / kBK);
    const size_t stage = kABytes + (few ? size_t(p.NT) * kBK : size_t(kABytes)), own = few ? kScaleBytes : kOutBytes;
    p.stages = int(std::min<size_t>(kMaxStages, (kSmemMax - 1024 - kBarBytes - own) / stage));
    p.accs = std::min(kMaxAccs, kTmemCols / p.NT);
    p.tmem_cols = 32;
    while (p.tmem_cols < uint32_t(p.accs * p.NT)) p.tmem_cols <<= 1;
    const bool maps = few ? encode(&p.tm, g.weight, vocab, g.hidden_dim, g.weight_stride, kBM) &&
                                encode(&p.tn, g.hidden, rows, g.hidden_dim, g.hidden_stride, p.NT)
                          : encode(&p.tm, g.hidden, rows, g.hidden_dim, g.hidden_stride, kBM) &&
                                encode(&p.tn, g.weight, vocab, g.hidden_dim, g.weight_stride, kBM);
    if (!maps) return SAMPLER_ERR_CUDA;
    p.hidden_scale = g.hidden_scale;
    p.weight_scale = g.weight_scale;
    p.hidden_scale_stride = g.hidden_scale_stride;
    p.weight_scale_stride = g.weight_scale_stride;
    p.wide_scales = g.hidden_scale_stride % 4 == 0 && reinterpret_cast<uintptr_t>(g.hidden_scale) % 16 == 0;
    p.logits = logits;
    p.ldl = ldl;
    p.wide_stores = ldl * (dtype == SAMPLER_DTYPE_BF16 ? 2 : 4) % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    p.rows = int(rows);
    p.V = int(vocab);
    p.timeouts = timeouts;
    const Kernel kernel = dtype == SAMPLER_DTYPE_BF16 ? kernel_for<uint16_t>(few, p.NT) : kernel_for<float>(few, p.NT);
    const size_t smem = 1024 + size_t(p.stages) * stage + own + kBarBytes;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(smem)) != cudaSuccess)
        return SAMPLER_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(few ? std::min(sms, p.tiles) : 2 * std::min(sms / 2, p.tiles)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
