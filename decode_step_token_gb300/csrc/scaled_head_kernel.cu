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
// Few rows (a small decode step; up to kFewRows) are taken transposed: a tile is
// 128 weight rows (M: one block of the weight's scales, so that scale is one
// number for a tile and block) by all hidden rows (N). The weight's bytes are all
// the time then. A column's scale is the same for all lanes and comes from shared
// memory; the accumulators are up to eight, and the lanes are neighbouring tokens
// of the vocabulary, so that the logits are stored as they lie.
//
// More rows are taken as they are: 128 hidden rows (M) by 256 weight rows (N). A
// lane is a hidden row here, so its scale is one register, two products are one
// instruction, and nothing is read from shared memory. The logits go through
// shared memory to the TMA engine, which stores them while the next tile is under
// way (a warp's own stores took 12 % of the time). N is as wide as two accumulators
// of tensor memory allow: the way of an accumulator round through the epilogue (its
// completion seen, its columns read, its release seen by the MMA warp) has to fit
// in one block's MMAs, and wider tiles load less from L2. Pairs of CTAs that share
// their weight tile by multicast load a third less, but wait for each other: 1.49
// against 1.46 ms at 4096 x 128000 x 4096, and one tile of 256 rows where CTAs
// alone have two (333 x 20011 x 1000: 41 against 30 us, with the stores as they were).
//
// Where the two meet, transposed / not, a call at a time after 268 MB of writes: over 1 to 32 rows, seven
// vocabularies of 4000 to 151936 and a K of 1024 and 4096, transposed is faster at
// 81 of 84 sizes (17 x 4000 x 1024 6.1 / 7.6 us, 16 x 64000 x 4096 57 / 63, 32 x
// 128000 x 4096 103 / 108) and up to 6 % slower at the others, all of 32 rows x 4096
// (64000 56.9 / 53.8, 100000 90.2 / 86.2, 151936 116.9 / 115.8). Beyond, with a form
// for up to 96 rows, call after call: 33 x 128000 x 4096 92 / 94, 64 x 128000 94 /
// 95.5, 64 x 64000 57 / 51, 64 x 256000 x 1024 60 / 51, 96 x 128000 121 / 97. (What
// decides at 32 rows and more is how the tiles fill the SMs in their last round.)
//
// Measured: 16 x 128000 x 4096 83-86 us (6.1-6.4 TB/s, 91-94 % of the copy rate); 4096 x
// 128000 x 4096 1.46-1.49 ms call after call (2880-2940 TFLOP/s), 1.66-1.70 ms where
// each call has inputs of its own that are not in L2 (2530-2590).
//
// Persistent, one CTA an SM; warp roles:
//   warps 0-7  the epilogue: two groups of four warps, each a half of the tile's
//              columns, a warp 32 of its lanes;
//   warp 8     issues the TMA loads of the operand ring;
//   warp 9     owns the tensor memory and issues the MMAs.
// Warps 10 and 11 fill up the third warpgroup, which gives its registers to the
// epilogue's where those hold 128 sums a thread (more rows).
// Every wait is bounded in time, with one answer for a warp; a CTA whose wait gives up counts itself in the
// handle's statistics and leaves its logits unwritten.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "launch.h"
#include "ptx.cuh"
#include "tensor_core.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace scaled {

constexpr int kBM = 128;                       // MMA M, and a block of the weight's scales
constexpr int kBK = 128;                       // K of a stage: a block of scales, one 128-byte swizzled row
constexpr int kUK = 32;                        // K of one tcgen05.mma of 8-bit operands
constexpr int kThreads = 384;
constexpr int kFewRegs = 24, kManyRegs = 240;  // many rows: 128 * 24 + 256 * 240 <= 384 * 168
constexpr int kGroupThreads = 128;             // of one half of the columns
constexpr int kMaxStages = 8;
constexpr int kMaxAccs = 8;
constexpr int kTmemCols = 512;
constexpr int kFewRows = 32;                   // the most that are taken transposed (see above)
constexpr int kWideN = 256;                    // weight rows of a tile of many hidden rows
constexpr int kWideAccs = kTmemCols / kWideN;
constexpr uint32_t kWideBytes = kWideN * kBK; // of a stage
constexpr int kLoad = 16;                      // columns that a thread reads at once (32: registers spill, 2264 TFLOP/s)
constexpr uint32_t kOutBytes = 8 * kBoxBytes;  // one for each warp of the epilogue: with more, a stage less
constexpr int kScaleBlocks = 4;                // blocks of K whose scales are fetched together
constexpr uint32_t kABytes = kBM * kBK;        // 16 KB a stage
constexpr size_t kScaleBytes = 2 * kScaleBlocks * kFewRows * 4;  // transposed: two buffers of every column's scales
constexpr size_t kBarBytes = 512;
constexpr size_t kSmemMax = 227 * 1024;

struct Params {
    CUtensorMap to;      // many rows: the logits, boxes of 128 bytes by 32 rows, 128-byte swizzle
    CUtensorMap tm, tn;  // the operands of M and N [rows, K], 128-byte swizzle: boxes of 128 bytes by 128 and NT
                         // rows
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
    int wide_scales;       // bits 0, 1: the hidden and the weight's scales can be read four at a time
    int tma_stores;        // the logits lie so that the TMA engine can write them
    uint64_t wait_ns;      // kWaitNs, or 0: every wait gives up
    unsigned long long* timeouts;
};

using Ring = RingPlace;

// kind::f8f6f4, fp32 accumulator, e4m3 A and B (type 0 each), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
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

// A whole warp waits for the phase of `bar` with the given parity, for `ns` at most.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint64_t ns)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || mbar_wait_warp(bar, parity, now_ns() + ns);
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
// Block n of a CTA (counted over its tiles) is in stage n % stages and
// accumulator n % accs. The MMA warp's own instructions are on the tensor cores'
// way (a wait takes it about 150 cycles even where nothing is left to wait for, a
// commit 100), so it has one barrier to wait for and one to commit to: block n's
// accumulator is free when the epilogue has read block n - accs, and the epilogue
// arrives for that on block n's own barrier. With stages > accs no barrier can get
// two phases ahead of one who waits for it.
struct Control {
    uint64_t ready[kMaxStages];  // of the block in a stage: its operands have come, and its accumulator has been read
                                 // by every warp of the epilogue
    uint64_t done[kMaxStages];   // its MMAs have completed: the accumulator can be read, the stage filled again
    uint64_t drained;            // every MMA of the CTA has completed
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(Control) <= kBarBytes, "");

__device__ __forceinline__ void begin(const Params& P, Control& C)
{
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&C.ready[s], 1 + 8);
            mbar_init(&C.done[s], 1);
        }
        mbar_init(&C.drained, 1);
        C.gave_up = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tm)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tn)) : "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&C.tmem)),
                     "r"(P.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
}

__device__ __forceinline__ void end(const Params& P, Control& C, uint32_t tmem)
{
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (threadIdx.x >> 5 == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
    if (threadIdx.x == 0 && C.gave_up && P.timeouts) atomicAdd(P.timeouts, 1ull);
}

// Tile t: its first rows of M and of N. (Of many rows, tiles that follow one
// another have the same weight rows, which are then in L2.)
template <bool kFew>
__device__ __forceinline__ void tile_at(const Params& P, int t, int& m, int& n)
{
    m = kFew ? t * kBM : t % P.row_tiles * kBM;
    n = kFew ? 0 : t / P.row_tiles * kWideN;
}

// The TMA warp. It and the MMA warp run as a whole, with elect_one around the
// issuing instructions: their operands are then known to be the same for all
// lanes, which those instructions need. (Inside `if (lane == 0)` an MMA took about
// 65 cycles to issue and a commit about 100, together more than the tensor cores
// took for a block.)
template <bool kFew>
__device__ __forceinline__ void produce(const Params& P, Control& C, unsigned char* sa, unsigned char* sb)
{
    const uint32_t S = uint32_t(P.stages), b_bytes = kFew ? uint32_t(P.NT) * kBK : kWideBytes;
    Ring s{0, 0};
    uint32_t issued = 0;
    bool ok = P.wait_ns != 0;  // 0: nothing is loaded, and the other warps' waits give up
    for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
        int m, n;
        tile_at<kFew>(P, t, m, n);
        for (int b = 0; b < P.blocks; ++b) {
            ok = wait(&C.done[s.at], s.phase ^ 1u, P.wait_ns);
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&C.ready[s.at], kABytes + b_bytes);
                tma_load_2d(smem_addr(sa + s.at * kABytes), &P.tm, b * kBK, m, smem_addr(&C.ready[s.at]));
                tma_load_2d(smem_addr(sb + s.at * b_bytes), &P.tn, b * kBK, n, smem_addr(&C.ready[s.at]));
            }
            __syncwarp();
            s.next(S);
            ++issued;
        }
    }
    if (!ok) C.gave_up = 1;
    // the last copies issued land before the CTA may exit
    for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j) wait(&C.ready[j % S], j / S & 1u, kWaitNs);
}

// The MMA warp: each block of K into the next accumulator.
template <bool kFew>
__device__ __forceinline__ void multiply(const Params& P, Control& C, unsigned char* sa, unsigned char* sb,
                                         uint32_t tmem)
{
    const uint32_t cols = kFew ? uint32_t(P.NT) : uint32_t(kWideN), b_bytes = cols * kBK;
    const uint32_t idesc = idesc_e4m3(kBM, int(cols)), accs = kFew ? uint32_t(P.accs) : uint32_t(kWideAccs);
    Ring s{0, 0}, acc{0, 0};
    bool ok = true;
    for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
        for (int b = 0; b < P.blocks; ++b) {
            const uint32_t d = tmem + acc.at * cols;
            const uint64_t da = desc_sw128(smem_addr(sa + s.at * kABytes));
            const uint64_t db = desc_sw128(smem_addr(sb + s.at * b_bytes));
            ok = wait(&C.ready[s.at], s.phase, P.wait_ns);
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBK / kUK; ++k)  // +32 bytes inside the 128-byte rows
                    mma_e4m3(d, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc, uint32_t(k));
                mma_commit(&C.done[s.at]);
            }
            __syncwarp();
            s.next(uint32_t(P.stages));
            acc.next(accs);
        }
    }
    if (!ok) C.gave_up = 1;
    if (elect_one()) mma_commit(&C.drained);
    __syncwarp();
    wait(&C.drained, 0, kWaitNs);
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

// The accumulators of the first blocks are free from the start.
__device__ __forceinline__ void free_first(const Params& P, Control& C, int lane)
{
    if (lane == 0)
        for (int k = 0; k < P.accs; ++k) mbar_arrive(&C.ready[k]);
    __syncwarp();
}

// Few rows: the weight is M, the hidden rows N = NT, 16 or 32.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) few_rows_kernel(const __grid_constant__ Params P)
{
    constexpr int kCols = kFewRows / 2;  // of a thread
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sa = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char* sb = sa + size_t(P.stages) * kABytes;
    float* scales = reinterpret_cast<float*>(sb + size_t(P.stages) * P.NT * kBK);  // [2][kScaleBlocks][kFewRows]
    Control& C = *reinterpret_cast<Control*>(reinterpret_cast<unsigned char*>(scales) + kScaleBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    begin(P, C);
    const uint32_t tmem = C.tmem;

    if (warp == 8) {
        produce<true>(P, C, sa, sb);
    } else if (warp == 9) {
        multiply<true>(P, C, sa, sb, tmem);
    } else if (warp < 8) {
        const int group = warp >> 2, quarter = warp & 3;  // quarter: the tensor-memory lanes a warp may read
        const int j = quarter * 32 + lane;                // thread of the group: it fetches column j's scales
        const int c0 = group * kCols, cols = max(0, min(kCols, P.NT - c0));  // 0 or kCols
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(c0);
        const bool has = j < cols && c0 + j < P.rows;
        const float* sh = P.hidden_scale + int64_t(c0 + j) * P.hidden_scale_stride;
        float* mine = scales + group * (kFewRows / 2);
        Ring acc{0, 0}, s{0, 0};
        uint32_t freed = uint32_t(P.accs);  // stage of the block that the accumulator now read is for next
        free_first(P, C, lane);
        uint32_t buffer = 0;
        bool ok = true;
        // raw scales of the next four blocks: they are fetched four blocks ahead and multiplied when those come
        float qh[kScaleBlocks], qw[kScaleBlocks];
        if (int(blockIdx.x) < P.tiles) {
            fetch_scales(qh, sh, 0, P.blocks, has, P.wide_scales & 1);
            fetch_scales(qw, P.weight_scale + blockIdx.x * P.weight_scale_stride, 0, P.blocks, true, P.wide_scales & 2);
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
                        fetch_scales(qh, sh, nb, P.blocks, has, P.wide_scales & 1);
                        fetch_scales(qw, P.weight_scale + nt * P.weight_scale_stride, nb, P.blocks, true, P.wide_scales & 2);
                    }
                }
                const float* row = mine + buffer * (kScaleBlocks * kFewRows) + b % kScaleBlocks * kFewRows;
                ok = ok && wait(&C.done[s.at], s.phase, P.wait_ns);
                if (ok) {
                    fence_after_sync();
                    const uint32_t at = lanes + acc.at * uint32_t(P.NT);
                    uint32_t r[kCols];
                    if (cols > 0) {
                        tmem_ld16(at, r);
                        tmem_wait();
                        tmem_take16(r);
#pragma unroll
                        for (int i = 0; i < kCols; i += 4) {
                            const float4 s = *reinterpret_cast<const float4*>(row + i);
                            fma2(sum[i / 2], r[i], r[i + 1], s.x, s.y);
                            fma2(sum[i / 2 + 1], r[i + 2], r[i + 3], s.z, s.w);
                        }
                    }
                    fence_before_sync();
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&C.ready[freed]);
                acc.next(uint32_t(P.accs));
                s.next(uint32_t(P.stages));
                freed = freed + 1 == uint32_t(P.stages) ? 0 : freed + 1;
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
    end(P, C, tmem);
}

// Many rows: the hidden rows are M, the weight N.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) many_rows_kernel(const __grid_constant__ Params P)
{
    constexpr int kCols = kWideN / 2;                  // of a thread: a block of the weight's scales
    constexpr int kBoxCols = 128 / int(sizeof(T));     // of a box of logits
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sa = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char* sb = sa + size_t(P.stages) * kABytes;
    unsigned char* outs = sb + size_t(P.stages) * kWideBytes;
    Control& C = *reinterpret_cast<Control*>(outs + kOutBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = int(blockIdx.x), step = int(gridDim.x);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    begin(P, C);
    const uint32_t tmem = C.tmem;

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 8) {
        produce<false>(P, C, sa, sb);
    } else if (warp == 9) {
        multiply<false>(P, C, sa, sb, tmem);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int group = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(group * kCols);
        unsigned char* out = outs + warp * kBoxBytes;
        Ring acc{0, 0}, s{0, 0};
        uint32_t freed = kWideAccs;  // stage of the block that the accumulator now read is for next
        free_first(P, C, lane);
        bool ok = true;
        // scales of a lane's hidden row and of the group's weight rows, fetched four blocks of K ahead
        float qh[kScaleBlocks], qw[kScaleBlocks];
        int row0 = 0, v0 = 0;  // of the tile that is fetched for
        const float *ph = nullptr, *pw = nullptr;
        auto place = [&](int t) {
            tile_at<false>(P, t, row0, v0);
            row0 += quarter * 32;
            v0 += group * kCols;
            ph = P.hidden_scale + int64_t(row0 + lane) * P.hidden_scale_stride;
            pw = P.weight_scale + int64_t(v0 / kBM) * P.weight_scale_stride;
        };
        auto fetch = [&](int b) {
            fetch_scales(qh, ph, b, P.blocks, row0 + lane < P.rows, P.wide_scales & 1);
            fetch_scales(qw, pw, b, P.blocks, v0 < P.V, P.wide_scales & 2);
        };
        if (first < P.tiles) {
            place(first);
            fetch(0);
        }
        for (int t = first; ok && t < P.tiles; t += step) {
            const int row = row0, v = v0;
            float2 sum[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = make_float2(0.f, 0.f);
            for (int b0 = 0; ok && b0 < P.blocks; b0 += kScaleBlocks) {
                float q[kScaleBlocks];
#pragma unroll
                for (int i = 0; i < kScaleBlocks; ++i) q[i] = qh[i] * qw[i];
                if (b0 + kScaleBlocks < P.blocks) {
                    fetch(b0 + kScaleBlocks);
                } else if (t + step < P.tiles) {
                    place(t + step);
                    fetch(0);
                }
#pragma unroll
                for (int i = 0; i < kScaleBlocks; ++i) {
                    if (b0 + i >= P.blocks) break;
                    ok = wait(&C.done[s.at], s.phase, P.wait_ns);
                    if (!ok) break;
                    fence_after_sync();
                    const uint32_t at = lanes + acc.at * uint32_t(kWideN);
                    uint32_t r[2][kLoad];
                    tmem_ld16(at, r[0]);
#pragma unroll
                    for (int c = 0; c < kCols; c += kLoad) {
                        uint32_t* now = r[c / kLoad & 1];
                        tmem_wait();
#pragma unroll
                        for (int k = 0; k < kLoad; k += 16) tmem_take16(now + k);
                        if (c + kLoad < kCols) {  // the next columns come while these are added
                            tmem_ld16(at + c + kLoad, r[c / kLoad + 1 & 1]);
                        } else {                  // all of the accumulator has been read
                            fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&C.ready[freed]);
                        }
#pragma unroll
                        for (int k = 0; k < kLoad; k += 2) fma2(sum[(c + k) / 2], now[k], now[k + 1], q[i], q[i]);
                    }
                    acc.next(kWideAccs);
                    s.next(uint32_t(P.stages));
                    freed = freed + 1 == uint32_t(P.stages) ? 0 : freed + 1;
                }
            }
            if (!ok) break;
            // (as store_logits does: called here, it spills registers of the fp32 form)
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
                    const int rows = min(32, P.rows - row), cols = min(kBoxCols, P.V - v - c0);
                    T* g = static_cast<T*>(P.logits) + int64_t(row) * P.ldl + v + c0;
#pragma unroll 8
                    for (int k = 0; k < 32; ++k) {
#pragma unroll
                        for (int c = lane; c < kBoxCols; c += 32)
                            if (k < rows && c < cols)
                                g[c] = *reinterpret_cast<const T*>(out + k * 128 + (c * int(sizeof(T)) ^ (k & 7) * 16));
                        g += P.ldl;
                    }
                    __syncwarp();
                }
            }
        }
        if (P.tma_stores && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok && lane == 0) C.gave_up = 1;
    }
    end(P, C, tmem);
}

using Kernel = void (*)(const Params);

}  // namespace scaled

int scaled_head_launch(const sampler_scaled_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows,
                       int64_t vocab, int sms, uint64_t wait_ns, unsigned long long* timeouts,
                       ScaledHeadGrants* grants, cudaStream_t stream)
{
    using namespace scaled;
    Params p;
    std::memset(&p, 0, sizeof p);
    const bool few = rows <= kFewRows;
    p.row_tiles = few ? 1 : int((rows + kBM - 1) / kBM);
    p.NT = few ? int((rows + 15) / 16 * 16) : kWideN;
    const int64_t tiles = (vocab + (few ? kBM : kWideN) - 1) / (few ? kBM : kWideN) * p.row_tiles;
    if (tiles > INT32_MAX - 65536) return SAMPLER_ERR_TOO_LARGE;
    p.tiles = int(tiles);
    p.blocks = int((g.hidden_dim + kBK - 1) / kBK);
    const int es = dtype == SAMPLER_DTYPE_BF16 ? 2 : 4;
    const size_t stage = kABytes + (few ? size_t(p.NT) * kBK : size_t(kWideBytes));
    const size_t own = few ? kScaleBytes : kOutBytes;
    p.stages = int(std::min<size_t>(kMaxStages, (kSmemMax - 1024 - kBarBytes - own) / stage));
    p.accs = std::min({kMaxAccs, kTmemCols / p.NT, p.stages - 1});
    p.tmem_cols = 32;
    while (p.tmem_cols < (few ? uint32_t(p.accs * p.NT) : uint32_t(kTmemCols))) p.tmem_cols <<= 1;
    const bool maps = few ? encode_bytes(&p.tm, g.weight, vocab, g.hidden_dim, g.weight_stride, kBM) &&
                                encode_bytes(&p.tn, g.hidden, rows, g.hidden_dim, g.hidden_stride, p.NT)
                          : encode_bytes(&p.tm, g.hidden, rows, g.hidden_dim, g.hidden_stride, kBM) &&
                                encode_bytes(&p.tn, g.weight, vocab, g.hidden_dim, g.weight_stride, kWideN);
    if (!maps) return SAMPLER_ERR_CUDA;
    p.hidden_scale = g.hidden_scale;
    p.weight_scale = g.weight_scale;
    p.hidden_scale_stride = g.hidden_scale_stride;
    p.weight_scale_stride = g.weight_scale_stride;
    p.wide_scales = (g.hidden_scale_stride % 4 == 0 && reinterpret_cast<uintptr_t>(g.hidden_scale) % 16 == 0 ? 1 : 0) |
                    (g.weight_scale_stride % 4 == 0 && reinterpret_cast<uintptr_t>(g.weight_scale) % 16 == 0 ? 2 : 0);
    p.logits = logits;
    p.ldl = ldl;
    p.tma_stores = !few && ldl * es % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    if (p.tma_stores && !encode_logits(&p.to, logits, dtype, rows, vocab, ldl)) return SAMPLER_ERR_CUDA;
    p.rows = int(rows);
    p.V = int(vocab);
    p.wait_ns = wait_ns;
    p.timeouts = timeouts;
    const bool bf16 = dtype == SAMPLER_DTYPE_BF16;
    const Kernel kernel = few    ? bf16 ? few_rows_kernel<uint16_t> : few_rows_kernel<float>
                          : bf16 ? many_rows_kernel<uint16_t> : many_rows_kernel<float>;
    const size_t smem = 1024 + size_t(p.stages) * stage + own + kBarBytes;
    // the limit belongs to the function, for all handles and threads: always the same one, so that no call takes
    // from another what it has been granted and not yet launched with
    bool& granted = grants->granted[few][bf16];
    if (!granted && cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMax)) != cudaSuccess)
        return SAMPLER_ERR_CUDA;
    granted = true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min(sms, p.tiles)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
