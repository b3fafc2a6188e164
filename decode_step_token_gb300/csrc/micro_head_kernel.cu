// micro_head_kernel.cu -- the LM head in microscaled 4 bits on the fifth-generation
// tensor cores: logits[i, v] = hidden_row_scale[i] * weight_row_scale[v] * sum_k of
// products of e2m1 values, each times its block's scale.
//
// tcgen05.mma takes the scales of the blocks itself, from tensor memory, so that
// the whole of K is one sum in fp32 tensor memory, and the epilogue's threads see a
// tile once. A stage of the operand ring is 256 of K: 128 bytes a row, one swizzled
// row, and the scales of its blocks as they lie in memory, tiles of 128 rows by 4
// blocks that tcgen05.cp spreads over the lanes of tensor memory. There are two
// places for a stage's scales there, one of which is filled while the MMAs read the
// other.
//
// Few rows (a decode step; up to kFewRows) are taken transposed: a tile is 128
// weight rows (M) by all hidden rows (N), and the weight's bytes are all the time.
// The lanes are then neighbouring tokens, and the logits are stored as they lie.
// More rows are taken as they are: 128 hidden rows (M) by 256 weight rows (N), the
// widest tile there is, for the bytes that a product takes from L2. Its accumulator
// and the scales leave no room for a second one: the epilogue reads it into registers
// first and gives it back, and scales, rounds and stores (through shared memory and the
// TMA engine) under the next tile's products.
//
// Persistent, one CTA an SM; warp roles:
//   warps 0-7  the epilogue: two groups of four warps, a warp 32 of the tile's lanes;
//   warp 8     loads the operand ring: the values by TMA tiles, the scales by bulk copies;
//   warp 9     owns the tensor memory and issues the copies of scales and the MMAs.
// Every wait is bounded in time, with one answer for a warp; a CTA whose wait gives
// up counts itself in the handle's statistics and leaves its logits unwritten.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "launch.h"
#include "ptx.cuh"
#include "tensor_core.cuh"
#include "warp_wait.cuh"

namespace dst {
namespace micro_head {

constexpr int kBM = 128;                     // MMA M, and the rows of a tile of scales
constexpr int kBK = 256;                     // K of a stage: 128 bytes a row
constexpr int kRowBytes = kBK / 2;
constexpr int kUK = 64;                      // K of one tcgen05.mma
constexpr int kThreads = 384;
constexpr int kEpilogue = 8;                 // warps
constexpr int kFewRegs = 24, kManyRegs = 240;  // many rows: 128 * 24 + 256 * 240 <= 384 * 168
constexpr int kMaxStages = 8;
constexpr int kFewRows = 128;                // the most that are taken transposed
constexpr int kWideN = 256;                  // weight rows of a tile of many hidden rows
constexpr uint32_t kABytes = kBM * kRowBytes;
constexpr uint32_t kScaleTile = 512;         // 128 rows by 4 blocks
constexpr uint32_t kOutBytes = kEpilogue * kBoxBytes;
constexpr uint32_t kRowScaleBytes = 2 * kWideN * 4;  // few rows: the columns' scales; many: two tiles' columns'
constexpr uint32_t kBarBytes = 512;
constexpr size_t kSmemMax = 227 * 1024;

struct Params {
    CUtensorMap to;      // many rows: the logits, boxes of 128 bytes by 32 rows, 128-byte swizzle
    CUtensorMap tm, tn;  // the operands of M and N [rows, K / 2 bytes], 128-byte swizzle: boxes of 128 bytes by 128 and
                         // NT rows
    const unsigned char *sm, *sn;             // their scales
    const float *row_scale_m, *row_scale_n;   // NULL = 1
    void* logits;
    int64_t ldl;
    int rows, V, NT;
    int m_tiles, n_tiles;  // tiles of 128 rows that the scales of either have
    int k_tiles;           // tiles of 4 blocks that a row of scales has
    int row_tiles, tiles;  // tiles of hidden rows (many rows); of both
    int K, steps;          // steps: stages of K
    int stages;
    uint32_t tmem_cols;
    int tma_stores;
    uint64_t wait_ns;      // kWaitNs, or 0: every wait gives up
    unsigned long long* timeouts;
};

struct Control {
    uint64_t ready[kMaxStages];  // a stage's operands and scales have come
    uint64_t done[kMaxStages];   // its MMAs have completed: it can be filled again
    uint64_t full[2], free[2];   // an accumulator holds a tile; every warp of the epilogue has read it
    uint64_t drained;            // every MMA of the CTA has completed
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(Control) <= kBarBytes, "");

// A whole warp waits for the phase of `bar` with the given parity, for `ns` at most.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint64_t ns)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || mbar_wait_warp(bar, parity, now_ns() + ns);
}

// Tiles of scales of 128 rows in a stage.
template <int kBlock>
constexpr int kStageTiles = kBK / (4 * kBlock);

// e2m1 A and B, both K-major; scales e4m3 (blocks of 16) or powers of two (32), of which blocks of 32 take two of a
// word's four bytes: `half` says which.
template <int kBlock>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int half)
{
    return (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (kBlock == 32 ? 1u << 23 : 0u) | (uint32_t(M >> 4) << 24) |
           (uint32_t(2 * half) << 4) | (uint32_t(2 * half) << 29);
}

// A tile of scales in shared memory: 32 rows of 16 bytes, 8 rows to 128 bytes.
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr)
{
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}

// To four columns of tensor memory, the same in all four quarters of its lanes. In order with the MMAs that the
// thread issues after it.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc_scales(smem)) : "memory");
}

template <int kBlock>
__device__ __forceinline__ void mma_micro(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                          uint32_t accumulate)
{
    if (kBlock == 16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// What a stage holds: M's values, N's, M's scales, N's (one tile of 128 rows after the other).
template <int kBlock, bool kFew>
struct Stage {
    static constexpr uint32_t kScales = kStageTiles<kBlock> * kScaleTile;   // of 128 rows
    static constexpr int kNTiles = kFew ? 1 : kWideN / 128;                  // of 128 rows of N
    static __host__ __device__ constexpr uint32_t bytes(int NT)
    {
        return kABytes + uint32_t(NT) * kRowBytes + (1 + kNTiles) * kScales;
    }
    static constexpr int kColsA = kStageTiles<kBlock> * 4, kColsB = kColsA * kNTiles;  // of tensor memory
};

// Tile t: its first rows of M and of N. (Of many rows, tiles that follow one
// another have the same weight rows, which are then in L2.)
template <bool kFew>
__device__ __forceinline__ void tile_at(const Params& P, int t, int& m, int& n)
{
    m = kFew ? t * kBM : t % P.row_tiles * kBM;
    n = kFew ? 0 : t / P.row_tiles * kWideN;
}

template <int kBlock, bool kFew>
__device__ __forceinline__ void produce(const Params& P, Control& C, unsigned char* ring)
{
    using S = Stage<kBlock, kFew>;
    const uint32_t stages = uint32_t(P.stages), b_bytes = uint32_t(P.NT) * kRowBytes, bytes = S::bytes(P.NT);
    RingPlace s{0, 0};
    uint32_t issued = 0;
    bool ok = P.wait_ns != 0;  // 0: nothing is loaded, and the other warps' waits give up
    for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
        int m, n;
        tile_at<kFew>(P, t, m, n);
        for (int b = 0; b < P.steps; ++b) {
            ok = wait(&C.done[s.at], s.phase ^ 1u, P.wait_ns);
            if (!ok) break;
            if (elect_one()) {
                unsigned char* at = ring + s.at * bytes;
                uint64_t* bar = &C.ready[s.at];
                const int first = b * kStageTiles<kBlock>;
                const uint32_t scales = uint32_t(min(kStageTiles<kBlock>, P.k_tiles - first)) * kScaleTile;
                const int nt = min(S::kNTiles, P.n_tiles - n / 128);
                mbar_arrive_expect_tx(bar, kABytes + b_bytes + scales * uint32_t(1 + nt));
                tma_load_2d(smem_addr(at), &P.tm, b * kRowBytes, m, smem_addr(bar));
                tma_load_2d(smem_addr(at + kABytes), &P.tn, b * kRowBytes, n, smem_addr(bar));
                unsigned char* to = at + kABytes + b_bytes;
                bulk_copy_g2s(to, P.sm + (int64_t(m / 128) * P.k_tiles + first) * kScaleTile, scales, bar);
                for (int j = 0; j < nt; ++j)
                    bulk_copy_g2s(to + (1 + j) * S::kScales, P.sn + (int64_t(n / 128 + j) * P.k_tiles + first) * kScaleTile,
                                  scales, bar);
            }
            __syncwarp();
            s.next(stages);
            ++issued;
        }
    }
    if (!ok) C.gave_up = 1;
    // the last copies issued land before the CTA may exit
    for (uint32_t j = issued > stages ? issued - stages : 0; j < issued; ++j) wait(&C.ready[j % stages], j / stages & 1u, kWaitNs);
}

template <int kBlock, bool kFew>
__device__ __forceinline__ void multiply(const Params& P, Control& C, unsigned char* ring, uint32_t tmem)
{
    using S = Stage<kBlock, kFew>;
    constexpr uint32_t kAccs = kFew ? 2 : 1;
    const uint32_t cols = kFew ? uint32_t(P.NT) : uint32_t(kWideN), bytes = S::bytes(int(cols));
    const uint32_t id0 = idesc<kBlock>(kBM, int(cols), 0), id1 = idesc<kBlock>(kBM, int(cols), kBlock == 32);
    uint32_t place = 0;  // of the stage's scales
    RingPlace s{0, 0}, acc{0, 0};
    bool ok = true;
    for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
        ok = wait(&C.free[acc.at], acc.phase ^ 1u, P.wait_ns);
        if (!ok) break;
        const uint32_t d = tmem + acc.at * cols;
        for (int b = 0; b < P.steps; ++b) {
            const uint32_t at = smem_addr(ring) + s.at * bytes, scales = at + kABytes + cols * kRowBytes;
            const uint64_t da = desc_sw128(at), db = desc_sw128(at + kABytes);
            const uint32_t sa = tmem + kAccs * cols + place * uint32_t(S::kColsA + S::kColsB), sb = sa + S::kColsA;
            const int parts = min(kBK, P.K - b * kBK + kUK - 1) / kUK;  // MMAs that hold some of K
            ok = wait(&C.ready[s.at], s.phase, P.wait_ns);
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < kStageTiles<kBlock>; ++j) {
                    copy_scales(sa + 4 * j, scales + j * kScaleTile);
#pragma unroll
                    for (int i = 0; i < S::kNTiles; ++i)  // the tiles of N side by side
                        copy_scales(sb + (j * S::kNTiles + i) * 4, scales + (1 + i) * S::kScales + j * kScaleTile);
                }
#pragma unroll
                for (int k = 0; k < kBK / kUK; ++k) {
                    const int j = k * kUK / (4 * kBlock);  // tile of scales
                    if (k < parts)
                        mma_micro<kBlock>(d, da + uint64_t(2 * k), db + uint64_t(2 * k), k & 1 ? id1 : id0, sa + 4 * j,
                                          sb + j * S::kNTiles * 4, uint32_t(b | k));
                }
                mma_commit(&C.done[s.at]);
                if (b + 1 == P.steps) mma_commit(&C.full[acc.at]);
            }
            __syncwarp();
            s.next(uint32_t(P.stages));
            place ^= 1u;
        }
        acc.next(kAccs);
    }
    if (!ok) C.gave_up = 1;
    if (elect_one()) mma_commit(&C.drained);
    __syncwarp();
    wait(&C.drained, 0, kWaitNs);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <typename T, int kBlock, bool kFew>
__global__ void __launch_bounds__(kThreads, 1) micro_head_kernel(const __grid_constant__ Params P)
{
    using S = Stage<kBlock, kFew>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char* outs = ring + size_t(P.stages) * S::bytes(P.NT);
    float* row_scales = reinterpret_cast<float*>(outs + (kFew ? 0 : kOutBytes));
    Control& C = *reinterpret_cast<Control*>(reinterpret_cast<unsigned char*>(row_scales) + kRowScaleBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&C.ready[i], 1);
            mbar_init(&C.done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&C.full[i], 1);
            mbar_init(&C.free[i], kEpilogue);
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
    if (kFew && tid < kFewRows) row_scales[tid] = P.row_scale_n && tid < P.rows ? P.row_scale_n[tid] : 1.f;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = C.tmem;

    if (!kFew && warp >= kEpilogue) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 8) {
        produce<kBlock, kFew>(P, C, ring);
    } else if (warp == 9) {
        multiply<kBlock, kFew>(P, C, ring, tmem);
    } else if (warp < kEpilogue) {
        if (!kFew) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int group = warp >> 2, quarter = warp & 3;  // quarter: the tensor-memory lanes a warp may read
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
        RingPlace acc{0, 0};
        bool ok = true;
        if constexpr (kFew) {
            for (int t = int(blockIdx.x); ok && t < P.tiles; t += int(gridDim.x)) {
                const int v = t * kBM + quarter * 32 + lane;
                const float mine = P.row_scale_m && v < P.V ? P.row_scale_m[v] : 1.f;
                T* out = static_cast<T*>(P.logits) + v;
                ok = wait(&C.full[acc.at], acc.phase, P.wait_ns);
                if (!ok) break;
                fence_after_sync();
                // the groups take 16 columns in turn
                for (int c0 = 16 * group; c0 < P.NT; c0 += 32) {
                    uint32_t r[16];
                    tmem_ld16(lanes + acc.at * uint32_t(P.NT) + uint32_t(c0), r);
                    tmem_wait();
                    tmem_take16(r);
                    if (v < P.V) {
                        const int n = P.rows - c0;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (c < n) put(out + int64_t(c0 + c) * P.ldl, __uint_as_float(r[c]) * row_scales[c0 + c] * mine);
                    }
                    __syncwarp();
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&C.free[acc.at]);
                acc.next(2);
            }
        } else {
            constexpr int kCols = kWideN / 2;  // of a thread
            unsigned char* out = outs + warp * kBoxBytes;
            int turn = 0;
            for (int t = int(blockIdx.x); t < P.tiles; t += int(gridDim.x), turn ^= 1) {  // to the end even where a wait
                                                                                          // gave up: its group's barriers
                                                                                          // count on it
                int row, v;
                tile_at<false>(P, t, row, v);
                row += quarter * 32;
                v += group * kCols;
                // this group's columns' scales: the other buffer's readers are past this barrier's last
                float* scales = row_scales + turn * kWideN + group * kCols;
                const int j = quarter * 32 + lane;
                scales[j] = P.row_scale_n && v + j < P.V ? P.row_scale_n[v + j] : 1.f;
                const float mine = P.row_scale_m && row + lane < P.rows ? P.row_scale_m[row + lane] : 1.f;
                if (group == 0)
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                else
                    asm volatile("bar.sync 2, 128;" ::: "memory");
                ok = ok && wait(&C.full[0], acc.phase, P.wait_ns);
                if (ok) {
                    fence_after_sync();
                    uint32_t raw[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) tmem_ld16(lanes + uint32_t(group * kCols + c), raw + c);
                    tmem_wait();
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) tmem_take16(raw + c);
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&C.free[0]);
                    float2 sum[kCols / 2];
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        const float4 s = *reinterpret_cast<const float4*>(scales + c);
                        sum[c / 2] = make_float2(__uint_as_float(raw[c]) * mine * s.x, __uint_as_float(raw[c + 1]) * mine * s.y);
                        sum[c / 2 + 1] =
                            make_float2(__uint_as_float(raw[c + 2]) * mine * s.z, __uint_as_float(raw[c + 3]) * mine * s.w);
                    }
                    store_logits<T, kCols>(P, out, row, v, sum);
                }
                acc.next(1);
            }
            if (P.tma_stores && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        if (!ok && lane == 0) C.gave_up = 1;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
    if (tid == 0 && C.gave_up && P.timeouts) atomicAdd(P.timeouts, 1ull);
}

using Kernel = void (*)(const Params);

template <int kBlock>
Kernel kernel_of(bool few, bool bf16)
{
    return few ? bf16 ? micro_head_kernel<uint16_t, kBlock, true> : micro_head_kernel<float, kBlock, true>
               : bf16 ? micro_head_kernel<uint16_t, kBlock, false> : micro_head_kernel<float, kBlock, false>;
}

template <int kBlock>
uint32_t stage_bytes(bool few, int NT)
{
    return few ? Stage<kBlock, true>::bytes(NT) : Stage<kBlock, false>::bytes(NT);
}

}  // namespace micro_head

int micro_head_launch(const sampler_micro_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows, int64_t vocab,
                      int sms, uint64_t wait_ns, unsigned long long* timeouts, MicroHeadGrants* grants, cudaStream_t stream)
{
    using namespace micro_head;
    Params p;
    std::memset(&p, 0, sizeof p);
    const bool few = rows <= kFewRows, wide = g.block == 32;
    p.row_tiles = few ? 1 : int((rows + kBM - 1) / kBM);
    p.NT = few ? int((rows + 15) / 16 * 16) : kWideN;
    const int64_t tiles = (vocab + (few ? kBM : kWideN) - 1) / (few ? kBM : kWideN) * p.row_tiles;
    if (tiles > INT32_MAX - 65536) return SAMPLER_ERR_TOO_LARGE;
    p.tiles = int(tiles);
    p.K = int(g.hidden_dim);
    p.steps = int((g.hidden_dim + kBK - 1) / kBK);
    p.k_tiles = int(((g.hidden_dim + g.block - 1) / g.block + 3) / 4);
    const int es = dtype == SAMPLER_DTYPE_BF16 ? 2 : 4;
    const size_t stage = wide ? stage_bytes<32>(few, p.NT) : stage_bytes<16>(few, p.NT);
    const size_t own = (few ? 0 : kOutBytes) + kRowScaleBytes + kBarBytes;
    p.stages = int(std::min<size_t>(kMaxStages, (kSmemMax - 1024 - own) / stage));
    const int scale_cols = kBK / g.block * (few ? 2 : 3);  // of a stage: 4 for a tile, of M and of N
    const uint32_t cols = uint32_t((few ? 2 : 1) * p.NT + 2 * scale_cols);
    p.tmem_cols = 32;
    while (p.tmem_cols < cols) p.tmem_cols <<= 1;
    const int64_t bytes = (g.hidden_dim + 1) / 2;
    const bool maps = few ? encode_bytes(&p.tm, g.weight, vocab, bytes, g.weight_stride, kBM) &&
                                encode_bytes(&p.tn, g.hidden, rows, bytes, g.hidden_stride, p.NT)
                          : encode_bytes(&p.tm, g.hidden, rows, bytes, g.hidden_stride, kBM) &&
                                encode_bytes(&p.tn, g.weight, vocab, bytes, g.weight_stride, kWideN);
    if (!maps) return SAMPLER_ERR_CUDA;
    const auto *hs = static_cast<const unsigned char*>(g.hidden_scale), *ws = static_cast<const unsigned char*>(g.weight_scale);
    p.sm = few ? ws : hs;
    p.sn = few ? hs : ws;
    p.row_scale_m = few ? g.weight_row_scale : g.hidden_row_scale;
    p.row_scale_n = few ? g.hidden_row_scale : g.weight_row_scale;
    p.m_tiles = int(((few ? vocab : rows) + 127) / 128);
    p.n_tiles = int(((few ? rows : vocab) + 127) / 128);
    p.logits = logits;
    p.ldl = ldl;
    p.tma_stores = !few && ldl * es % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    if (p.tma_stores && !encode_logits(&p.to, logits, dtype, rows, vocab, ldl)) return SAMPLER_ERR_CUDA;
    p.rows = int(rows);
    p.V = int(vocab);
    p.wait_ns = wait_ns;
    p.timeouts = timeouts;
    const bool bf16 = dtype == SAMPLER_DTYPE_BF16;
    const Kernel kernel = wide ? kernel_of<32>(few, bf16) : kernel_of<16>(few, bf16);
    const size_t smem = 1024 + size_t(p.stages) * stage + own;
    // the limit belongs to the function, for all handles and threads: always the same one
    bool& granted = grants->granted[wide][few][bf16];
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
