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
// A call's tiles have one of three forms.
//   few    transposed, for a decode step: 128 weight rows (M) by all hidden rows (N),
//          and the weight's bytes are all the time. The lanes are then neighbouring
//          tokens, and the logits are stored as they lie.
//   many   128 hidden rows (M) by 256 weight rows (N).
//   pairs  two CTAs of a cluster take 256 hidden rows by 256 weight rows together
//          (tcgen05 with cta_group::2): each holds the values of its own 128 hidden
//          rows and of half of the weight rows, and all of the weight's scales, so that
//          an SM takes 38 KB a stage from L2 in place of 54 and five stages fit in
//          place of three. The first CTA's barriers count the copies of both, its
//          thread issues for both, and its commits arrive in both. 4096 x 128000 x 4096
//          bf16, codes and scales at random: 655 us (6.6 PFLOP/s, 0.86 of four times the
//          measured bf16 rate) against 890 of many; with scales that are all alike 639
//          and 886. Power has its share in that.
// Of many rows one accumulator and the scales leave no room for a second: the epilogue
// reads it into registers first and gives it back, and scales, rounds and stores
// (through shared memory and the TMA engine) under the next tile's products.
//
// Persistent, one CTA an SM; warp roles:
//   warps 0-7  the epilogue: two groups of four warps, a warp 32 of the tile's lanes;
//   warp 8     loads the operand ring by TMA tiles, the scales' among them;
//   warp 9     owns the tensor memory and issues the copies of scales and the MMAs
//              (of a pair the first CTA's).
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

// How a call's tiles are taken (see above).
enum Form : int { kFew, kMany, kPair };

constexpr int kBM = 128;                     // rows of M in a CTA, and of a tile of scales
constexpr int kBK = 256;                     // K of a stage: 128 bytes a row
constexpr int kRowBytes = kBK / 2;
constexpr int kUK = 64;                      // K of one tcgen05.mma
constexpr int kThreads = 384;
constexpr int kEpilogue = 8;                 // warps
constexpr int kFewRegs = 40, kManyRegs = 232;  // many rows: 128 * 40 + 256 * 232 <= 384 * 168
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
    CUtensorMap tsm, tsn;  // their scales [tiles of rows, tiles of 4 blocks, a tile's 512 bytes]
    const float *row_scale_m, *row_scale_n;   // NULL = 1
    void* logits;
    int64_t ldl;
    int rows, V, NT;
    int row_tiles, tiles;  // tiles of hidden rows (many rows); of both
    int K, steps;          // steps: stages of K
    int stages;
    uint32_t tmem_cols;
    int tma_stores;
    uint64_t wait_ns;      // kWaitNs, or 0: every wait gives up
    unsigned long long* timeouts;
};

struct Control {
    uint64_t ready[kMaxStages];  // a stage's operands and scales have come (of a pair: those of both CTAs, at the first one's)
    uint64_t done[kMaxStages];   // its MMAs have completed: it can be filled again
    uint64_t full[2], free[2];   // an accumulator holds a tile; every warp of the epilogue (of both CTAs) has read it
    uint64_t drained;            // every MMA of the CTA has completed
    uint32_t tmem;
    uint32_t issued;             // stages that the CTA has loaded
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

// To four columns of tensor memory, the same in all four quarters of its lanes (of a pair: in both CTAs, each from its
// own shared memory). In order with the MMAs that the thread issues after it.
template <Form kForm>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem)
{
    if (kForm == kPair)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc_scales(smem)) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc_scales(smem)) : "memory");
}

// Arrives on a barrier once all that the thread has issued has completed; of a pair on the one at its place in both CTAs.
template <Form kForm>
__device__ __forceinline__ void commit(uint64_t* bar)
{
    if (kForm == kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         smem_addr(bar)),
                     "h"(uint16_t(3))
                     : "memory");
    else
        mma_commit(bar);
}

// Arrives on a barrier of the pair's first CTA. What the arrival hands over is tensor memory that completed loads have
// read, ordered by the tcgen05 fences on both sides; no memory that a thread wrote, for which it would have to release at
// the cluster's scope (that waits for the warp's stores of logits: 720 us in place of 632, scales that are all alike).
__device__ __forceinline__ void arrive_first(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(dsmem_map(smem_addr(bar), 0)) : "memory");
}

// A tile of an operand or of its scales into this CTA's shared memory, and its bytes to a barrier, a pair's at the
// first CTA's.
template <Form kForm>
__device__ __forceinline__ void load_values(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    if (kForm == kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        tma_load_2d(dst, map, x, y, bar);
}

template <Form kForm>
__device__ __forceinline__ void load_scales(uint32_t dst, const CUtensorMap* map, int k_tile, int row_tile, uint32_t bar)
{
    if (kForm == kPair)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], "
            "[%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k_tile), "r"(row_tile), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(k_tile), "r"(row_tile), "r"(bar)
            : "memory");
}

template <int kBlock, Form kForm>
__device__ __forceinline__ void mma_micro(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                          uint32_t accumulate)
{
    if (kBlock == 16 && kForm != kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else if (kForm != kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else if (kBlock == 16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// What a stage of a CTA holds: M's values, N's, M's scales, N's (one tile of 128 rows after the other). A pair's CTAs
// each hold half of N's values, and all of its scales.
template <int kBlock, Form kForm>
struct Stage {
    static constexpr uint32_t kScales = kStageTiles<kBlock> * kScaleTile;   // of 128 rows
    static constexpr int kNTiles = kForm == kFew ? 1 : kWideN / 128;         // of 128 rows of N
    static __host__ __device__ constexpr uint32_t b_bytes(int NT) { return uint32_t(kForm == kPair ? NT / 2 : NT) * kRowBytes; }
    static __host__ __device__ constexpr uint32_t bytes(int NT) { return kABytes + b_bytes(NT) + (1 + kNTiles) * kScales; }
    static constexpr int kColsA = kStageTiles<kBlock> * 4, kColsB = kColsA * kNTiles;  // of tensor memory
};

// The tiles of a CTA or pair: the first, and how far apart.
template <Form kForm>
__device__ __forceinline__ int first_tile()
{
    return kForm == kPair ? int(blockIdx.x) / 2 : int(blockIdx.x);
}

template <Form kForm>
__device__ __forceinline__ int tile_step()
{
    return kForm == kPair ? int(gridDim.x) / 2 : int(gridDim.x);
}

// Tile t: its first rows of M (in this CTA) and of N. (Of many rows, tiles that follow one another have the same weight
// rows, which are then in L2.)
template <Form kForm>
__device__ __forceinline__ void tile_at(const Params& P, int t, int& m, int& n)
{
    m = kForm == kFew ? t * kBM : t % P.row_tiles * (kForm == kPair ? 2 * kBM : kBM);
    if (kForm == kPair) m += int(cluster_ctarank()) * kBM;
    n = kForm == kFew ? 0 : t / P.row_tiles * kWideN;
}

template <int kBlock, Form kForm>
__device__ __forceinline__ void produce(const Params& P, Control& C, unsigned char* ring)
{
    using S = Stage<kBlock, kForm>;
    const uint32_t stages = uint32_t(P.stages), b_bytes = S::b_bytes(P.NT), bytes = S::bytes(P.NT);
    const bool first = kForm != kPair || cluster_ctarank() == 0;
    const int half = first ? 0 : kWideN / 2;  // of N's values
    RingPlace s{0, 0};
    uint32_t issued = 0;
    bool ok = P.wait_ns != 0;  // 0: nothing is loaded, and the other warps' waits give up
    for (int t = first_tile<kForm>(); ok && t < P.tiles; t += tile_step<kForm>()) {
        int m, n;
        tile_at<kForm>(P, t, m, n);
        for (int b = 0; b < P.steps; ++b) {
            ok = wait(&C.done[s.at], s.phase ^ 1u, P.wait_ns);
            if (!ok) break;
            if (elect_one()) {
                const uint32_t at = smem_addr(ring) + s.at * bytes, scales = at + kABytes + b_bytes;
                uint32_t bar = smem_addr(&C.ready[s.at]);
                if (first) mbar_arrive_expect_tx(&C.ready[s.at], kForm == kPair ? 2 * bytes : bytes);
                if (kForm == kPair) bar = dsmem_map(bar, 0);
                load_values<kForm>(at, &P.tm, b * kRowBytes, m, bar);
                load_values<kForm>(at + kABytes, &P.tn, b * kRowBytes, n + half, bar);
                load_scales<kForm>(scales, &P.tsm, b * kStageTiles<kBlock>, m / 128, bar);
                load_scales<kForm>(scales + S::kScales, &P.tsn, b * kStageTiles<kBlock>, n / 128, bar);
            }
            __syncwarp();
            s.next(stages);
            ++issued;
        }
    }
    if (!ok) C.gave_up = 1;
    C.issued = issued;
    // the last copies issued land before the CTA may exit
    if (first)
        for (uint32_t j = issued > stages ? issued - stages : 0; j < issued; ++j) wait(&C.ready[j % stages], j / stages & 1u, kWaitNs);
}

// A pair's copies of its second CTA land at the first one's barriers: after a wait that gave up the second may have
// issued some that the first did not count on.
template <int kBlock>
__device__ __forceinline__ void land(const Params& P, Control& C)
{
    const uint32_t stages = uint32_t(P.stages), theirs = dsmem_ld_u32(dsmem_map(smem_addr(&C.issued), 1));
    for (uint32_t j = C.issued; j < theirs; ++j) {
        if (elect_one()) mbar_arrive_expect_tx(&C.ready[j % stages], Stage<kBlock, kPair>::bytes(kWideN));
        __syncwarp();
        wait(&C.ready[j % stages], j / stages & 1u, kWaitNs);
    }
}

template <int kBlock, Form kForm>
__device__ __forceinline__ void multiply(const Params& P, Control& C, unsigned char* ring, uint32_t tmem)
{
    using S = Stage<kBlock, kForm>;
    constexpr uint32_t kAccs = kForm == kFew ? 2 : 1;
    const uint32_t cols = kForm == kFew ? uint32_t(P.NT) : uint32_t(kWideN), bytes = S::bytes(int(cols)), b_bytes = S::b_bytes(int(cols));
    constexpr int kM = kForm == kPair ? 2 * kBM : kBM;
    const uint32_t id0 = idesc<kBlock>(kM, int(cols), 0), id1 = idesc<kBlock>(kM, int(cols), kBlock == 32);
    uint32_t place = 0;  // of the stage's scales
    RingPlace s{0, 0}, acc{0, 0};
    bool ok = true;
    for (int t = first_tile<kForm>(); ok && t < P.tiles; t += tile_step<kForm>()) {
        ok = wait(&C.free[acc.at], acc.phase ^ 1u, P.wait_ns);
        if (!ok) break;
        const uint32_t d = tmem + acc.at * cols;
        for (int b = 0; b < P.steps; ++b) {
            const uint32_t at = smem_addr(ring) + s.at * bytes, scales = at + kABytes + b_bytes;
            const uint64_t da = desc_sw128(at), db = desc_sw128(at + kABytes);
            const uint32_t sa = tmem + kAccs * cols + place * uint32_t(S::kColsA + S::kColsB), sb = sa + S::kColsA;
            const int parts = min(kBK, P.K - b * kBK + kUK - 1) / kUK;  // MMAs that hold some of K
            ok = wait(&C.ready[s.at], s.phase, P.wait_ns);
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < kStageTiles<kBlock>; ++j) {
                    copy_scales<kForm>(sa + 4 * j, scales + j * kScaleTile);
#pragma unroll
                    for (int i = 0; i < S::kNTiles; ++i)  // the tiles of N side by side
                        copy_scales<kForm>(sb + (j * S::kNTiles + i) * 4, scales + (1 + i) * S::kScales + j * kScaleTile);
                }
#pragma unroll
                for (int k = 0; k < kBK / kUK; ++k) {
                    const int j = k * kUK / (4 * kBlock);  // tile of scales
                    if (k < parts)
                        mma_micro<kBlock, kForm>(d, da + uint64_t(2 * k), db + uint64_t(2 * k), k & 1 ? id1 : id0, sa + 4 * j,
                                                 sb + j * S::kNTiles * 4, uint32_t(b | k));
                }
                commit<kForm>(&C.done[s.at]);
                if (b + 1 == P.steps) commit<kForm>(&C.full[acc.at]);
            }
            __syncwarp();
            s.next(uint32_t(P.stages));
            place ^= 1u;
        }
        acc.next(kAccs);
    }
    if (!ok) C.gave_up = 1;
    if (elect_one()) commit<kForm>(&C.drained);
    __syncwarp();
    wait(&C.drained, 0, kWaitNs);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

template <typename T, int kBlock, Form kForm>
__global__ void __launch_bounds__(kThreads, 1) micro_head_kernel(const __grid_constant__ Params P)
{
    using S = Stage<kBlock, kForm>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char* outs = ring + size_t(P.stages) * S::bytes(P.NT);
    float* row_scales = reinterpret_cast<float*>(outs + (kForm == kFew ? 0 : kOutBytes));
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
            mbar_init(&C.free[i], kForm == kPair ? 2 * kEpilogue : kEpilogue);
        }
        mbar_init(&C.drained, 1);
        C.gave_up = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tm)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.tn)) : "memory");
    }
    if (warp == 9) {
        if (kForm == kPair) {
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
    if (kForm == kFew && tid < kFewRows) row_scales[tid] = P.row_scale_n && tid < P.rows ? P.row_scale_n[tid] : 1.f;
    fence_before_sync();
    __syncthreads();
    if (kForm == kPair) cluster_sync();  // the other CTA's barriers and tensor memory are there, too
    fence_after_sync();
    const uint32_t tmem = C.tmem;

    if (kForm != kFew && warp >= kEpilogue) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 8) {
        produce<kBlock, kForm>(P, C, ring);
    } else if (warp == 9) {
        if (kForm != kPair || cluster_ctarank() == 0) multiply<kBlock, kForm>(P, C, ring, tmem);
    } else if (warp < kEpilogue) {
        if (kForm != kFew) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int group = warp >> 2, quarter = warp & 3;  // quarter: the tensor-memory lanes a warp may read
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
        RingPlace acc{0, 0};
        bool ok = true;
        if constexpr (kForm == kFew) {
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
            for (int t = first_tile<kForm>(); t < P.tiles; t += tile_step<kForm>(), turn ^= 1) {  // to the end even where a wait
                                                                                          // gave up: its group's barriers
                                                                                          // count on it
                int row, v;
                tile_at<kForm>(P, t, row, v);
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
                    if (lane == 0) {
                        if (kForm == kPair)
                            arrive_first(&C.free[0]);
                        else
                            mbar_arrive(&C.free[0]);
                    }
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
    if (kForm == kPair) {  // neither CTA's memory is used by the other's MMAs, copies and arrivals any more
        cluster_sync();
        if (warp == 8 && cluster_ctarank() == 0) land<kBlock>(P, C);
        if (warp == 9 && cluster_ctarank() == 1) wait(&C.drained, 0, kWaitNs);
        __syncwarp();
        cluster_sync();
    }
    fence_after_sync();
    if (warp == 9) {
        if (kForm == kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
    }
    if (tid == 0 && C.gave_up && P.timeouts) atomicAdd(P.timeouts, 1ull);
}

using Kernel = void (*)(const Params);

template <int kBlock>
Kernel kernel_of(Form form, bool bf16)
{
    switch (form) {
    case kFew: return bf16 ? micro_head_kernel<uint16_t, kBlock, kFew> : micro_head_kernel<float, kBlock, kFew>;
    case kMany: return bf16 ? micro_head_kernel<uint16_t, kBlock, kMany> : micro_head_kernel<float, kBlock, kMany>;
    default: return bf16 ? micro_head_kernel<uint16_t, kBlock, kPair> : micro_head_kernel<float, kBlock, kPair>;
    }
}

template <int kBlock>
uint32_t stage_bytes(Form form, int NT)
{
    return form == kFew ? Stage<kBlock, kFew>::bytes(NT) : form == kMany ? Stage<kBlock, kMany>::bytes(NT) : Stage<kBlock, kPair>::bytes(NT);
}

// The form of a call's tiles, by what they take one after the other. Measured (bf16 logits, 16 a block, weights in L2
// where they fit; us):
//   rows x vocabulary x hidden     few  many  pairs
//   64 x 128000 x 4096            55.4  58.6   58.6     the weight's bytes
//   32 x 32000 x 4096             16.3  17.6   21.5
//   64 x 32000 x 4096             17.6  14.6   19.2     125 wide tiles are one turn of the SMs, 250 narrow ones two
//   128 x 48000 x 2048            19.2  16.3   19.1     (two turns against three: left to few, 15.5 to 16.4 at 64 rows, and
//                                                        24.6 to 24.6 at 128 where the weight comes from HBM)
//   300 x 42000 x 1024                  17.5   19.4     little to multiply: a pair starts and ends later
//   300 x 42000 x 2112                  27.8   28.3
//   512 x 32000 x 4096                  43.0   36.0
//   4096 x 128000 x 1024               331    253
//   4096 x 128000 x 4096               890    655      (codes and scales at random)
// With the weight from HBM (the clock's step is 2 us):
//   128 x 128000 x 1024           36.9  26.6   30.8     four stages of K: the logits' stores of a narrow tile, by element,
//   96 x 100000 x 1024            28.7  22.5   26.6      take longer than its products
//   128 x 42000 x 1024            20.5  16.4   18.4
//   64 x 128000 x 1024            28.7  24.6   28.7     (left to few)
//   128 x 16000 x 1024            12.3  12.3   12.3
//   128 x 128000 x 2048           41.1  41.0   45.1
//   128 x 128000 x 4096           67.6  69.6   69.7
Form form_of(int64_t rows, int64_t vocab, int64_t hidden, int sms)
{
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    if (rows <= kFewRows) {
        const int64_t narrow = up(up(vocab, kBM), sms), wide = up(up(vocab, kWideN), sms);  // turns
        if (rows > kFewRows / 2 && hidden <= 4 * kBK && narrow > 1) return kMany;
        return rows > 32 && 2 * wide <= narrow && narrow <= 4 ? kMany : kFew;
    }
    const int64_t turns = up(up(rows, 2 * kBM) * up(vocab, kWideN), sms / 2);
    return sms % 2 == 0 && turns * up(hidden, kBK) >= 24 ? kPair : kMany;
}

// Tensor map of the scales of `rows` rows, boxes of `tiles` tiles of blocks by `row_tiles` tiles of rows; tiles behind
// the last read as zero.
bool encode_scales(CUtensorMap* map, const void* base, int64_t rows, int64_t k_tiles, int tiles, int row_tiles)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {kScaleTile / 4, cuuint64_t(k_tiles), cuuint64_t((rows + 127) / 128)};
    const cuuint64_t strides[2] = {kScaleTile, cuuint64_t(k_tiles) * kScaleTile};
    const cuuint32_t box[3] = {kScaleTile / 4, cuuint32_t(tiles), cuuint32_t(row_tiles)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace micro_head

int micro_head_launch(const sampler_micro_head_t& g, void* logits, int dtype, int64_t ldl, int64_t rows, int64_t vocab,
                      int sms, uint64_t wait_ns, unsigned long long* timeouts, MicroHeadGrants* grants, cudaStream_t stream)
{
    using namespace micro_head;
    Params p;
    std::memset(&p, 0, sizeof p);
    const Form form = form_of(rows, vocab, g.hidden_dim, sms);
    const bool few = form == kFew, wide = g.block == 32;
    const int m_rows = form == kPair ? 2 * kBM : kBM;
    p.row_tiles = few ? 1 : int((rows + m_rows - 1) / m_rows);
    p.NT = few ? int((rows + 15) / 16 * 16) : kWideN;
    const int64_t tiles = (vocab + (few ? kBM : kWideN) - 1) / (few ? kBM : kWideN) * p.row_tiles;
    if (tiles > INT32_MAX - 65536) return SAMPLER_ERR_TOO_LARGE;
    p.tiles = int(tiles);
    p.K = int(g.hidden_dim);
    p.steps = int((g.hidden_dim + kBK - 1) / kBK);
    const int es = dtype == SAMPLER_DTYPE_BF16 ? 2 : 4;
    const size_t stage = wide ? stage_bytes<32>(form, p.NT) : stage_bytes<16>(form, p.NT);
    const size_t own = (few ? 0 : kOutBytes) + kRowScaleBytes + kBarBytes;
    p.stages = int(std::min<size_t>(kMaxStages, (kSmemMax - 1024 - own) / stage));
    const int scale_cols = kBK / g.block * (few ? 2 : 3);  // of a stage: 4 for a tile, of M and of N
    const uint32_t cols = uint32_t((few ? 2 : 1) * p.NT + 2 * scale_cols);
    p.tmem_cols = 32;
    while (p.tmem_cols < cols) p.tmem_cols <<= 1;
    const int64_t bytes = (g.hidden_dim + 1) / 2, k_tiles = ((g.hidden_dim + g.block - 1) / g.block + 3) / 4;
    const int wide_rows = form == kPair ? kWideN / 2 : kWideN, stage_tiles = kBK / (4 * g.block);
    const bool maps =
        few ? encode_bytes(&p.tm, g.weight, vocab, bytes, g.weight_stride, kBM) &&
                  encode_bytes(&p.tn, g.hidden, rows, bytes, g.hidden_stride, p.NT) &&
                  encode_scales(&p.tsm, g.weight_scale, vocab, k_tiles, stage_tiles, 1) &&
                  encode_scales(&p.tsn, g.hidden_scale, rows, k_tiles, stage_tiles, 1)
            : encode_bytes(&p.tm, g.hidden, rows, bytes, g.hidden_stride, kBM) &&
                  encode_bytes(&p.tn, g.weight, vocab, bytes, g.weight_stride, wide_rows) &&
                  encode_scales(&p.tsm, g.hidden_scale, rows, k_tiles, stage_tiles, 1) &&
                  encode_scales(&p.tsn, g.weight_scale, vocab, k_tiles, stage_tiles, kWideN / 128);
    if (!maps) return SAMPLER_ERR_CUDA;
    p.row_scale_m = few ? g.weight_row_scale : g.hidden_row_scale;
    p.row_scale_n = few ? g.hidden_row_scale : g.weight_row_scale;
    p.logits = logits;
    p.ldl = ldl;
    p.tma_stores = !few && ldl * es % 16 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
    if (p.tma_stores && !encode_logits(&p.to, logits, dtype, rows, vocab, ldl)) return SAMPLER_ERR_CUDA;
    p.rows = int(rows);
    p.V = int(vocab);
    p.wait_ns = wait_ns;
    p.timeouts = timeouts;
    const bool bf16 = dtype == SAMPLER_DTYPE_BF16;
    const Kernel kernel = wide ? kernel_of<32>(form, bf16) : kernel_of<16>(form, bf16);
    const size_t smem = 1024 + size_t(p.stages) * stage + own;
    // the limit belongs to the function, for all handles and threads: always the same one
    bool& granted = grants->granted[wide][form][bf16];
    if (!granted && cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemMax)) != cudaSuccess)
        return SAMPLER_ERR_CUDA;
    granted = true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(form == kPair ? 2 * std::min(sms / 2, p.tiles) : std::min(sms, p.tiles)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {2u, 1u, 1u};
    cfg.attrs = &attr;
    cfg.numAttrs = form == kPair ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
