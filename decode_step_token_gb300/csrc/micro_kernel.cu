// micro_kernel.cu -- rows to microscaled 4 bits (e2m1 values with a scale for each
// block of 16 or 32) and back.
//
// Every step is exact or one rounding, so that the codes follow from the
// definition bit for bit: the row's scale is a power of two, a block's scale has
// at most four digits, and a quotient is on the exact one's side of every tie
// between codes. (A product with the rounded reciprocal would put many of the
// quotients that are such a tie on a side: bf16 values over a scale of four digits
// often are. For bf16, not for fp32, a product with the reciprocal rounded up, rounded
// towards 0, has every code right; not built.)
//
// A block's codes need the block's largest magnitude and, for blocks of 16, the
// row's, so a row stays in registers: 16 neighbouring values in each thread, one
// to four times, 4 to 256 threads to a row. Rows of more than 16384 values are
// read twice where the row's largest is needed.
// Scales are laid out as the tensor cores take them: 512 bytes for 128 rows by 4
// blocks, (row % 32) * 16 + (row / 32 % 4) * 4 + block % 4. The four bytes of a
// row are stored as one word.
//
// What bounds both ways is memory, for blocks of 16 the instructions too: 128000 x
// 4096 bf16 takes 220 us with blocks of 32 and 300 of 16 (0.89 and 0.66 of the copy
// rate), and 222 back from either (0.88). A value at a time as fp32, with one row
// in hand, they were 287 and 423; a vector a thread back, 369 and 386. Rows of 1000
// (20000 of them: 20 and 25 us, 0.37 and 0.30) leave half of a group's threads without
// a chunk.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"

namespace dst {
namespace micro {

constexpr int kThreads = 256;
constexpr int kPer = 16;                     // values of a thread
constexpr int kVectors = 4;                  // of a thread of the rows read back
constexpr float kLeast = 7.888609052e-31f;   // 2^-100: keeps a row's scale and its quotients normal
constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ float power(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// The exponent of the least power of two p with m <= f p, from the bits of m, for an f of 1 to 2 with the mantissa
// bits `f`.
__device__ __forceinline__ int least_power(uint32_t m, uint32_t f)
{
    return int(m >> 23) - 127 + ((m & 0x7fffffu) > f ? 1 : 0);
}

// Eight values (four pairs) to eight codes, the first in the lowest four bits; ties to even, beyond 6 to 6.
__device__ __forceinline__ uint32_t codes8(const unsigned long long* q)
{
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("mov.b64 {%0, %1}, %2;" : "=f"(x[2 * j]), "=f"(x[2 * j + 1]) : "l"(q[j]));
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// A value to its e4m3 code, and that code's value.
__device__ __forceinline__ uint32_t e4m3_code(float x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code)
{
    float y;
    asm("{\n\t.reg .b32 w;\n\t.reg .b16 lo, hi;\n\tcvt.rn.f16x2.e4m3x2 w, %1;\n\tmov.b32 {lo, hi}, w;\n\t"
        "cvt.f32.f16 %0, lo;\n\t}"
        : "=f"(y)
        : "h"(uint16_t(code)));
    return y;
}

// The value of a block's scale; the codes 0x7f (blocks of 16) and 0xff (of 32) are NaN.
template <int kBlock>
__device__ __forceinline__ float scale_value(uint32_t code)
{
    if (kBlock == 16) return e4m3_value(code);
    uint32_t w;  // as bf16, which has all of them
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(w) : "h"(uint16_t(code)));
    return __uint_as_float(w << 16);
}

// 16 values of a row as they lie in memory.
template <typename T>
struct Raw {
    static constexpr int kWords = int(sizeof(T)) * kPer / 4;
    uint32_t w[kWords];
};

// The first `count` of 16 values, zeros after them. Values that do not lie in whole vectors are cut out of the 16-byte
// vectors that hold them, and never out of one that holds none (20000 rows of 1001 bf16: 25 us for 31 one by one; of
// fp32 31 for 46, though 4001 of 5003 take 35 for 31).
template <typename T>
__device__ __forceinline__ void load16(Raw<T>& x, const T* p, int count, bool vec)
{
    constexpr int kWords = Raw<T>::kWords;
    if (vec && count == kPer) {
#pragma unroll
        for (int j = 0; j < kWords / 4; ++j) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + j);
            x.w[4 * j] = v.x;
            x.w[4 * j + 1] = v.y;
            x.w[4 * j + 2] = v.z;
            x.w[4 * j + 3] = v.w;
        }
        return;
    }
    const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
    const int end = count > 0 ? int(off) + count * int(sizeof(T)) : 0;
    uint32_t w[kWords + 4];
#pragma unroll
    for (int j = 0; j <= kWords / 4; ++j) {
        const uint4 v = 16 * j < end ? __ldg(from + j) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * j] = v.x;
        w[4 * j + 1] = v.y;
        w[4 * j + 2] = v.z;
        w[4 * j + 3] = v.w;
    }
    if (off & 8u) {
#pragma unroll
        for (int j = 0; j < kWords + 2; ++j) w[j] = w[j + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int j = 0; j < kWords + 1; ++j) w[j] = w[j + 1];
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) x.w[j] = sizeof(T) == 2 ? __funnelshift_r(w[j], w[j + 1], (off & 2u) * 8u) : w[j];
    if (count < kPer) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const int left = count * int(sizeof(T)) / 2 - 2 * j;  // halves of the word
            x.w[j] = left >= 2 ? x.w[j] : left == 1 ? x.w[j] & 0xffffu : 0u;
        }
    }
}

// Two neighbouring values as a pair of fp32.
using Two = unsigned long long;

__device__ __forceinline__ Two two(uint32_t a, uint32_t b)
{
    Two y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "r"(a), "r"(b));
    return y;
}

__device__ __forceinline__ Two pair_at(const Raw<float>& x, int j) { return two(x.w[2 * j], x.w[2 * j + 1]); }
__device__ __forceinline__ Two pair_at(const Raw<uint16_t>& x, int j) { return two(x.w[j] << 16, x.w[j] & 0xffff0000u); }

__device__ __forceinline__ Two times(Two a, Two b)
{
    Two y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

__device__ __forceinline__ Two times_add(Two a, Two b, Two c)
{
    Two y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}

// The largest magnitude of 16 values as fp32 bits: kInf or more where one is not finite.
__device__ __forceinline__ uint32_t largest(const Raw<float>& x)
{
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, x.w[j] & 0x7fffffffu);
    return m;
}

__device__ __forceinline__ uint32_t largest(const Raw<uint16_t>& x)
{
    uint32_t m = x.w[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < 8; ++j) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(x.w[j] & 0x7fff7fffu));
    return max(m & 0xffff0000u, m << 16);
}

__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x / d by a reciprocal that may be a unit off, with one step on the remainder (Newton): off by 2^-45 before it is
// rounded. What it is rounded to, a code of few digits, is then the exact quotient's: a tie between two codes comes out as
// itself, and x and d, of 24 digits and of four, have quotients on either side of one that are 2^-25 of it away at least.
__device__ __forceinline__ float quotient(float x, float d, float inv)
{
    const float y = x * inv;
    return fmaf(fmaf(-d, y, x), inv, y);
}

// What a call's shape makes of it. group: threads to a row.
struct Plan {
    int group, chunks, tiles;  // chunks of 16 values, and tiles of scales, in a row
    int64_t padded;            // rows, rounded up to whole tiles
    bool vec_in, vec_out;
};

// The codes of one chunk and its block's scale code, given the block's largest magnitude and (blocks of 16) the row's
// scale 2^g.
template <typename T, int kBlock>
__device__ __forceinline__ uint2 encode(const Raw<T>& x, uint32_t most, int g, uint32_t& code)
{
    Two q[kPer / 2];
    const bool finite = most < kInf;
    if (kBlock == 32) {
        const int e = max(least_power(most, 0x400000u) - 2, -127);  // m <= 1.5 * 4 * 2^e
        code = finite ? uint32_t(e + 127) : 0xffu;
        const uint32_t up = __float_as_uint(power(-max(min(e, 126), -127)));  // its reciprocal: a product with it is exact
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) q[j] = times(pair_at(x, j), two(up, up));
    } else {
        // (m / 2^g, exact where it is not far below the least scale, over 6)
        code = finite ? e4m3_code(quotient(__uint_as_float(most) * power(-g), 6.f, 1.f / 6.f)) : 0x7fu;
        const float unit = (finite ? e4m3_value(code) : 0.f) * power(g);
        const uint32_t i = __float_as_uint(unit > 0.f ? -reciprocal(unit) : -0.f), u = __float_as_uint(unit);
        const Two less = two(i, i), d = two(u, u);
        // as quotient(), two at a time, and with the other sign: the remainder of -0 is 0, which the last step adds as -0
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
            const Two v = pair_at(x, j), y = times(v, less);
            q[j] = times_add(times_add(y, d, v), less, y);
        }
    }
    const uint32_t keep = finite ? 0xffffffffu : 0u, sign = kBlock == 16 ? 0x88888888u : 0u;
    return make_uint2((codes8(q) ^ sign) & keep, (codes8(q + 4) ^ sign) & keep);
}

// Store a chunk's codes: 8 bytes where they lie so, else the `bytes` that belong to the row.
__device__ __forceinline__ void put_codes(uint8_t* to, uint2 c, int bytes, bool vec)
{
    if (vec && bytes == 8) {
        *reinterpret_cast<uint2*>(to) = c;
    } else {
        const uint64_t w = uint64_t(c.y) << 32 | c.x;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < bytes) to[j] = uint8_t(w >> 8 * j);
    }
}

__device__ __forceinline__ int64_t scale_word(int64_t row, int tile, int tiles)
{
    return (row / 128 * tiles + tile) * 128 + (row % 32) * 4 + row / 32 % 4;
}

// kChunks: of a row in a thread, in registers; 0: any number, read twice where blocks are of 16. kRows: that a group of
// threads has in hand.
template <typename T, int kBlock, int kChunks, int kRows>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const sampler_micro_t q, const Plan plan)
{
    constexpr int kHeld = kChunks ? kChunks : 1;
    constexpr int kOfTile = 4 * kBlock / kPer;  // chunks that one word of scales belongs to
    const int group = plan.group, t = threadIdx.x & (group - 1), groups = kThreads / group;
    const int64_t row0 = int64_t(blockIdx.x) * (groups * kRows) + threadIdx.x / group;  // rows of a group: `groups` apart
    uint32_t* words = static_cast<uint32_t*>(q.scales);
    Raw<T> x[kRows][kHeld];
    auto load = [&](int r, int k, int chunk) {
        const int64_t row = row0 + r * groups, left = row < q.rows ? q.cols - int64_t(chunk) * kPer : 0;
        const T* src = static_cast<const T*>(q.src) + (row < q.rows ? row * q.src_stride : 0) + int64_t(chunk) * kPer;
        load16<T>(x[r][k], src, int(max(int64_t(0), min(int64_t(kPer), left))), plan.vec_in);
    };
    int g[kRows] = {};
    uint32_t most[kRows][kHeld];
    if (kChunks) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < kHeld; ++k) load(r, k, t + k * group);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                most[r][k] = largest(x[r][k]);
                if (kBlock == 32) most[r][k] = max(most[r][k], __shfl_xor_sync(0xffffffffu, most[r][k], 1));
            }
    }
    if (kBlock == 16) {
        // each row's largest, of its blocks without a NaN or an infinity
        __shared__ uint32_t part[kRows][kThreads / 32];
        uint32_t m[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            m[r] = __float_as_uint(kLeast);
            if (kChunks) {
#pragma unroll
                for (int k = 0; k < kHeld; ++k) m[r] = max(m[r], most[r][k] < kInf ? most[r][k] : 0u);
            } else {
                for (int chunk = t; chunk < plan.chunks; chunk += group) {
                    load(r, 0, chunk);
                    const uint32_t n = largest(x[r][0]);
                    m[r] = max(m[r], n < kInf ? n : 0u);
                }
            }
            if (group >= 32)
                m[r] = __reduce_max_sync(0xffffffffu, m[r]);
            else
                for (int o = group / 2; o > 0; o >>= 1) m[r] = max(m[r], __shfl_xor_sync(0xffffffffu, m[r], o));
        }
        if (group > 32) {
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int r = 0; r < kRows; ++r) part[r][threadIdx.x >> 5] = m[r];
            __syncthreads();
            const int first = threadIdx.x / group * (group / 32);
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                for (int w = 0; w < group / 32; ++w) m[r] = max(m[r], part[r][first + w]);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) g[r] = least_power(m[r], 0x280000u) - 11;  // m <= 448 * 6 * 2^g = 1.3125 * 2^11 * 2^g
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t row = row0 + r * groups;
        const bool in = row < q.rows;
        if (in && t == 0) q.row_scale[row] = kBlock == 16 ? power(g[r]) : 1.f;
        uint8_t* values = static_cast<uint8_t*>(q.values) + (in ? row * q.values_stride : 0);
        uint32_t* to = words + scale_word(row, 0, plan.tiles);
        auto finish = [&](int k, int chunk, uint32_t m) {
            uint32_t code;
            const uint2 c = encode<T, kBlock>(x[r][k], m, g[r], code);
            const bool there = in && chunk < plan.chunks;
            if (there) {
                const int64_t bytes = (q.cols + 1) / 2 - int64_t(chunk) * 8;
                put_codes(values + int64_t(chunk) * 8, c, int(min(int64_t(8), bytes)), plan.vec_out);
            }
            // the word of a row's four blocks, from the threads that have them; scales that belong to no block are 0
            uint32_t w = there ? code << 8 * (chunk * kPer / kBlock & 3) : 0u;
#pragma unroll
            for (int o = kOfTile / 2; o > 0; o >>= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
            const int tile = chunk / kOfTile;
            if (t % kOfTile == 0 && tile < plan.tiles && row < plan.padded) to[tile * 128] = w;
        };
        if (kChunks) {
#pragma unroll
            for (int k = 0; k < kHeld; ++k) finish(k, t + k * group, most[r][k]);
        } else {
            // all threads of a row (256) take as many turns
            for (int first = 0; first < plan.chunks; first += group) {
                load(r, 0, first + t);
                uint32_t m = largest(x[r][0]);
                if (kBlock == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                finish(0, first + t, m);
            }
        }
    }
}

template <typename T, int kBlock>
cudaError_t launch_quantize(const sampler_micro_t& q, int sms, cudaStream_t stream)
{
    Plan p;
    const int64_t chunks = (q.cols + kPer - 1) / kPer;
    p.chunks = int(chunks);
    p.tiles = int(((q.cols + kBlock - 1) / kBlock + 3) / 4);
    p.padded = (q.rows + 127) / 128 * 128;
    p.vec_in = reinterpret_cast<uintptr_t>(q.src) % 16 == 0 && q.src_stride * int64_t(sizeof(T)) % 16 == 0;
    p.vec_out = reinterpret_cast<uintptr_t>(q.values) % 8 == 0 && q.values_stride % 8 == 0;
    p.group = 4 * kBlock / kPer;  // the threads that share a word of scales
    while (p.group < kThreads && p.group < chunks) p.group *= 2;
    const int held = chunks <= p.group ? 1 : chunks <= 2 * kThreads ? 2 : chunks <= 4 * kThreads ? 4 : 0;
    // Rows in hand, for the loads under way: two where there are more than eight blocks' worth for each SM and they lie in
    // whole vectors, four of bf16 whose blocks need no row's largest, where every thread has a chunk. Measured, us by one,
    // two and four:
    //   128000 x 4096 bf16    336  300  304, blocks of 32: 271  233  220
    //   64000 x 4096 fp32     210  199  244, blocks of 32: 189  183  232
    //   150000 x 1000 bf16    124  126  150, blocks of 32: 105   97  103
    //   20001 x 1001 fp32      27   31   42
    constexpr bool kFour = sizeof(T) == 2 && kBlock == 32;
    const int rows = held != 1 || !p.vec_in || p.padded * p.group <= int64_t(sms) * 8 * kThreads ? 1
                     : kFour && chunks == p.group                                               ? 4
                                                                                                : 2;
    const int64_t per = kThreads / p.group * rows;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((p.padded + per - 1) / per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    const auto kernel = rows == 4   ? quantize_kernel<T, kBlock, 1, kFour ? 4 : 2>
                        : rows == 2 ? quantize_kernel<T, kBlock, 1, 2>
                        : held == 1 ? quantize_kernel<T, kBlock, 1, 1>
                        : held == 2 ? quantize_kernel<T, kBlock, 2, 1>
                        : held == 4 ? quantize_kernel<T, kBlock, 4, 1>
                                    : quantize_kernel<T, kBlock, 0, 1>;
    return cudaLaunchKernelEx(&cfg, kernel, q, p);
}

// ---------------------------------------------------------------- reading back
// Two codes of a byte to two values, exactly.
__device__ __forceinline__ float2 values2(uint32_t byte)
{
    float2 y;
    asm("{\n\t.reg .b8 c;\n\t.reg .b32 w;\n\t.reg .b16 lo, hi, s;\n\tcvt.u16.u32 s, %2;\n\tcvt.u8.u16 c, s;\n\t"
        "cvt.rn.f16x2.e2m1x2 w, c;\n\tmov.b32 {lo, hi}, w;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "r"(byte));
    return y;
}

template <typename T>
struct Out;
template <>
struct Out<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ uint4 pack(const float* x)
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Out<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ uint4 pack(const float* x)
    {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Eight codes of a row from column `col` on, in a word (of columns before the first, 0; `words` of codes are the row's). Both
// words are read, so that nothing waits for a branch.
__device__ __forceinline__ uint32_t codes_at(const uint8_t* row, int col, int words)
{
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
    const int i = col >> 3;  // (rounded down)
    const uint32_t a = __ldg(w + max(i, 0)), b = __ldg(w + min(i + 1, words - 1));
    return __funnelshift_r(i < 0 ? 0u : a, b, 4 * (col & 7));
}

// kVectors 16-byte vectors of the output in each thread, `group` of them side by side. kCut (bf16 whose rows begin within
// a vector): the vectors are the output's, whose codes and scales are cut out of the row's, and not the row's, stored one
// by one: 3000 x 15001 takes 43 us in place of 127. In fp32, with half as many values in a vector, it would be 36 in place
// of 29 (20001 x 1001).
template <typename T, int kBlock, bool kCut>
__global__ void __launch_bounds__(kThreads) rows_kernel(const sampler_micro_rows_t q, int group, int vectors, int tiles,
                                                        bool vec_in, bool vec_out)
{
    constexpr int kVec = Out<T>::kVec;
    const int64_t r = int64_t(blockIdx.x) * (kThreads / group) + threadIdx.x / group;
    const int first = int(blockIdx.y) * (group * kVectors) + (threadIdx.x & (group - 1));
    if (r >= q.n || first >= vectors) return;
    const int64_t row = q.ids ? int64_t(__ldg(q.ids + r)) : r;
    const bool there = row >= 0 && row < q.rows;
    const uint8_t* v = static_cast<const uint8_t*>(q.values) + (there ? row * q.values_stride : 0);
    const uint8_t* s = static_cast<const uint8_t*>(q.scales) + (there ? scale_word(row, 0, tiles) * 4 : 0);
    T* out = static_cast<T*>(q.out) + r * q.out_stride;
    const float row_scale = !there ? __int_as_float(0x7fc00000) : q.row_scale ? __ldg(q.row_scale + row) : 1.f;
    const int cols = int(q.cols), bytes = (cols + 1) / 2;
    const int head = kCut ? int(reinterpret_cast<uintptr_t>(out) & 15u) / int(sizeof(T)) : 0;  // columns of the first vector before the row
    uint32_t codes[kVectors], scale[kVectors], next[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        int col = (first + k * group) * kVec - head;
        codes[k] = scale[k] = next[k] = 0u;
        if (!there || (!kCut && col >= cols)) continue;
        if (kCut) {
            col = min(col, cols - 1);  // (a vector that is not there reads what is not used)
            if (vec_in) {
                codes[k] = codes_at(v, col, (bytes + 3) / 4);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (col + j >= 0 && col + j < cols) codes[k] |= (uint32_t(v[(col + j) / 2]) >> 4 * ((col + j) & 1) & 15u) << 4 * j;
            }
            const int b0 = max(col, 0) / kBlock, b1 = min(col + kVec - 1, cols - 1) / kBlock;
            scale[k] = __ldg(s + (b0 / 4) * 512 + b0 % 4);
            next[k] = __ldg(s + (b1 / 4) * 512 + b1 % 4);
        } else {
            const uint8_t* p = v + col / 2;
            if (vec_in && col + kVec <= cols) {
                codes[k] = kVec == 8 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p)));
            } else {
#pragma unroll
                for (int j = 0; j < kVec / 2; ++j)
                    if (col + 2 * j < cols) codes[k] |= uint32_t(p[j]) << 8 * j;
            }
            const int b = col / kBlock;
            scale[k] = __ldg(s + (b / 4) * 512 + b % 4);
        }
    }
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        const int col = (first + k * group) * kVec - head;
        if (col >= cols) break;
        const float unit = scale_value<kBlock>(scale[k]) * row_scale, after = kCut ? scale_value<kBlock>(next[k]) * row_scale : unit;
        float x[kVec];
#pragma unroll
        for (int j = 0; j < kVec; j += 2) {
            const float2 y = values2(codes[k] >> 4 * j & 0xffu);
            // (a block that begins within the vector begins where the row's first column is in its own)
            const Two u = kCut ? two(__float_as_uint(j >= head ? after : unit), __float_as_uint(j + 1 >= head ? after : unit))
                               : two(__float_as_uint(unit), __float_as_uint(unit));
            const Two z = times(two(__float_as_uint(y.x), __float_as_uint(y.y)), u);
            x[j] = __uint_as_float(uint32_t(z));
            x[j + 1] = __uint_as_float(uint32_t(z >> 32));
        }
        const uint4 y = Out<T>::pack(x);
        if (vec_out && (!kCut || col >= 0) && col + kVec <= cols) {
            __stcs(reinterpret_cast<uint4*>(out + col), y);
        } else {
            const T* e = reinterpret_cast<const T*>(&y);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if ((!kCut || col + j >= 0) && col + j < cols) out[col + j] = e[j];
        }
    }
}

template <typename T, int kBlock>
cudaError_t launch_rows(const sampler_micro_rows_t& q, cudaStream_t stream)
{
    constexpr int kVec = Out<T>::kVec;
    const bool vec_in = reinterpret_cast<uintptr_t>(q.values) % (kVec / 2) == 0 && q.values_stride % (kVec / 2) == 0;
    const bool whole = reinterpret_cast<uintptr_t>(q.out) % 16 == 0 && q.out_stride * int64_t(sizeof(T)) % 16 == 0;
    const bool cut = sizeof(T) == 2 && !whole;
    const int64_t vectors = (q.cols + (cut ? 2 * kVec - 2 : kVec - 1)) / kVec;  // the most that a row touches
    int group = 2;
    while (group < kThreads && group * kVectors < vectors) group *= 2;
    const int64_t per = kThreads / group;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((q.n + per - 1) / per), unsigned((vectors + group * kVectors - 1) / (group * kVectors)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    const int tiles = int(((q.cols + kBlock - 1) / kBlock + 3) / 4);
    const auto kernel = sizeof(T) == 2 && cut ? rows_kernel<T, kBlock, sizeof(T) == 2> : rows_kernel<T, kBlock, false>;
    return cudaLaunchKernelEx(&cfg, kernel, q, group, int(vectors), tiles, vec_in, whole || cut);
}

}  // namespace micro

int micro_quantize_launch(const sampler_micro_t& q, int sms, cudaStream_t stream)
{
    using namespace micro;
    const bool bf16 = q.dtype == SAMPLER_DTYPE_BF16;
    const cudaError_t e = q.block == 16 ? bf16 ? launch_quantize<uint16_t, 16>(q, sms, stream) : launch_quantize<float, 16>(q, sms, stream)
                          : bf16        ? launch_quantize<uint16_t, 32>(q, sms, stream)
                                        : launch_quantize<float, 32>(q, sms, stream);
    return e == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

int micro_rows_launch(const sampler_micro_rows_t& q, cudaStream_t stream)
{
    using namespace micro;
    const bool bf16 = q.dtype == SAMPLER_DTYPE_BF16;
    const cudaError_t e = q.block == 16 ? bf16 ? launch_rows<uint16_t, 16>(q, stream) : launch_rows<float, 16>(q, stream)
                          : bf16        ? launch_rows<uint16_t, 32>(q, stream)
                                        : launch_rows<float, 32>(q, stream);
    return e == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

}  // namespace dst
