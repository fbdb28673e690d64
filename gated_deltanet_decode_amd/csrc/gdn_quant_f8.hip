// gdn_quant_f8.hip - gdn_quantize_f8: e4m3 codes with one scale for each block of
// 128 elements of a row, or of 128 rows by 128 elements.
//
// Mathematics.  With G the block's largest magnitude, scale = G / 448 and the
// codes are 448 x / G rounded to e4m3, ties to even: three bits behind the first,
// steps of 2^-9 below 2^-6.  The quotient is formed in binary32, within 2^-22 of
// itself.  A tie between two codes is o 2^e with o odd and below 32, and
// 7 x 2^k - G o is an integer in units of the elements' last places: a quotient that is
// no tie is off one by 1 / (31 G) of itself or more, 2^-13 for bfloat16's 8 bits
// and 2^-16 for binary16's 11.  Rounding it to 16 and 20 bits first makes a tie
// exact and moves nothing else across one.  For binary32 a quotient next to a tie
// is settled in binary64, where one that is no tie is 2^-29 or more off and a tie is
// exact.  One pass: 16 elements a lane, eight lanes a block's row.
//
// Memory bounds it: 32768 x 2048 bf16 31 us (6.7 TB/s), f32 60 (5.6); 12352 x 2048 f32 in
// squares 26 (4.8).  bf16 with the check of binary32 48 us, 8 elements a lane and the
// check 53, two pieces a thread and the check 53.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_f8.hpp"

namespace gdn {
namespace {

constexpr int kT = 256;
constexpr int N = 16;                        // elements a thread takes at a time
constexpr int kLanes = kF8Block / N;         // lanes of a block's row

// Bits that a quotient is rounded to before its code is taken.
template <typename XT> constexpr int kPlaces = 24;
template <> constexpr int kPlaces<BF16> = 16;
template <> constexpr int kPlaces<F16> = 20;

// 448 x / top as the nearest e4m3 value.
__device__ __forceinline__ float settled(float x, double top) {
    const double q = 448.0 * static_cast<double>(x) / top;
    const int e = static_cast<int>(__builtin_bit_cast(uint64_t, q) >> 52 & 2047) - 1023;
    const double step = __builtin_bit_cast(double, static_cast<uint64_t>(max(e, -6) - 3 + 1023) << 52);
    return static_cast<float>(rint(q / step) * step);
}

// Sixteen elements from p, those from `live` on zero.
template <typename XT>
__device__ __forceinline__ void load(const typename XT::bits *p, int live, float (&x)[N]) {
    typedef typename XT::bits bits;
    constexpr int V = 16 / sizeof(bits);
    if (live >= N) {
#pragma unroll
        for (int i = 0; i < N / V; ++i) {
            const auto v = Pack<bits, V>::load(p + i * V);
#pragma unroll
            for (int j = 0; j < V; ++j) x[i * V + j] = XT::get(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = j < live ? XT::get(p[j]) : 0.0f;
    }
}

// Half the step of e4m3 at y less 2^-16 of itself: the quotient is known to 2^-22 of
// itself, below 2^-17 of the half step.
__device__ __forceinline__ float nearly(float y) {
    const uint32_t b = __builtin_bit_cast(uint32_t, y) & 0x7f800000u;
    return __builtin_bit_cast(float, max(b, 0x3c800000u) - ((4u << 23) + 256));
}

template <typename XT>
__device__ __forceinline__ void codes(float (&x)[N], uint32_t m, uint32_t (&w)[N / 4]) {
    const float top = __builtin_bit_cast(float, m);
    // 2^-100 <= top < 2^120: neither the reciprocal nor a product over- or underflows
    // where it counts
    const bool plain = m >= 0x0d800000u && m < 0x7b800000u;
    const float inv = plain ? 448.0f / top : 0.0f;
    float y[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        y[j] = plain ? x[j] * inv : 0.0f;
        if constexpr (kPlaces<XT> < 24) {
            constexpr uint32_t kCut = 1u << (24 - kPlaces<XT>);
            y[j] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, y[j]) + kCut / 2) & ~(kCut - 1));
        }
    }
    float past = -1.0f;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int c = 0;
        c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], c, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], c, true);
        w[i] = static_cast<uint32_t>(c);
        if constexpr (kPlaces<XT> == 24) {
            const float d[4] = {__builtin_amdgcn_cvt_f32_fp8(c, 0), __builtin_amdgcn_cvt_f32_fp8(c, 1),
                                __builtin_amdgcn_cvt_f32_fp8(c, 2), __builtin_amdgcn_cvt_f32_fp8(c, 3)};
#pragma unroll
            for (int j = 0; j < 4; ++j) past = fmaxf(past, fabsf(y[4 * i + j] - d[j]) - nearly(y[4 * i + j]));
        }
    }
    uint32_t near = plain || m == 0 || m >= 0x7f800000u ? 0u : (1u << N) - 1;
    if (past >= 0.0f)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float d = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w[j / 4] >> 8 * (j & 3)), 0);
            near |= fabsf(y[j] - d) >= nearly(y[j]) ? 1u << j : 0u;
        }
    while (near) {                                        // seldom: one element at a time
        const int k = __ffs(near) - 1;
        near &= near - 1;
        float g = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) g = j == k ? x[j] : g;
        const float v = settled(g, static_cast<double>(top));
        const uint32_t c = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false)) & 255u;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const int at = 8 * (k & 3);
            w[i] = i == k >> 2 ? (w[i] & ~(255u << at)) | c << at : w[i];
        }
    }
}

__device__ __forceinline__ void store(uint8_t *q, int live, const uint32_t (&w)[N / 4]) {
    if (live >= N) {
        typedef uint32_t any __attribute__((ext_vector_type(4), aligned(1)));
        *reinterpret_cast<any *>(q) = any{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < live) q[j] = static_cast<uint8_t>(w[j / 4] >> 8 * (j & 3));
    }
}

// Zero for a block of zeros, NaN for one with a NaN or an infinity.
__device__ __forceinline__ float scale_of(uint32_t m) {
    return m >= 0x7f800000u ? __builtin_nanf("") : __builtin_bit_cast(float, m) / 448.0f;
}

// The largest magnitude of eight lanes (by DPP: lanes 1 and 2 apart, then mirrored).
__device__ __forceinline__ uint32_t largest(const float (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, __builtin_bit_cast(uint32_t, x[j]) & 0x7fffffffu);
    m = max(m, dpp<0xB1>(m));
    m = max(m, dpp<0x4E>(m));
    return max(m, dpp<0x141>(m));
}

// One block of a row per eight lanes.
template <typename XT>
__global__ __launch_bounds__(kT) void k_rows(QuantF8Args a, uint32_t blocks, uint32_t all) {
    const uint32_t id = (blockIdx.x * kT + threadIdx.x) / kLanes;
    if (id >= all) return;                                // whole groups of lanes
    const uint32_t row = id / blocks, b = id - row * blocks;
    const int at = b * kF8Block + (threadIdx.x % kLanes) * N;
    const int64_t i = static_cast<int64_t>(row) * a.n + at;
    float x[N];
    uint32_t w[N / 4];
    load<XT>(static_cast<const typename XT::bits *>(a.x) + i, a.n - at, x);
    const uint32_t m = largest(x);
    codes<XT>(x, m, w);
    store(a.q + i, a.n - at, w);
    if (threadIdx.x % kLanes == 0) a.scale[id] = scale_of(m);
}

// One block of 128 rows per workgroup, in registers.
template <typename XT>
__global__ __launch_bounds__(kT) void k_square(QuantF8Args a, uint32_t blocks) {
    constexpr int R = kF8Block * kLanes / kT;             // rows a thread has a piece of
    __shared__ uint32_t tops[kT / 64];
    const uint32_t rb = blockIdx.x / blocks, b = blockIdx.x - rb * blocks;
    const int at = b * kF8Block + (threadIdx.x % kLanes) * N;
    float x[R][N];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t row = static_cast<int64_t>(rb) * kF8Block + k * (kT / kLanes) + threadIdx.x / kLanes;
        load<XT>(static_cast<const typename XT::bits *>(a.x) + row * a.n + at, row < a.rows ? a.n - at : 0, x[k]);
        m = max(m, largest(x[k]));
    }
#pragma unroll
    for (int d = kLanes; d < 64; d *= 2) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) m = max(m, tops[w]);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t row = static_cast<int64_t>(rb) * kF8Block + k * (kT / kLanes) + threadIdx.x / kLanes;
        uint32_t w[N / 4];
        codes<XT>(x[k], m, w);
        if (row < a.rows) store(a.q + row * a.n + at, a.n - at, w);
    }
    if (threadIdx.x == 0) a.scale[blockIdx.x] = scale_of(m);
}

template <typename XT>
hipError_t launch(const QuantF8Args &a, hipStream_t s) {
    const int64_t blocks = (a.n + kF8Block - 1) / kF8Block;
    if (a.block_rows == 1) {
        const int64_t all = a.rows * blocks, per = kT / kLanes;
        k_rows<XT><<<dim3(static_cast<unsigned>((all + per - 1) / per)), dim3(kT), 0, s>>>(
            a, static_cast<uint32_t>(blocks), static_cast<uint32_t>(all));
    } else {
        const int64_t tall = (a.rows + kF8Block - 1) / kF8Block;
        k_square<XT><<<dim3(static_cast<unsigned>(tall * blocks)), dim3(kT), 0, s>>>(a, static_cast<uint32_t>(blocks));
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_f8(const QuantF8Args &a, hipStream_t s) {
    switch (a.x_type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
