// gdn_mma.hpp - matrix instructions on float32 values, for the kernels of the
// delta rule in chunks.  Included by kernel sources only.
//
// A product that has to be right to binary32 runs on the bf16 matrix
// instructions: a float is taken apart into bf16 pieces ("planes"), each the nearest
// to what the ones before it leave, and the products of the pieces that matter are
// summed in the instruction's binary32 accumulators.  bf16 inputs are one
// plane, fp16 ones two, float32 values three; with planes numbered from 0, the
// products i + j <= 2 keep an error below 2^-24 of a term, i + j <= 1 one of
// 2^-16, which is far below half a step of a 16-bit result.  Three products
// of one plane with three run at 833 TFLOP/s of the dense bf16 peak, the
// float32 matrix instructions at 157.
//
// Operands of 16 x 16 x 32: lane r + 16 g supplies eight k of row (or column) r
// and receives rows 4 g..4 g+3 of column r.  Which k a slot (g, e) stands for is
// free as long as both operands agree, so the two results of 16 rows that a
// lane holds become an operand of 32 k as they are: slots e < 4 are rows
// 4 g + e of the first, the others of the second.  Swapping the operands
// transposes the result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// 16 x 16 x 16 in binary32: k slot (g, s) is element s of a lane's four.
__device__ __forceinline__ f4 mma32(f4 a, f4 b, f4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
}

// The products i + j <= L of an operand of NA planes with one of NB.
template <int L, int NA, int NB>
__device__ __forceinline__ f4 mma_planes(const u4 (&a)[NA], const u4 (&b)[NB], f4 c) {
#pragma unroll
    for (int t = L; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (i + j == t) c = mma(a[i], b[j], c);
    return c;
}

// The same for N operands against one, plane by plane, so that neighbouring
// instructions do not wait for each other; kFirst: the N come first.
template <int L, bool kFirst, int N, int NA, int NB>
__device__ __forceinline__ void mma_planes(const u4 (&a)[N][NA], const u4 (&b)[NB], f4 (&c)[N]) {
#pragma unroll
    for (int t = L; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (i + j == t)
#pragma unroll
                    for (int n = 0; n < N; ++n) c[n] = kFirst ? mma(a[n][i], b[j], c[n]) : mma(b[j], a[n][i], c[n]);
}

// Two floats as bf16, to nearest.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{lo, hi}, b2));
}

// The first N planes of eight floats.  To nearest, so that what is left has either
// sign: cut off towards zero, the products left out add up over a chunk whose
// corrections telescope (128 keys that are all alike: 3.7e-6 of the state for 1.6e-6).
// Each remainder is exact; a magnitude past 3.38e38 becomes an infinity.
template <int N>
__device__ __forceinline__ void planes_of(f4 a, f4 b, u4 (&p)[N]) {
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[n][i] = bf16_pair(x[2 * i], x[2 * i + 1]);
            if (n + 1 < N) {
                x[2 * i] -= __builtin_bit_cast(float, p[n][i] << 16);
                x[2 * i + 1] -= __builtin_bit_cast(float, p[n][i] & 0xffff0000u);
            }
        }
    }
}

// Four 16-bit values of column i (the lane's place among its 16) out of four rows:
// lane 4 e + c of the sixteen names four consecutive values of row e, columns
// 4 c..4 c+3.
__device__ __forceinline__ u2 read_columns(const char *p) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 *lds4;
    return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p)));
}

// At most N of this wave's vector-memory operations are still on their way, and
// none of its LDS operations.
template <int N>
__device__ __forceinline__ void wait_all() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
// What is issued above stays ahead of what is issued below, so that a wait can count.
__device__ __forceinline__ void in_order() { asm volatile("" ::: "memory"); }
// None of this wave's LDS operations is still on its way.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Rows of a head's tokens in a [tokens][heads][128] tensor, those of one chunk: an
// access past the last row reads zero and writes nothing.
template <typename ET>
struct Rows {
    typedef typename ET::bits bits;
    static constexpr int kBytes = sizeof(bits);
    __amdgpu_buffer_rsrc_t rows;
    int stride;                                           // bytes from token to token
    // `first` tokens into the tensor, n of them, head h of H
    __device__ __forceinline__ Rows(const void *base, int64_t first, int n, int h, int H) {
        stride = H * 128 * kBytes;
        rows = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(static_cast<const char *>(base)) + (first * H + h) * (128 * kBytes), 0,
            static_cast<uint32_t>(n - 1) * stride + 128 * kBytes, 0x00020000);
    }
    __device__ __forceinline__ bits load(int token, int at) const {
        if constexpr (kBytes == 2)
            return __builtin_bit_cast(bits, __builtin_amdgcn_raw_buffer_load_b16(rows, token * stride + at * kBytes, 0, 0));
        else
            return __builtin_bit_cast(bits, __builtin_amdgcn_raw_buffer_load_b32(rows, token * stride + at * kBytes, 0, 0));
    }
    __device__ __forceinline__ f4 load4(int token, int at) const {
        if constexpr (kBytes == 2) {
            typedef bits b4 __attribute__((ext_vector_type(4)));
            const b4 v = __builtin_bit_cast(b4, __builtin_amdgcn_raw_buffer_load_b64(rows, token * stride + at * kBytes, 0, 0));
            return f4{ET::get(v[0]), ET::get(v[1]), ET::get(v[2]), ET::get(v[3])};
        } else {
            return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rows, token * stride + at * kBytes, 0, 0));
        }
    }
    // eight elements as they are in memory, and their values
    struct Eight { u4 x[kBytes / 2]; };
    __device__ __forceinline__ Eight load8(int token, int at) const {
        Eight v;
#pragma unroll
        for (int i = 0; i < kBytes / 2; ++i)
            v.x[i] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rows, token * stride + at * kBytes + 16 * i, 0, 0));
        return v;
    }
    static __device__ __forceinline__ f4 four(const Eight &v, int i) {
        if constexpr (kBytes == 2) {
            typedef bits b8 __attribute__((ext_vector_type(8)));
            const b8 y = __builtin_bit_cast(b8, v.x[0]);
            return f4{ET::get(y[4 * i]), ET::get(y[4 * i + 1]), ET::get(y[4 * i + 2]), ET::get(y[4 * i + 3])};
        } else {
            return __builtin_bit_cast(f4, v.x[i]);
        }
    }
    __device__ __forceinline__ void store(int token, int at, float x) const {
        if constexpr (kBytes == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, ET::put(x)), rows, token * stride + at * kBytes, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), rows, token * stride + at * kBytes, 0, 0);
    }
    __device__ __forceinline__ void store4(int token, int at, f4 x) const {
        if constexpr (kBytes == 2) {
            typedef bits b4 __attribute__((ext_vector_type(4)));
            const b4 v = {ET::put(x[0]), ET::put(x[1]), ET::put(x[2]), ET::put(x[3])};
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, v), rows, token * stride + at * kBytes, 0, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), rows, token * stride + at * kBytes, 0, 0);
        }
    }
};

}  // namespace
}  // namespace gdn
