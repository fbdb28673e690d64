// gdn_elem.hpp - device-side element types of the operators around the
// recurrent branch: conversions to and from binary32, vector accesses at any
// element's alignment, and moves between a wave's lanes.  Included by kernel
// sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {
namespace {

// Storage types.  Every conversion to float is exact; from float rounds to
// nearest, ties to even.
struct F32 {
    typedef uint32_t bits;
    static __device__ __forceinline__ float get(uint32_t b) { return __builtin_bit_cast(float, b); }
    static __device__ __forceinline__ uint32_t put(float x) {
        return __builtin_bit_cast(uint32_t, x);
    }
};
struct BF16 {
    typedef uint16_t bits;
    static __device__ __forceinline__ float get(uint16_t b) {
        return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16);
    }
    static __device__ __forceinline__ uint16_t put(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    }
};
struct F16 {
    typedef uint16_t bits;
    static __device__ __forceinline__ float get(uint16_t b) {
        return static_cast<float>(__builtin_bit_cast(_Float16, b));
    }
    static __device__ __forceinline__ uint16_t put(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    }
};

// N consecutive elements that need no more than one element's alignment (an
// odd row length puts rows at any element): one wide access, which the memory
// system takes at any byte address.
template <typename B, int N>
struct Pack {
    typedef B vec __attribute__((ext_vector_type(N)));
    typedef B any __attribute__((ext_vector_type(N), aligned(sizeof(B))));
    static __device__ __forceinline__ vec load(const B *p) {
        return *reinterpret_cast<const any *>(p);
    }
    static __device__ __forceinline__ void store(B *p, vec v) { *reinterpret_cast<any *>(p) = v; }
};

// Moves of values between a wave's lanes: by DPP control within rows of 16 lanes
// (0 where there is no source lane), and one lane's value to all.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, static_cast<uint64_t>(dpp<CTRL>(static_cast<uint32_t>(b >> 32))) << 32 |
                                          dpp<CTRL>(static_cast<uint32_t>(b)));
}
__device__ __forceinline__ uint32_t lane_of(uint32_t x, int l) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), l));
}
__device__ __forceinline__ double lane_of(double x, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, static_cast<uint64_t>(lane_of(static_cast<uint32_t>(b >> 32), l)) << 32 |
                                          lane_of(static_cast<uint32_t>(b), l));
}

}  // namespace
}  // namespace gdn
