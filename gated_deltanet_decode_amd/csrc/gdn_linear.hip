// gdn_linear.hip - gdn_linear_q8: int8 rows times int8 weights on the matrix
// cores, scaled by row and channel and written to up to four output tensors.
//
// Mathematics.  y[m][c] = (sum_k a[m][k] w[c][k]) a_scale[m] w_scale[c] + bias[c].
// The integer sum is exact in 32 bits, so neither the order of k nor a split
// of it over waves changes a result.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_serve.hpp"

namespace gdn {
namespace {

typedef int32_t i4 __attribute__((ext_vector_type(4)));

// Sixteen bytes at k of a row of K bytes, zero past its end.
__device__ __forceinline__ i4 load16(const int8_t *row, int k, int K) {
    typedef int32_t any __attribute__((ext_vector_type(4), aligned(1)));
    i4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        v = *reinterpret_cast<const any *>(row + k);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k + i < K) v[i / 4] |= static_cast<int32_t>(static_cast<uint8_t>(row[k + i]))
                                       << (8 * (i % 4));
    }
    return v;
}

// Writes the scaled sums of 4 consecutive channels c.. of token m.
template <typename OT>
__device__ __forceinline__ void put4(const LinearArgs &a, int m, int c, i4 acc) {
    const float sa = a.a_scale[m];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ch = c + i;
        if (ch >= a.N) return;
        float y = static_cast<float>(acc[i]) * sa * a.w_scale[ch];
        if (a.bias) y += a.bias[ch];
        int s = 0, first = 0;
#pragma unroll
        for (int j = 0; j < kLinearMaxOuts - 1; ++j)
            if (ch >= a.end[j]) {
                s = j + 1;
                first = a.end[j];
            }
        typename OT::bits *out = static_cast<typename OT::bits *>(a.out[s]);
        out[static_cast<int64_t>(m) * (a.end[s] - first) + (ch - first)] = OT::put(y);
    }
}

// Four waves, each a 16 (channels) x 64 (tokens) tile of a 64 x 64 block.
template <typename OT>
__global__ __launch_bounds__(256) void k_linear(LinearArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tiles_n = (a.N + 63) / 64;
    const int tn = blockIdx.x % tiles_n, tm = blockIdx.x / tiles_n;
    const int r = lane & 15, g = lane >> 4;
    const int c0 = tn * 64 + wave * 16, m0 = tm * 64;
    const int8_t *w = a.w + static_cast<int64_t>(min(c0 + r, a.N - 1)) * a.K;
    const int8_t *x[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
        x[t] = a.a + static_cast<int64_t>(min(m0 + 16 * t + r, a.M - 1)) * a.K;
    i4 acc[4] = {};
    for (int k = 16 * g; k - 16 * g < a.K; k += 64) {
        const i4 wv = load16(w, k, a.K);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, load16(x[t], k, a.K), acc[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int m = m0 + 16 * t + r;
        if (m < a.M) put4<OT>(a, m, c0 + 4 * g, acc[t]);
    }
}

template <typename OT>
hipError_t launch(const LinearArgs &a, hipStream_t s) {
    const int64_t tiles = (static_cast<int64_t>(a.M) + 63) / 64 * ((a.N + 63) / 64);
    k_linear<OT><<<dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
    switch (a.out_type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
