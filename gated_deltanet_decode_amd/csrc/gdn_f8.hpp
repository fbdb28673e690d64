// gdn_f8.hpp - internal interface between gdn_f8_api.cpp and the kernels of the
// 8-bit floating point operators (gdn_quant_f8.hip, gdn_linear_f8.hip).  Not
// installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "gdn_serve.hpp"

namespace gdn {

constexpr int kF8Block = 128;        // elements of a row that share a scale

struct QuantF8Args {
    const void *x;
    uint8_t *q;
    float *scale;
    int32_t rows;
    int32_t n;
    int32_t block_rows;              // 1 or 128
    int32_t x_type;
};

struct LinearF8Args {
    const int8_t *a;                 // bytes of e4m3
    const float *a_scale;            // [M][ceil(K / 128)]
    const int8_t *w;
    const float *w_scale;            // [ceil(N / 128)][ceil(K / 128)]
    const float *bias;               // NULL: none
    void *out[kLinearMaxOuts];
    int32_t end[kLinearMaxOuts];     // one past the group's last channel
    int32_t M;
    int32_t N;
    int32_t K;
    int32_t out_type;
};

hipError_t launch_quant_f8(const QuantF8Args &a, hipStream_t s);
hipError_t launch_linear_f8(const LinearF8Args &a, hipStream_t s);

}  // namespace gdn
