// gdn_logprobs.hpp - internal interface between gdn_logprobs_api.cpp
// and gdn_logprobs.hip.  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace gdn {

struct LogprobsArgs {
    const void *logits;
    int64_t ld;                      // elements from row to row
    const int32_t *tokens;           // NULL: not wanted
    float *logprob;
    float *entropy;                  // NULL: not wanted
    int32_t *top_ids;
    float *top_logprobs;
    double *sums;                    // [rows][units][3], in the workspace
    uint64_t *keys;                  // [rows][units][top]
    int32_t rows;
    int32_t V;
    int32_t top;
    int32_t type;
};

constexpr int kLogprobsMaxTop = 64;
constexpr int kLogprobsMaxUnits = 64;

// Units that a row is read in, a workgroup each.
constexpr int64_t logprobs_units(int64_t rows, int64_t V) {
    const int64_t fill = (1024 + rows - 1) / rows, most = (V + 4095) / 4096;
    const int64_t n = fill < most ? fill : most;
    return n < kLogprobsMaxUnits ? n : kLogprobsMaxUnits;
}

hipError_t launch_logprobs(const LogprobsArgs &a, hipStream_t s);

}  // namespace gdn
