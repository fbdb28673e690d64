// gdn_serve.hpp - internal interface between gdn_serve_api.cpp and the kernels
// of the operators around the recurrent branch (gdn_quant.hip,
// gdn_linear.hip, gdn_verify.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace gdn {

// Element types, by the codes of gdn.h (GDN_F32, GDN_BF16, GDN_F16, GDN_NONE).
struct QuantArgs {
    const void *x;
    const void *residual;      // NULL: none
    void *residual_out;
    const float *norm_w;       // NULL: no norm (the codes of x itself)
    int8_t *q;
    float *scale;
    float eps;
    int32_t rows;
    int32_t n;
    int32_t x_type;
    int32_t residual_type;
};

// Threads per row, at most one workgroup of them per row.
constexpr int kQuantMaxThreads = 1024;

constexpr int kLinearMaxOuts = 4;

struct LinearArgs {
    const int8_t *a;
    const float *a_scale;
    const int8_t *w;
    const float *w_scale;
    const float *bias;               // NULL: none
    void *out[kLinearMaxOuts];
    int32_t end[kLinearMaxOuts];     // one past the group's last channel
    int32_t M;
    int32_t N;
    int32_t K;
    int32_t out_type;
};

struct VerifyArgs {
    const void *target;
    const void *draft;               // NULL: greedy drafts
    const int32_t *draft_tokens;
    const int32_t *n_draft;          // NULL: K everywhere
    const float *u_accept;
    const float *u_sample;
    int32_t *accepted;
    int32_t *tokens;
    double *partial;                 // [B][kVerifyUnits] sums, in the workspace
    int32_t *rows;                   // [B][4] decisions, in the workspace
    int32_t B;
    int32_t K;
    int32_t V;
    int32_t prob_type;
};

// Units that a row is summed in, at most.
constexpr int kVerifyUnits = 256;
// Bytes of workspace a sequence takes: its units' sums and its decision.
constexpr size_t kVerifyBytes = kVerifyUnits * sizeof(double) + 4 * sizeof(int32_t);

// Copies one sequence's state and ring per accepted sequence and layer.
struct CommitArgs {
    const int32_t *accepted;
    float *state;
    const float *state_next;
    float *ring;                     // NULL: none
    const float *ring_next;
    int32_t layers;
    int32_t B;
    int64_t state_f4;                // float4s of one sequence's state in one layer
    int32_t ring_f4;
};

// float4s that one workgroup of the commit copies, and its threads.
constexpr int kCommitF4 = 2048;
constexpr int kCommitThreads = 256;
constexpr int64_t commit_blocks(int64_t f4) { return (f4 + kCommitF4 - 1) / kCommitF4; }

hipError_t launch_quant(const QuantArgs &a, hipStream_t s);
hipError_t launch_linear(const LinearArgs &a, hipStream_t s);
hipError_t launch_verify(const VerifyArgs &a, hipStream_t s);
hipError_t launch_commit(const CommitArgs &a, hipStream_t s);

}  // namespace gdn
