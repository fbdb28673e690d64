// gdn_chunk.hpp - internal interface between gdn_chunk_api.cpp and the kernels
// of the delta rule over packed sequences (gdn_chunk.hip, gdn_chunk_back.hip,
// gdn_decode.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn_launch.hpp"

namespace gdn {

constexpr int kChunk = 64;                       // tokens of a chunk
constexpr int kPlaneBytes = kChunk * kHeadDim * 2;   // one bf16 plane of a chunk's rows

// Packed sequences: sequence b holds tokens offsets[b] .. offsets[b+1] - 1, or
// tokens / B of them without offsets; its state is at slots[b], or at b.
struct Packed {
    const int32_t *offsets;          // [B+1] or NULL
    const int32_t *slots;            // [B] or NULL
    int32_t B;
    int32_t tokens;
    int32_t n_slots;
    int32_t Hv;
    int32_t Hk;
    int32_t type;                    // of q, k, v, out
};

// Chunk c of sequence b has place first / 64 + b + c among those of the
// workspace (first: the sequence's first token): no two chunks share one.
constexpr int64_t chunk_places(int64_t B, int64_t tokens) { return tokens / kChunk + B; }

// Planes that cut a value of the type exactly, and those of a product whose result
// is of the type.
constexpr int planes_in(int type) { return type == 0 ? 3 : type == 1 ? 1 : 2; }
constexpr int planes_out(int type) { return type == 0 ? 3 : 2; }

// What a chunk's tokens do to each other, a block per chunk place and value head, as
// LDS holds it:
//   T    (I + A)^-1 in three bf16 planes: six operands of 16 tokens x 32 tokens each
//        (the others lie above the diagonal);
//   P    the masked, decayed and scaled Q K^T, likewise, in as many planes as the
//        outputs need;
//   vec  rise, fall and beta of the 64 tokens.
// And, unless the inputs are bf16, the planes of k and q per chunk place and key
// head.
constexpr int kPBlocks = 6;
constexpr int kTBytes = kPBlocks * 1024 * 3;
constexpr int kVecFloats = 3 * kChunk;
constexpr int within_bytes(int planes) { return kTBytes + kPBlocks * 1024 * planes + 1024; }

struct ChunkArgs {
    Packed s;
    const void *q;
    const void *k;
    const void *v;
    const float *beta;
    const float *gate;
    const float *state;              // NULL: zeros
    float *state_out;                // NULL: not wanted
    void *out;
    // workspace
    char *within;                    // T, P and vec
    char *kq;                        // NULL for bf16
    // the backward pass alone
    const void *d_out;
    float *states;                   // [place][Hv][dv][dk] that enter the chunks
    float *delta;                    // [place][Hv][64][dv]
    float *od;                       // [place][Hv][8][64] sums of out * d_out over 16 rows each
};

// The backward pass.  After k_prep and k_walk, k_back goes along the sequences in
// reverse with the state's gradient, and k_grad forms what remains per chunk.
struct BackArgs {
    ChunkArgs f;
    const float *d_state_out;        // NULL: zeros
    float *d_state;                  // NULL: not wanted
    void *dq;
    void *dk;
    void *dv;
    float *dbeta;
    float *dgate;
    // workspace
    char *back;                      // as within: T read along its columns, P transposed, vec
    double *gsum;                    // [place][Hv][64] running sums of the gates, times log2 e
    float *dstates;                  // [place][Hv][dv][dk] that leave the chunks
    float *r;                        // [place][Hv][64][dv]
    float *du;                       // [place][Hv][8] sums of delta * (gradient of M' k) over 16 rows
};

struct DecodeArgs {
    Packed s;
    const void *q;
    const void *k;
    const void *v;
    const float *beta;
    const float *gate;
    const float *state;
    float *state_out;
    void *out;
};

hipError_t launch_chunk(const ChunkArgs &a, hipStream_t s);
hipError_t launch_chunk_backward(const BackArgs &a, hipStream_t s);
hipError_t launch_decode(const DecodeArgs &a, hipStream_t s);

}  // namespace gdn
