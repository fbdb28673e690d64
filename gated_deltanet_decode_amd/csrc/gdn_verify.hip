// gdn_verify.hip - gdn_verify (speculative verification from given random
// numbers) and gdn_pair_commit (the accepted sequences' tentative states).
//
// Mathematics.  Drafted token d of position i is accepted when all before it
// are and u q_i(d) < p_i(d); the token after the accepted run is drawn by
// inverting the cumulative sum of w = max(p - q, 0) at the refusal (or of p
// when no draft is left).  Probabilities of at most 24 significant bits make
// the product exact in binary64 and the sums good to 1e-16 of the total, so
// the outcome is the formula's whatever the order of the sums.
//
// Only one row of the target and at most one of the draft matter to a
// sequence, once the run of accepted tokens is known, and that takes 2 K
// single entries.  Two launches: the rows' chunks are summed by a workgroup
// each, then one workgroup per sequence finds the chunk and the entry in it.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_serve.hpp"

namespace gdn {
namespace {

constexpr int kT = 256;
constexpr int kPer = kVerifyChunk / kT;      // entries of a chunk per thread: 16

// Negative, infinite and NaN entries count as 0.
__device__ __forceinline__ double weight(float p) {
    return p > 0.0f && p <= 3.402823466e38f ? static_cast<double>(p) : 0.0;
}

struct Row {          // what a sequence's next token is drawn from
    int accepted;
    bool refused;     // position `accepted` refused a draft
    int token;        // that draft
};

// The run of accepted drafts of sequence b.  Called by whole waves; every
// lane returns the same.
template <typename PT>
__device__ __forceinline__ Row decide(const VerifyArgs &a, int64_t b) {
    typedef typename PT::bits bits;
    const int lane = threadIdx.x & 63;
    int n = a.n_draft ? a.n_draft[b] : a.K;
    n = max(0, min(n, a.K));
    Row row{n, false, -1};
    for (int i0 = 0; i0 < n; i0 += 64) {
        const int i = i0 + lane;
        bool bad = false;
        int d = -1;
        if (i < n) {
            d = a.draft_tokens[b * a.K + i];
            bad = true;
            if (d >= 0 && d < a.V) {
                const double p = weight(PT::get(
                    static_cast<const bits *>(a.target)[(b * (a.K + 1) + i) * a.V + d]));
                const double q = a.draft ? weight(PT::get(
                    static_cast<const bits *>(a.draft)[(b * a.K + i) * a.V + d])) : 1.0;
                bad = !(static_cast<double>(a.u_accept[b * a.K + i]) * q < p);
            }
        }
        const unsigned long long m = __ballot(bad);
        if (m) {
            const int first = __ffsll(m) - 1;
            row.accepted = i0 + first;
            row.refused = true;
            row.token = __shfl(d, first, 64);
            break;
        }
    }
    return row;
}

// The weights at v of the row: `rest` is max(p - q, 0), `all` is p.
template <typename PT>
struct Weights {
    typedef typename PT::bits bits;
    const bits *p;
    const bits *q;     // NULL: no draft row
    int one;           // the entry where a greedy draft's q is 1, else -1

    __device__ __forceinline__ Weights(const VerifyArgs &a, int64_t b, const Row &r) {
        p = static_cast<const bits *>(a.target) + (b * (a.K + 1) + r.accepted) * a.V;
        q = r.refused && a.draft
                ? static_cast<const bits *>(a.draft) + (b * a.K + r.accepted) * a.V
                : nullptr;
        one = r.refused && !a.draft ? r.token : -1;
    }
    __device__ __forceinline__ void at(int v, double &rest, double &all) const {
        all = weight(PT::get(p[v]));
        double d = q ? weight(PT::get(q[v])) : 0.0;
        if (v == one) d = 1.0;
        rest = fmax(all - d, 0.0);
    }
};

// Sums of a chunk's weights: partial[b][chunk] = {sum of rest, sum of all}.
template <typename PT>
__global__ __launch_bounds__(kT) void k_verify_sums(VerifyArgs a) {
    __shared__ double red[2][kT / 64];
    const int64_t b = blockIdx.y;
    const Weights<PT> w(a, b, decide<PT>(a, b));
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kVerifyChunk + threadIdx.x * kPer;
    double rest = 0.0, all = 0.0;
    for (int j = 0; j < kPer; ++j)
        if (v0 + j < a.V) {
            double x, y;
            w.at(static_cast<int>(v0 + j), x, y);
            rest += x;
            all += y;
        }
    rest = wave_sum(rest);
    all = wave_sum(all);
    if ((threadIdx.x & 63) == 0) {
        red[0][threadIdx.x >> 6] = rest;
        red[1][threadIdx.x >> 6] = all;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double *out = a.partial + (b * gridDim.x + blockIdx.x) * 2;
        out[0] = ((red[0][0] + red[0][1]) + red[0][2]) + red[0][3];
        out[1] = ((red[1][0] + red[1][1]) + red[1][2]) + red[1][3];
    }
}

// Inclusive sums over the workgroup's threads, in thread order.
__device__ __forceinline__ double block_scan(double x, double *red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    __syncthreads();                 // red may still be read from a call before
    if (lane == 63) red[wave] = x;
    __syncthreads();
    double base = 0.0;
    for (int w = 0; w < wave; ++w) base += red[w];
    return base + x;
}

// Finds the chunk and the entry where the cumulative sum passes u_sample times
// the total, and writes the sequence's answer.
template <typename PT>
__global__ __launch_bounds__(kT) void k_verify_pick(VerifyArgs a, int chunks) {
    __shared__ double red[kT / 64];
    __shared__ double total[2], before;
    __shared__ int chunk, pick, last;
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x;
    const Row row = decide<PT>(a, b);
    const double *part = a.partial + b * chunks * 2;
    if (tid == 0) {
        chunk = chunks;
        pick = a.V;
        last = -1;
        double rest = 0.0, all = 0.0;
        for (int c = 0; c < chunks; ++c) {
            rest += part[2 * c];
            all += part[2 * c + 1];
        }
        total[0] = rest;
        total[1] = all;
    }
    __syncthreads();
    const int which = total[0] > 0.0 ? 0 : 1;
    const double goal = static_cast<double>(a.u_sample[b]) * total[which];
    if (tid == 0) {
        double run = 0.0;
        before = 0.0;
        for (int c = 0; c < chunks; ++c) {
            const double x = part[2 * c + which];
            if (x > 0.0) {
                chunk = c;            // the last one with a weight, if none passes
                before = run;
                if (run + x > goal) break;
            }
            run += x;
        }
    }
    __syncthreads();
    int token = -1;
    if (chunk < chunks) {
        const Weights<PT> w(a, b, row);
        const int64_t v0 = static_cast<int64_t>(chunk) * kVerifyChunk + tid * kPer;
        double sum = 0.0;
        for (int j = 0; j < kPer; ++j)
            if (v0 + j < a.V) {
                double x, y;
                w.at(static_cast<int>(v0 + j), x, y);
                sum += which ? y : x;
            }
        double run = before + (block_scan(sum, red) - sum);
        int mine = a.V, end = -1;
        for (int j = 0; j < kPer; ++j)
            if (v0 + j < a.V) {
                double x, y;
                w.at(static_cast<int>(v0 + j), x, y);
                const double z = which ? y : x;
                run += z;
                if (z > 0.0) {
                    end = static_cast<int>(v0 + j);
                    if (run > goal && mine == a.V) mine = end;
                }
            }
        if (mine < a.V) atomicMin(&pick, mine);
        if (end >= 0) atomicMax(&last, end);
        __syncthreads();
        token = pick < a.V ? pick : last;
    }
    for (int i = tid; i <= a.K; i += kT)
        a.tokens[b * (a.K + 1) + i] = i < row.accepted    ? a.draft_tokens[b * a.K + i]
                                      : i == row.accepted ? token
                                                          : -1;
    if (tid == 0) a.accepted[b] = row.accepted;
}

template <typename PT>
hipError_t launch(const VerifyArgs &a, hipStream_t s) {
    const unsigned chunks = static_cast<unsigned>(verify_chunks(a.V));
    k_verify_sums<PT><<<dim3(chunks, static_cast<unsigned>(a.B)), dim3(kT), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_verify_pick<PT><<<dim3(static_cast<unsigned>(a.B)), dim3(kT), 0, s>>>(
        a, static_cast<int>(chunks));
    return hipGetLastError();
}

// ------------------------------------------------------------------ commit
typedef float f4 __attribute__((ext_vector_type(4)));

// One workgroup copies kCommitF4 float4s of one sequence's state or ring in
// one layer, if its draft was accepted.
__global__ __launch_bounds__(kCommitThreads) void k_commit(CommitArgs a, int per_state,
                                                           int per_seq) {
    const int64_t lb = blockIdx.x / per_seq;             // layer * B + b
    const int part = static_cast<int>(blockIdx.x - lb * per_seq);
    if (a.accepted[lb % a.B] < 1) return;
    const bool ring = part >= per_state;
    const int64_t n = ring ? a.ring_f4 : a.state_f4;
    const f4 *src = reinterpret_cast<const f4 *>(ring ? a.ring_next : a.state_next) + lb * n;
    f4 *dst = reinterpret_cast<f4 *>(ring ? a.ring : a.state) + lb * n;
    const int64_t i0 = static_cast<int64_t>(ring ? part - per_state : part) * kCommitF4;
#pragma unroll
    for (int j = 0; j < kCommitF4 / kCommitThreads; ++j) {
        const int64_t i = i0 + j * kCommitThreads + threadIdx.x;
        if (i < n) dst[i] = src[i];
    }
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s) {
    switch (a.prob_type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_commit(const CommitArgs &a, hipStream_t s) {
    const int per_state = static_cast<int>(commit_blocks(a.state_f4));
    const int per_seq = per_state + static_cast<int>(commit_blocks(a.ring_f4));
    const int64_t blocks = static_cast<int64_t>(per_seq) * a.layers * a.B;
    k_commit<<<dim3(static_cast<unsigned>(blocks)), dim3(kCommitThreads), 0, s>>>(a, per_state,
                                                                                  per_seq);
    return hipGetLastError();
}

}  // namespace gdn
