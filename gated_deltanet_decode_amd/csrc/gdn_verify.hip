// gdn_verify.hip - gdn_verify (speculative verification from given random
// numbers) and gdn_pair_commit (the accepted sequences' tentative states).
//
// Mathematics.  Drafted token d of position i is accepted when all before it
// are and u q_i(d) < p_i(d); the token after the accepted run is drawn by
// inverting the cumulative sum of w = max(p - q, 0) at the refusal (or of p
// when no draft is left).  Probabilities of at most 24 significant bits make
// the product exact in binary64, and with it what is accepted.  The sums round:
// a lane's 16 or 32 terms (V / 16384 of a large V), the scans over lanes, units
// and entries, and scans less their own term: at most 80 + V / 16384 roundings of
// 2^-53 of the total on a path.  The token is the definition's unless the goal
// lies that close to a cumulative sum; then it may be another entry with a weight
// and a sum as close (where the unit's entries, summed in another order than the
// units, do not pass the goal, the unit's last one with a weight).
//
// Only one row of the target and at most one of the draft matter to a
// sequence, once the run of accepted tokens is known, and that takes 2 K
// single entries.  The row is summed in at most kVerifyUnits units, a wave each;
// the sums' own cumulative sum names the unit where the goal is passed, and
// only that unit is read again.  One launch sums the units, a second one picks;
// nothing has to be cleared between calls.  One sequence: 6.3 us from a graph for
// 32000 and 6.8 for 262144 entries, a chain of about five dependent loads and
// two launches (a single workgroup for all of it took 15 and 31; 1024 threads
// that pick instead of 256, 14).  256 sequences x 3 drafts x 131071 bf16: 20 us
// for the sums and 5 to pick; the rows that matter come at 4.5 TB/s sampled
// (91 MB) and 3.3 greedy (67 MB), and the vector units are busy 63 and 73 % of
// that time: the binary64 conversions and sums of each entry weigh more than
// memory.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_launch.hpp"
#include "gdn_serve.hpp"

namespace gdn {
namespace {

constexpr int kT = 256;                      // threads of a workgroup

// Negative, infinite and NaN entries count as 0.
__device__ __forceinline__ double weight(float p) {
    const float c = fmaxf(p, 0.0f);                       // NaN too
    return static_cast<double>(c <= 3.402823466e38f ? c : 0.0f);
}

struct Row {          // what a sequence's next token is drawn from
    int accepted;
    int refused;      // position `accepted` refused a draft
    int token;        // that draft
};

// The run of accepted drafts of sequence b.  Called by whole waves; every lane
// returns the same.  Each position's entries are fetched whether or not it has
// a draft, so that they do not wait for n_draft.
template <typename PT>
__device__ __forceinline__ Row decide(const VerifyArgs &a, int64_t b) {
    typedef typename PT::bits bits;
    const int lane = threadIdx.x & 63;
    const int given = a.n_draft ? a.n_draft[b] : a.K;
    for (int i0 = 0;; i0 += 64) {
        const int i = i0 + lane;
        bool good = false;
        int d = -1;
        if (i < a.K) {
            d = a.draft_tokens[b * a.K + i];
            const float u = a.u_accept[b * a.K + i];
            if (d >= 0 && d < a.V) {
                const double p = weight(PT::get(
                    static_cast<const bits *>(a.target)[(b * (a.K + 1) + i) * a.V + d]));
                const double q = a.draft ? weight(PT::get(
                    static_cast<const bits *>(a.draft)[(b * a.K + i) * a.V + d])) : 1.0;
                good = static_cast<double>(u) * q < p;
            }
        }
        const int n = max(0, min(given, a.K));
        const unsigned long long m = __ballot(i < n && !good);
        if (m) {
            const int first = __ffsll(m) - 1;
            return Row{i0 + first, 1, __builtin_amdgcn_readlane(d, first)};
        }
        if (i0 + 64 >= n) return Row{n, 0, -1};
    }
}

// The weights of the row: max(p - q, 0), or p.
enum Mode { kPlain, kDraft, kGreedy };    // p; p - q; p less 1 at one entry
template <typename PT>
struct Weights {
    typedef typename PT::bits bits;
    const bits *p;
    const bits *q;
    int one;           // the entry where a greedy draft's q is 1
    int V;
    Mode mode;

    __device__ __forceinline__ Weights(const VerifyArgs &a, int64_t b, const Row &r) {
        p = static_cast<const bits *>(a.target) + (b * (a.K + 1) + r.accepted) * a.V;
        q = static_cast<const bits *>(a.draft) + (b * a.K + r.accepted) * a.V;
        one = r.token;
        V = a.V;
        mode = !r.refused ? kPlain : a.draft ? kDraft : kGreedy;
    }
    // N entries from v on as they are stored (kIn: they lie in the row).  A vector
    // that would pass the row's end is fetched further left, so that no load waits
    // for a branch; `first` is its first entry.
    template <int N>
    struct Raw {
        typename Pack<bits, N>::vec p, q;
        int64_t v, first;
    };
    template <int N, Mode kMode, bool kIn>
    __device__ __forceinline__ void fetch(int64_t v, Raw<N> &r) const {
        r.v = v;
        r.first = kIn ? v : min(v, static_cast<int64_t>(V) - N);
        if (kIn || V >= N) {
            r.p = Pack<bits, N>::load(p + r.first);
            if constexpr (kMode == kDraft) r.q = Pack<bits, N>::load(q + r.first);
        } else {                                          // a row shorter than a vector
            r.p = {};
            r.q = {};
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (r.first + j >= 0) {
                    r.p[j] = p[r.first + j];
                    if constexpr (kMode == kDraft) r.q[j] = q[r.first + j];
                }
        }
    }
    // The weight of its entry first + j, 0 for those before v.
    template <int N, Mode kMode, bool kIn>
    __device__ __forceinline__ double value(const Raw<N> &r, int j) const {
        double z = weight(PT::get(r.p[j]));
        if constexpr (kMode == kDraft) z = fmax(z - weight(PT::get(r.q[j])), 0.0);
        if constexpr (kMode == kGreedy) z = r.first + j == one ? fmax(z - 1.0, 0.0) : z;
        return kIn || r.first + j >= r.v ? z : 0.0;
    }
    template <int N, Mode kMode>
    __device__ __forceinline__ int64_t at(int64_t v, double (&z)[N]) const {
        Raw<N> r;
        fetch<N, kMode, false>(v, r);
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = value<N, kMode, false>(r, j);
        return r.first;
    }
    // N weights from v on, zeros past the row; returns the entry of the first.
    template <int N>
    __device__ __forceinline__ int64_t any(int64_t v, double (&z)[N]) const {
        if (mode == kPlain) return at<N, kPlain>(v, z);
        if (mode == kDraft) return at<N, kDraft>(v, z);
        return at<N, kGreedy>(v, z);
    }
};

// Inclusive sums over the wave's lanes, and the total: within rows of 16 lanes by
// DPP, then the rows' sums by lane reads.
__device__ __forceinline__ double scan(double x, double &total) {
    x += dpp<0x111>(x);                                   // row_shr 1, 2, 4, 8
    x += dpp<0x112>(x);
    x += dpp<0x114>(x);
    x += dpp<0x118>(x);
    const double r0 = lane_of(x, 15), r1 = lane_of(x, 31), r2 = lane_of(x, 47), r3 = lane_of(x, 63);
    const int row = (threadIdx.x & 63) >> 4;
    const double r01 = r0 + r1, r012 = r01 + r2;
    total = r012 + r3;
    return (row == 0 ? 0.0 : row == 1 ? r0 : row == 2 ? r01 : r012) + x;
}

constexpr int kAhead = 4;                    // vectors of a row that a lane fetches at once

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

// The sum of a unit's weights, by one wave; every lane gets the same.
template <typename PT, Mode kMode>
__device__ __forceinline__ double unit_sum(const Weights<PT> &w, int64_t v0, int unit) {
    constexpr int N = 16 / sizeof(typename PT::bits);
    const int lane = threadIdx.x & 63;
    double s = 0.0, total;
    const auto sum = [&](auto in) {
        constexpr bool kIn = decltype(in)::value;
        for (int i = 0; i < unit && v0 + i < w.V; i += 64 * N * kAhead) {
            typename Weights<PT>::template Raw<N> r[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                w.template fetch<N, kMode, kIn>(v0 + i + (k * 64 + lane) * N, r[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int j = 0; j < N; ++j) s += w.template value<N, kMode, kIn>(r[k], j);
        }
    };
    if (v0 + unit <= w.V) sum(Flag<true>{});
    else sum(Flag<false>{});
    scan(s, total);
    return total;
}
template <typename PT>
__device__ __forceinline__ double unit_sum(const Weights<PT> &w, int64_t v0, int unit) {
    if (w.mode == kPlain) return unit_sum<PT, kPlain>(w, v0, unit);
    if (w.mode == kDraft) return unit_sum<PT, kDraft>(w, v0, unit);
    return unit_sum<PT, kGreedy>(w, v0, unit);
}

// Finds the unit and the entry where the cumulative sum passes u_sample times the
// total, and writes the sequence's answer.  sums[0..kVerifyUnits) holds the
// units' sums, zeros past the last, behind a barrier; the whole workgroup calls.
template <typename PT>
__device__ __forceinline__ void pick(const VerifyArgs &a, int64_t b, const Row &row, int unit,
                                     double *sums) {
    __shared__ double totals[2][kT / 64];
    __shared__ int hits[kT / 64], ends[kT / 64];          // a wave's first entry past the goal, its last live one
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float u_sample = a.u_sample[b];
    const int drafted = tid < a.K ? a.draft_tokens[b * a.K + tid] : -1;
    Weights<PT> w(a, b, row);
    // every wave finds the unit by itself: four sums a lane
    constexpr int S = kVerifyUnits / 64;
    double x[S], run, total;
    for (;;) {
        double own = 0.0;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            x[j] = sums[lane * S + j];
            own += x[j];
        }
        run = scan(own, total) - own;
        if (total > 0.0 || w.mode == kPlain) break;
        // nothing is left of p behind the draft: p itself, seldom
        w.mode = kPlain;
        __syncthreads();
        for (int u = wave; static_cast<int64_t>(u) * unit < w.V; u += kT / 64) {
            const double s = unit_sum(w, static_cast<int64_t>(u) * unit, unit);
            if (lane == 0) sums[u] = s;
        }
        __syncthreads();
    }
    const double goal = static_cast<double>(u_sample) * total;
    int hit = -1, end = -1;                               // this lane's first unit past the goal, last live one
    double hit_base = 0.0, end_base = 0.0;
#pragma unroll
    for (int j = 0; j < S; ++j) {
        if (x[j] > 0.0) {
            end = lane * S + j;
            end_base = run;
            if (run + x[j] > goal && hit < 0) {
                hit = end;
                hit_base = run;
            }
        }
        run += x[j];
    }
    int u = -1;                                           // -1: no entry has a weight
    double base = 0.0;
    if (const unsigned long long m = __ballot(hit >= 0)) {
        const int l = __ffsll(m) - 1;
        u = __builtin_amdgcn_readlane(hit, l);
        base = lane_of(hit_base, l);
    } else if (const unsigned long long e = __ballot(end >= 0)) {
        const int l = 63 - __clzll(e);
        u = __builtin_amdgcn_readlane(end, l);
        base = lane_of(end_base, l);
    }
    int token = -1;
    if (u >= 0) {
        int found = -1;
        end = -1;
        for (int i = 0, turn = 0; i < unit; i += 4 * kT, turn ^= 1) {
            const int64_t v = static_cast<int64_t>(u) * unit + i + tid * 4;
            double z[4], wave_total;
            const int64_t first = w.any(v, z);
            const double sum = ((z[0] + z[1]) + z[2]) + z[3];
            double c = scan(sum, wave_total) - sum;
            if (lane == 0) totals[turn][wave] = wave_total;
            __syncthreads();
            double all = base;
#pragma unroll
            for (int k = 0; k < kT / 64; ++k) {
                if (k == wave) c += all;
                all += totals[turn][k];
            }
            base = all;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c += z[j];
                if (z[j] > 0.0) {
                    end = static_cast<int>(first + j);
                    if (c > goal && found < 0) found = end;
                }
            }
            // entries lie in the order of lanes, waves and turns; the barrier above is
            // behind every read of the turn before
            const unsigned long long h = __ballot(found >= 0), e = __ballot(end >= 0);
            const int first_hit = h ? __builtin_amdgcn_readlane(found, __ffsll(h) - 1) : -1;
            const int last_end = e ? __builtin_amdgcn_readlane(end, 63 - __clzll(e)) : -1;
            if (lane == 0) {
                hits[wave] = first_hit;
                ends[wave] = last_end;
            }
            __syncthreads();
            int hit_now = -1;
#pragma unroll
            for (int k = kT / 64 - 1; k >= 0; --k) hit_now = hits[k] >= 0 ? hits[k] : hit_now;
#pragma unroll
            for (int k = 0; k < kT / 64; ++k) token = ends[k] >= 0 ? ends[k] : token;
            if (hit_now >= 0) {
                token = hit_now;
                break;
            }
            found = end = -1;
        }
    }
    int32_t *out = a.tokens + b * (a.K + 1);
    if (tid < a.K) out[tid] = tid < row.accepted ? drafted : tid == row.accepted ? token : -1;
    for (int i = tid + kT; i < a.K; i += kT)
        out[i] = i < row.accepted ? a.draft_tokens[b * a.K + i] : i == row.accepted ? token : -1;
    if (tid == 0) {
        out[a.K] = row.accepted == a.K ? token : -1;
        a.accepted[b] = row.accepted;
    }
}

// The units' sums, a wave each, and the decision, for k_verify_pick.
template <typename PT>
__global__ __launch_bounds__(kT) void k_verify_sums(VerifyArgs a, int unit, int units) {
    const int64_t b = blockIdx.y;
    const Row row = decide<PT>(a, b);
    const Weights<PT> w(a, b, row);
    for (int u = blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += gridDim.x * 4) {
        const double s = unit_sum(w, static_cast<int64_t>(u) * unit, unit);
        if ((threadIdx.x & 63) == 0) a.partial[b * kVerifyUnits + u] = s;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        int32_t *r = a.rows + b * 4;
        r[0] = row.accepted;
        r[1] = row.refused;
        r[2] = row.token;
    }
}
template <typename PT>
__global__ __launch_bounds__(kT) void k_verify_pick(VerifyArgs a, int unit, int units) {
    __shared__ double sums[kVerifyUnits];
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x;
    const int32_t *r = a.rows + b * 4;
    const Row row{r[0], r[1], r[2]};
    static_assert(kVerifyUnits == kT, "");
    sums[tid] = tid < units ? a.partial[b * kVerifyUnits + tid] : 0.0;
    __syncthreads();
    pick<PT>(a, b, row, unit, sums);
}

template <typename PT>
hipError_t launch(const VerifyArgs &a, hipStream_t s) {
    // a unit is what a wave fetches at once, or more where that makes over
    // kVerifyUnits of them
    const int64_t step = 64 * kAhead * (16 / sizeof(typename PT::bits));
    const int64_t turns = (a.V + step * kVerifyUnits - 1) / (step * kVerifyUnits);
    const int unit = static_cast<int>(step * turns);
    const int units = static_cast<int>((a.V + static_cast<int64_t>(unit) - 1) / unit);
    // a wave per unit, or about 2048 workgroups in all (1024 to 8192 within 5 %)
    const int most = (2048 + a.B - 1) / a.B;
    const unsigned wide = static_cast<unsigned>(min((units + 3) / 4, most));
    k_verify_sums<PT><<<dim3(wide, static_cast<unsigned>(a.B)), dim3(kT), 0, s>>>(a, unit, units);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_verify_pick<PT><<<dim3(static_cast<unsigned>(a.B)), dim3(kT), 0, s>>>(a, unit, units);
    return hipGetLastError();
}

// ------------------------------------------------------------------ commit
typedef float f4 __attribute__((ext_vector_type(4)));

// One workgroup copies kCommitF4 float4s (32 KiB) of one sequence's state or ring
// in one layer, if its draft was accepted: a copy, bound by memory.  All its loads
// are on their way before the first store, and both stream past the caches as
// the step does: 256 sequences, 70 % accepted, 128 us = 6.1 TB/s (140-153 us
// through the caches or with loads and stores in turn).
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
    constexpr int N = kCommitF4 / kCommitThreads;
    if (i0 + kCommitF4 <= n) {
        f4 v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = __builtin_nontemporal_load(src + i0 + j * kCommitThreads + threadIdx.x);
#pragma unroll
        for (int j = 0; j < N; ++j)
            __builtin_nontemporal_store(v[j], dst + i0 + j * kCommitThreads + threadIdx.x);
    } else {
        for (int64_t i = i0 + threadIdx.x; i < n; i += kCommitThreads) dst[i] = src[i];
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
