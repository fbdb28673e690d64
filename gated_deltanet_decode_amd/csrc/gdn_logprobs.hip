// gdn_logprobs.hip - gdn_logprobs: log probabilities of given tokens, the
// entropy of each row, and its most likely tokens.
//
// Mathematics.  With m the row's largest logit, Z = sum exp(x - m) and
// T = sum exp(x - m) (x - m):
//   log p(v) = x_v - m - log Z,   H = log Z - T / Z.
// A thread keeps its own m and rescales Z and T when it grows; threads are joined
// in binary64, so that log p of a nearly certain token keeps its digits.
//
// The most likely tokens need no work per entry: the K-th largest of the
// groups' own maxima (a group: the entries of four neighbouring threads) bounds
// the K-th largest entry from below, only the groups that reach it are read
// again (from the caches), and what passes is ranked.  Orders by value, then by
// the lower id: a 64-bit key of both.
//
// One pass over memory, a row in as many units as fill the chip; a second launch
// joins the units where there are several.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_launch.hpp"
#include "gdn_logprobs.hpp"

namespace gdn {
namespace {

constexpr int kT = 256;                      // threads of a workgroup
constexpr int kGroups = kT / 4;
constexpr int kAhead = 4;                    // vectors that a thread fetches at once
constexpr int kList = 512;                   // entries that are ranked at most
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLeast = -3.402823466e38f;

// Orders as the values, -0 as 0; 0 is below every float's.
__device__ __forceinline__ uint32_t order(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __builtin_bit_cast(float, o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int id) {
    return static_cast<uint64_t>(order(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(id));
}
__device__ __forceinline__ int id_of(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }
constexpr uint64_t kNone = 0;                // below every entry's key

// Sums of entries relative to m.
struct Sums {
    float m;
    double z, t;
};
// a joined with b; of NaNs, NaN.
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
    Sums c;
    c.m = fmaxf(a.m, b.m);
    const double da = static_cast<double>(a.m) - c.m, db = static_cast<double>(b.m) - c.m;
    const double ea = exp(da), eb = exp(db);
    c.z = a.z * ea + b.z * eb;
    // the weight of what is far below is 0, whatever its distance
    c.t = (ea > 0.0 ? ea * (a.t + da * a.z) : a.z * 0.0) + (eb > 0.0 ? eb * (b.t + db * b.z) : b.z * 0.0);
    return c;
}
__device__ __forceinline__ Sums from_lane(const Sums &s, int d) {
    return Sums{__shfl_xor(s.m, d), __shfl_xor(s.z, d), __shfl_xor(s.t, d)};
}

// Entries v.. of a row, N of them; those past its end or before v are -inf.
template <typename LT, int N>
__device__ __forceinline__ void load(const typename LT::bits *row, int64_t v, int V, float (&x)[N]) {
    typedef typename LT::bits bits;
    if (v + N <= V) {
        const auto w = Pack<bits, N>::load(row + v);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = LT::get(w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = v + j < V ? LT::get(row[v + j]) : -__builtin_inff();
    }
}

// A row's answer from its sums and its best keys (best[0..top), kNone where there
// are fewer above -inf); the first wave of a workgroup calls it.
template <typename LT>
__device__ __forceinline__ void answer(const LogprobsArgs &a, int64_t row, const Sums &s, const uint64_t *best) {
    const int lane = threadIdx.x & 63;
    const typename LT::bits *x = static_cast<const typename LT::bits *>(a.logits) + row * a.ld;
    const bool bad = !(s.z >= 0.0) || s.m == __builtin_inff();       // a NaN or +inf
    const bool none = s.z == 0.0;                                    // nothing above -inf
    const double lz = log(s.z);
    const auto logprob = [&](float v) {
        // m first: a row of the type's lowest value is uniform
        return bad ? __builtin_nanf("")
                   : none ? -__builtin_inff() : static_cast<float>((static_cast<double>(v) - s.m) - lz);
    };
    if (lane == 0) {
        if (a.entropy) a.entropy[row] = bad ? __builtin_nanf("") : none ? 0.0f : static_cast<float>(lz - s.t / s.z);
        if (a.tokens) {
            const int t = a.tokens[row];
            a.logprob[row] = t >= 0 && t < a.V ? logprob(LT::get(x[t])) : bad ? __builtin_nanf("") : -__builtin_inff();
        }
    }
    if (a.top == 0) return;
    const uint64_t key = lane < a.top ? best[lane] : kNone;
    int found = __popcll(__ballot(key != kNone));
    if (lane < found) {
        a.top_ids[row * a.top + lane] = bad ? -1 : id_of(key);
        a.top_logprobs[row * a.top + lane] = logprob(value_of(key));
    }
    // the others are the first entries of -inf
    for (int64_t v0 = 0; found < a.top && v0 < a.V; v0 += 64) {
        const int64_t v = v0 + lane;
        const bool is = v < a.V && !(LT::get(x[v]) > -__builtin_inff());
        const unsigned long long m = __ballot(is);
        const int at = found + __popcll(m & ((1ull << lane) - 1));
        if (is && at < a.top) {
            a.top_ids[row * a.top + at] = bad ? -1 : static_cast<int>(v);
            a.top_logprobs[row * a.top + at] = bad ? __builtin_nanf("") : -__builtin_inff();
        }
        found += __popcll(m);
    }
}

// One unit of a row: its sums, and its `top` best keys in order.  With one unit a
// row (kOne) the answer follows.  A thread takes N neighbouring entries at a time.
template <typename LT, int N, bool kOne>
__global__ __launch_bounds__(kT) void k_logprobs(LogprobsArgs a, int unit, int units) {
    typedef typename LT::bits bits;
    __shared__ Sums sums[kT / 64];
    __shared__ alignas(16) uint32_t tops[kGroups];
    __shared__ uint64_t list[kList], best[kLogprobsMaxTop];
    __shared__ int groups[kGroups];
    __shared__ int n_groups, n_list;
    __shared__ uint32_t bound_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = kOne ? blockIdx.x : blockIdx.x / units;
    const int u = kOne ? 0 : static_cast<int>(blockIdx.x - row * units);
    const bits *x = static_cast<const bits *>(a.logits) + row * a.ld;
    const int64_t v0 = static_cast<int64_t>(u) * unit;
    const int end = static_cast<int>(min(static_cast<int64_t>(a.V), v0 + unit));
    const int turns = static_cast<int>((end - v0 + kT * N - 1) / (kT * N));   // vectors of a thread

    float m = kLeast, z = 0.0f, t = 0.0f;
    const auto add = [&](const float (&y)[N]) {
        float top = y[0];
#pragma unroll
        for (int j = 1; j < N; ++j) top = fmaxf(top, y[j]);
        if (top > m) {
            const float d = m - top, e = __builtin_amdgcn_exp2f(d * kLog2e);
            t = e > 0.0f ? e * fmaf(d, z, t) : z * 0.0f;
            z *= e;
            m = top;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float d = y[j] - m, e = __builtin_amdgcn_exp2f(d * kLog2e);
            z += e;
            t = fmaf(e, fmaxf(d, -200.0f), t);            // of -inf: 0
        }
    };
    int i = 0;
    for (; v0 + static_cast<int64_t>(i + kAhead) * (kT * N) <= end; i += kAhead) {
        typename Pack<bits, N>::vec w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) w[k] = Pack<bits, N>::load(x + v0 + (static_cast<int64_t>(i + k) * kT + tid) * N);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float y[N];
#pragma unroll
            for (int j = 0; j < N; ++j) y[j] = LT::get(w[k][j]);
            add(y);
        }
    }
    for (; i < turns; ++i) {
        float y[N];
        load<LT, N>(x, v0 + (static_cast<int64_t>(i) * kT + tid) * N, end, y);
        add(y);
    }
    // groups' maxima; the best `top` entries
    if (a.top > 0) {
        float gm = fmaxf(m, __shfl_xor(m, 1));
        gm = fmaxf(gm, __shfl_xor(gm, 2));
        if ((tid & 3) == 0) tops[tid >> 2] = order(gm);
        if (tid == 0) n_groups = n_list = 0;
        if (tid < kLogprobsMaxTop) best[tid] = kNone;
    }
    Sums s{m, z, t};
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s = join(s, from_lane(s, d));
    if (lane == 0) sums[wave] = s;
    __syncthreads();
    if (a.top > 0) {
        if (wave == 0) {
            // a bound that `top` groups at least reach: the top-th largest maximum
            const uint32_t mine = tops[lane];
            int above = 0;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) above += tops[j] > mine || (tops[j] == mine && j < lane);
            const uint32_t least = order(kLeast);
            if (above == min(a.top, kGroups) - 1) bound_s = max(mine, least);
        }
        __syncthreads();
        const uint32_t bound = bound_s;
        if (wave == 0) {
            const bool in = tops[lane] >= bound;
            const unsigned long long b = __ballot(in);
            if (in) groups[__popcll(b & ((1ull << lane) - 1))] = lane;
            if (lane == 0) n_groups = __popcll(b);
        }
        __syncthreads();
        // a wave per listed group, a lane per vector of its threads
        for (int k = wave; k < n_groups; k += kT / 64) {
            const int g4 = groups[k] * 4;
            for (int w = lane; w < turns * 4; w += 64) {
                const int64_t v = v0 + (static_cast<int64_t>(w >> 2) * kT + g4 + (w & 3)) * N;
                float y[N];
                load<LT, N>(x, v, end, y);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (y[j] >= kLeast && order(y[j]) >= bound) {
                        const int at = atomicAdd(&n_list, 1);
                        if (at < kList) list[at] = key_of(y[j], static_cast<int>(v + j));
                    }
            }
        }
        __syncthreads();
        const int n = n_list;
        if (n <= kList) {
            for (int k = tid; k < n; k += kT) {
                const uint64_t key = list[k];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += list[j] > key;
                if (rank < a.top) best[rank] = key;
            }
        } else {
            // many alike: the best one below the last, `top` times
            uint64_t last = ~0ull;
            for (int k = 0; k < a.top; ++k) {
                uint64_t key = kNone;
                for (int w = 0; w < turns; ++w) {
                    const int64_t v = v0 + (static_cast<int64_t>(w) * kT + tid) * N;
                    float y[N];
                    load<LT, N>(x, v, end, y);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const uint64_t c = y[j] >= kLeast ? key_of(y[j], static_cast<int>(v + j)) : kNone;
                        key = c < last && c > key ? c : key;
                    }
                }
#pragma unroll
                for (int d = 1; d < 64; d *= 2) {
                    const uint64_t o = __shfl_xor(static_cast<unsigned long long>(key), d);
                    key = o > key ? o : key;
                }
                __syncthreads();
                if (lane == 0) list[wave] = key;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kT / 64; ++w) key = list[w] > key ? list[w] : key;
                if (tid == 0) best[k] = key;
                last = key;
            }
        }
        __syncthreads();
    }
    if (wave > 0) return;
    s = sums[0];
#pragma unroll
    for (int w = 1; w < kT / 64; ++w) s = join(s, sums[w]);
    if constexpr (kOne) {
        answer<LT>(a, row, s, best);
    } else {
        if (lane == 0) {
            double *to = a.sums + (row * units + u) * 3;
            to[0] = s.m;
            to[1] = s.z;
            to[2] = s.t;
        }
        if (lane < a.top) a.keys[(row * units + u) * a.top + lane] = best[lane];
    }
}

// The units of a row joined by one wave, a unit a lane.
template <typename LT>
__global__ __launch_bounds__(64) void k_join(LogprobsArgs a, int units) {
    __shared__ uint64_t best[kLogprobsMaxTop];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    Sums s{kLeast, 0.0, 0.0};
    const int64_t at = row * units + lane;
    if (lane < units) s = Sums{static_cast<float>(a.sums[at * 3]), a.sums[at * 3 + 1], a.sums[at * 3 + 2]};
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s = join(s, from_lane(s, d));
    int next = 0;                                         // of this lane's unit
    uint64_t head = lane < units && a.top > 0 ? a.keys[at * a.top] : kNone;
    for (int k = 0; k < a.top; ++k) {
        uint64_t key = head;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint64_t o = __shfl_xor(static_cast<unsigned long long>(key), d);
            key = o > key ? o : key;
        }
        if (lane == 0) best[k] = key;
        if (key != kNone && head == key) {
            ++next;
            head = next < a.top ? a.keys[at * a.top + next] : kNone;
        }
    }
    __syncthreads();
    answer<LT>(a, row, s, best);
}

template <typename LT, int N>
hipError_t launch(const LogprobsArgs &a, int64_t units, hipStream_t s) {
    const int unit = static_cast<int>(((a.V + units - 1) / units + N - 1) / N * N);
    if (units == 1) {
        k_logprobs<LT, N, true><<<dim3(static_cast<unsigned>(a.rows)), dim3(kT), 0, s>>>(a, unit, 1);
        return hipGetLastError();
    }
    k_logprobs<LT, N, false>
        <<<dim3(static_cast<unsigned>(a.rows * units)), dim3(kT), 0, s>>>(a, unit, static_cast<int>(units));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_join<LT><<<dim3(static_cast<unsigned>(a.rows)), dim3(64), 0, s>>>(a, static_cast<int>(units));
    return hipGetLastError();
}

template <typename LT>
hipError_t launch(const LogprobsArgs &a, hipStream_t s) {
    // 16 bytes at a time, or single entries where that would leave threads, and so
    // groups, without one: their maxima would not bound anything
    constexpr int N = 16 / sizeof(typename LT::bits);
    const int64_t units = logprobs_units(a.rows, a.V);
    return a.V / units >= kT * N ? launch<LT, N>(a, units, s) : launch<LT, 1>(a, units, s);
}

}  // namespace

hipError_t launch_logprobs(const LogprobsArgs &a, hipStream_t s) {
    switch (a.type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
