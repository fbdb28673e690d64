// gdn_logprobs.hip - gdn_logprobs: log probabilities of given tokens, the
// entropy of each row, and its most likely tokens.
//
// Mathematics.  With m the row's largest logit, Z = sum exp(x - m) and
// T = sum exp(x - m) (x - m):
//   log p(v) = x_v - m - log Z,   H = log Z - T / Z.
// A thread keeps its own m and rescales Z and T when it grows; threads are joined
// in binary64, so that log p of a nearly certain token keeps its digits.  In
// powers of two, with c the binary32 number next to log2 e: each term is
// 2^(c x - R), one fma and one exponential, where R is c m rounded to binary32.  From
// |m| = 2^20 on, where that rounding would no longer be small beside 1 (from 2^31 on it
// may pass 2^7: the largest term overflows or vanishes), R is c m itself and a term
// 2^(c (x - m)).  The reference is then R / c in place of m; and as c log 2 = 1 - e,
// e = 1.3e-8, log Z lacks e times the mean of x - R / c, which T gives.
//
// The most likely tokens need no work per entry: the K-th largest of the maxima of
// groups (the entries of four neighbouring threads) bounds the K-th largest entry
// from below, only the entries of threads whose own maximum reaches it are read
// again (from the caches), and what passes is ranked.  Orders by value, then by
// the lower id: a 64-bit key of both.
//
// One pass over memory, a row in as many units as give every compute unit four; a
// second launch joins the units where there are several.  Memory and the vector units
// bound it in turn: eight instructions an entry, one of them an exponential at a quarter of
// the rate, keep these two thirds busy, and the waves wait for memory 72 % of their time.
// 1024 rows x 131071 bf16 54-62 us (4.3-5.0 TB/s), the best 20 with them 73-82 (vectors
// from the row's own start, unaligned: 66 and 85; two units a row and their join: 75 and
// 94); 32 x 128000 with 20 16 us; the next vectors on their way during the sums: no
// gain.  With top near 64 the bound is nearly the groups' smallest maximum, and more
// entries than the list has pass it: then each of the best takes a pass of its own (top
// 48 94 us, 63 119, 64 2400; 32 x 128000 20, 77 and 135).
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
constexpr double kLn2 = 0.693147180559945309417, kLacks = 1.0 - kLn2 * kLog2e;
constexpr float kLarge = 0x1p20f;            // R of a smaller m is off c m by 2^-4 at most
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

// R of m.
__device__ __forceinline__ double reference(float m) {
    return fabsf(m) < kLarge ? static_cast<double>(m * kLog2e) : static_cast<double>(m) * kLog2e;
}
// Sums of the entries' 2^(c x - R) and of these times c x - R.
struct Sums {
    float m;
    double z, t;
};
// L lanes' sums joined in each of them; of NaNs, NaN.
template <int L>
__device__ __forceinline__ Sums joined(const Sums &s) {
    Sums c;
    c.m = s.m;
#pragma unroll
    for (int d = 1; d < L; d *= 2) c.m = fmaxf(c.m, __shfl_xor(c.m, d));
    const double d = reference(s.m) - reference(c.m), e = exp2(d);
    c.z = s.z * e;
    c.t = e > 0.0 ? e * (s.t + d * s.z) : s.z * 0.0;      // what is far below counts 0, whatever its distance
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
        c.z += __shfl_xor(c.z, d);
        c.t += __shfl_xor(c.t, d);
    }
    return c;
}

// Entries v.. of a row, N of them; those outside [first, end) are -inf.
template <typename LT, int N>
__device__ __forceinline__ void load(const typename LT::bits *row, int64_t v, int first, int64_t end, float (&x)[N]) {
    typedef typename LT::bits bits;
    if (v >= first && v + N <= end) {
        const auto w = Pack<bits, N>::load(row + v);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = LT::get(w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = v + j >= first && v + j < end ? LT::get(row[v + j]) : -__builtin_inff();
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
    const double ref = reference(s.m) / kLog2e, mean = s.t / s.z / kLog2e, lz = log(s.z) + kLacks * mean;
    const auto logprob = [&](float v) {
        // m first: a row of the type's lowest value is uniform
        return bad ? __builtin_nanf("")
                   : none ? -__builtin_inff() : static_cast<float>((static_cast<double>(v) - ref) - lz);
    };
    if (lane == 0) {
        if (a.entropy) a.entropy[row] = bad ? __builtin_nanf("") : none ? 0.0f : static_cast<float>(lz - mean);
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
    __shared__ int threads[kT];
    __shared__ int n_threads, n_list;
    __shared__ uint32_t bound_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = kOne ? blockIdx.x : blockIdx.x / units;
    const int u = kOne ? 0 : static_cast<int>(blockIdx.x - row * units);
    // Counted from the 16 bytes that the row begins in, so that vectors are aligned: the
    // first `skip` entries are not the row's.
    const bits *x = static_cast<const bits *>(a.logits) + row * a.ld;
    const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(bits) % N);
    x -= skip;
    const int64_t v0 = static_cast<int64_t>(u) * unit;
    const int end = static_cast<int>(min(static_cast<int64_t>(a.V) + skip, v0 + unit));
    const int turns = static_cast<int>((end - v0 + kT * N - 1) / (kT * N));   // vectors of a thread

    float m = kLeast, z = 0.0f, t = 0.0f;
    // the batch's largest, then its entries by get(j)
    const auto add = [&](float top, int n, auto get) {
        if (top > m) {
            const float d = static_cast<float>(reference(m) - reference(top)), e = __builtin_amdgcn_exp2f(d);
            t = e > 0.0f ? e * fmaf(d, z, t) : z * 0.0f;
            z *= e;
            m = top;
        }
        if (fabsf(m) < kLarge) {
            const float r = m * kLog2e;
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const float d = fmaf(get(j), kLog2e, -r), e = __builtin_amdgcn_exp2f(d);
                z += e;
                t = fmaf(e, fmaxf(d, -300.0f), t);        // of -inf: 0
            }
        } else {
            for (int j = 0; j < n; ++j) {
                const float d = (get(j) - m) * kLog2e, e = __builtin_amdgcn_exp2f(d);
                z += e;
                t = fmaf(e, fmaxf(d, -300.0f), t);
            }
        }
    };
    int i = 0;
    const auto slow = [&](int i) {                        // a vector that may reach over the row's ends
        float y[N];
        load<LT, N>(x, v0 + (static_cast<int64_t>(i) * kT + tid) * N, skip, end, y);
        float top = y[0];
#pragma unroll
        for (int j = 1; j < N; ++j) top = fmaxf(top, y[j]);
        add(top, N, [&](int j) { return y[j]; });
    };
    if (v0 < skip) slow(i++);
    for (; v0 + static_cast<int64_t>(i + kAhead) * (kT * N) <= end; i += kAhead) {
        typename Pack<bits, N>::vec w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) w[k] = Pack<bits, N>::load(x + v0 + (static_cast<int64_t>(i + k) * kT + tid) * N);
        float top = LT::get(w[0][0]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) top = fmaxf(top, LT::get(w[k][j]));
        add(top, kAhead * N, [&](int j) { return LT::get(w[j / N][j % N]); });
    }
    for (; i < turns; ++i) slow(i);
    // groups' maxima; the best `top` entries
    if (a.top > 0) {
        float gm = fmaxf(m, __shfl_xor(m, 1));
        gm = fmaxf(gm, __shfl_xor(gm, 2));
        if ((tid & 3) == 0) tops[tid >> 2] = order(gm);
        if (tid == 0) n_threads = n_list = 0;
        if (tid < kLogprobsMaxTop) best[tid] = kNone;
    }
    Sums s = joined<64>(Sums{m, z, t});
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
        if (order(m) >= bound) threads[atomicAdd(&n_threads, 1)] = tid;
        __syncthreads();
        // the listed threads' vectors, neighbouring threads' side by side
        const int listed = n_threads;
        for (int w = tid; w < listed * turns; w += kT) {
            const int turn = w / listed;
            const int64_t v = v0 + (static_cast<int64_t>(turn) * kT + threads[w - turn * listed]) * N;
            float y[N];
            load<LT, N>(x, v, skip, end, y);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (y[j] >= kLeast && order(y[j]) >= bound) {
                    const int at = atomicAdd(&n_list, 1);
                    if (at < kList) list[at] = key_of(y[j], static_cast<int>(v + j) - skip);
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
                    load<LT, N>(x, v, skip, end, y);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const uint64_t c = y[j] >= kLeast ? key_of(y[j], static_cast<int>(v + j) - skip) : kNone;
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
    s = joined<kT / 64>(sums[lane % (kT / 64)]);
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

// The units of a row joined: the sums by the first wave, and each unit's keys, which
// are in order: those that reach a bound, which `top` of them do, are ranked.
template <typename LT>
__global__ __launch_bounds__(kT) void k_join(LogprobsArgs a, int units) {
    constexpr int kKeys = kLogprobsMaxUnits * kLogprobsMaxTop;
    __shared__ uint64_t keys[kKeys], list[kKeys], best[kLogprobsMaxTop], bound;
    __shared__ int n_list;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    Sums s{kLeast, 0.0, 0.0};
    if (tid < units) {
        const double *from = a.sums + (row * units + tid) * 3;
        s = Sums{static_cast<float>(from[0]), from[1], from[2]};
    }
    if (a.top > 0) {
        const int all = units * a.top;
        for (int i = tid; i < all; i += kT) keys[i] = a.keys[row * all + i];
        if (tid < kLogprobsMaxTop) best[tid] = kNone;
        if (tid == 0) n_list = 0;
        __syncthreads();
        // `of` units have `each` keys at or above the bound, `top` together
        const int each = min(a.top, (2 * a.top + units - 1) / units), of = (a.top + each - 1) / each;
        if (tid < units) {
            const uint64_t mine = keys[tid * a.top + each - 1];
            int above = 0;
            for (int u = 0; u < units; ++u) {
                const uint64_t key = keys[u * a.top + each - 1];
                above += key > mine || (key == mine && u < tid);
            }
            if (above == of - 1) bound = mine;
        }
        __syncthreads();
        for (int i = tid; i < all; i += kT)
            if (keys[i] != kNone && keys[i] >= bound) list[atomicAdd(&n_list, 1)] = keys[i];
        __syncthreads();
        const int n = n_list;
        for (int i = tid; i < n; i += kT) {
            const uint64_t key = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += list[j] > key;
            if (rank < a.top) best[rank] = key;
        }
        __syncthreads();
    }
    if (tid >= 64) return;
    s = joined<64>(s);
    answer<LT>(a, row, s, best);
}

template <typename LT, int N>
hipError_t launch(const LogprobsArgs &a, int64_t units, hipStream_t s) {
    // (a row's first vector may begin N - 1 entries before it)
    const int unit = static_cast<int>(((a.V + N - 1 + units - 1) / units + N - 1) / N * N);
    if (units == 1) {
        k_logprobs<LT, N, true><<<dim3(static_cast<unsigned>(a.rows)), dim3(kT), 0, s>>>(a, unit, 1);
        return hipGetLastError();
    }
    k_logprobs<LT, N, false>
        <<<dim3(static_cast<unsigned>(a.rows * units)), dim3(kT), 0, s>>>(a, unit, static_cast<int>(units));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_join<LT><<<dim3(static_cast<unsigned>(a.rows)), dim3(kT), 0, s>>>(a, static_cast<int>(units));
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
