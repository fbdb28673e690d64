// gdn_quant.hip - gdn_add_rmsnorm_q8 and gdn_quantize_q8: residual addition,
// RMS norm and 8-bit codes of a row, in one pass over memory.
//
// Mathematics.  With h the (summed) row, g_i = h_i w_i, G = max|g_i| and
// r = 1 / sqrt(mean(h^2) + eps), the normed row is y_i = r g_i and its codes
// are rint(127 y_i / max|y|).  r cancels: q_i = rint(127 g_i / G), and only the
// scale r G / 127 needs it.  h and w are binary32, so g_i is exact in binary64
// and a code depends on nothing but the row's own products.  The quotient is
// formed as g_i (127 / G), in binary32 for rows of ordinary magnitude (at most
// 3.1e-5 off) and in binary64 for the others and for long rows (4e-14); a value
// that close to a border is settled by an exact comparison, ties included.  The sum
// of squares is kept in binary64, so that the scale rounds once.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_serve.hpp"

namespace gdn {
namespace {

struct NoType {
    typedef uint32_t bits;
};

constexpr double kRound = 6755399441055744.0;             // 1.5 * 2^52
constexpr float kRound32 = 12582912.0f;                   // 1.5 * 2^23

// The code of a product whose quotient t = 127 g / top, known to 4e-5, lies near a
// border k + 1/2 (k = floor(|t|)): 254 |g| against (2 k + 1) top, exactly.  g and
// top are products of two 24-bit numbers, multiples of units u and v with
// |g| < 2^48 u and top < 2^48 v; next to a border 256 |g| - (2 k + 1) top is about
// 2 |g| <= 2 top, and so below 2^50 times the smaller unit: the fused step and the
// subtraction after it are exact.  127 g alone takes up to 55 bits, so a rounded
// quotient is not enough here.  It is without a norm, where g and top have 24 bits:
// 127 g is exact, and a quotient that is no tie is 2^-33 or more off one (20001 x
// 4097 bf16 40 us for 42 with the comparison).
template <bool kNorm>
__device__ __forceinline__ uint32_t settled(double g, double top) {
    if constexpr (!kNorm) return static_cast<uint32_t>(__builtin_bit_cast(uint64_t, 127.0 * g / top + kRound));
    const double a = fabs(g), k = floor(127.0 * a / top);
    const double past = fma(-(2.0 * k + 1.0), top, 256.0 * a) - 2.0 * a;
    const int n = static_cast<int>(k), q = past > 0.0 ? n + 1 : past < 0.0 ? n : n + (n & 1);
    return static_cast<uint32_t>(g < 0.0 ? -q : q);
}

// One code, as the low byte of a word, in binary64: t = g * (127 / G) is within
// 4e-14 of 127 g / G, and a value that near a border is settled.  Adding 1.5 * 2^52
// rounds t to an integer, ties to even, and leaves it in the low word.
template <bool kNorm>
__device__ __forceinline__ uint32_t code(double g, double inv, double top) {
    const double t = g * inv, s = t + kRound;
    if (fabs(t - (s - kRound)) > 0.5 - 1e-12) return settled<kNorm>(g, top);
    return static_cast<uint32_t>(__builtin_bit_cast(uint64_t, s));
}

__device__ __forceinline__ uint32_t magnitude(float x) {  // orders as |x|, infinities and NaN last
    return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// Reductions over a row's T threads; every thread gets the same bits.  Within
// sixteen lanes by DPP (xor 1, xor 2, mirrors of 8 and 16), then over the wave's
// four rows of lanes, then over the waves through `red` (a value each).
template <int T, typename V, typename F>
__device__ __forceinline__ V reduce(V x, V *red, F join) {
    x = join(x, dpp<0xB1>(x));
    x = join(x, dpp<0x4E>(x));
    x = join(x, dpp<0x141>(x));
    x = join(x, dpp<0x140>(x));
    if constexpr (T > 16) x = join(join(lane_of(x, 0), lane_of(x, 16)), join(lane_of(x, 32), lane_of(x, 48)));
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) x = join(x, red[w]);
    }
    return x;
}
__device__ __forceinline__ double larger(double x, double y) { return fmax(x, y); }
__device__ __forceinline__ double plus(double x, double y) { return x + y; }

// 127 / top for the codes (0: all codes are 0) and the row's scale, from its largest
// product and its sum of squares, which is NaN where a product is not finite.
__device__ __forceinline__ bool finite(double ss) { return ss <= 1.7976931348623157e308; }
__device__ __forceinline__ double inverse(double top, double ss) {
    return top > 0.0 && finite(ss) ? 127.0 / top : 0.0;
}
template <bool kNorm>
__device__ __forceinline__ float scale_of(const QuantArgs &a, double top, double ss) {
    if (!finite(ss)) return __builtin_nanf("");
    if (top == 0.0) return 0.0f;
    double s = top / 127.0;
    if constexpr (kNorm) s = s / sqrt(ss / static_cast<double>(a.n) + static_cast<double>(a.eps));
    return static_cast<float>(s);
}

// A row's elements 0..end-1, whole chunks of V, read and written at any element's
// alignment.
template <typename XT, typename RT>
constexpr int chunk_of() {                                // 16 bytes of the wider input
    return sizeof(typename XT::bits) == 4 || (!__is_same(RT, NoType) && sizeof(typename RT::bits) == 4) ? 4 : 8;
}
template <typename XT, typename RT, bool kNorm, int V>
struct RowOf {
    static constexpr bool kRes = !__is_same(RT, NoType);
    typedef typename XT::bits xbits;
    typedef typename RT::bits rbits;
    const xbits *x;
    const rbits *r;
    rbits *ro;
    const float *w;
    int8_t *q;
    int end;

    struct Chunk {
        typename Pack<xbits, V>::vec x;
        typename Pack<rbits, V>::vec r;
        typename Pack<float, V>::vec w;
    };

    __device__ __forceinline__ RowOf(const QuantArgs &a, int64_t row) {
        const int64_t at = row * a.n;
        x = static_cast<const xbits *>(a.x) + at;
        r = static_cast<const rbits *>(a.residual) + at;
        ro = static_cast<rbits *>(a.residual_out) + at;
        w = a.norm_w;
        q = a.q + at;
        end = a.n - a.n % V;
    }
    // Elements i..i+V-1, zeros past the end.
    __device__ __forceinline__ void load(Chunk &c, int i) const {
        if (i < end) {
            c.x = Pack<xbits, V>::load(x + i);
            if constexpr (kRes) c.r = Pack<rbits, V>::load(r + i);
            if constexpr (kNorm) c.w = Pack<float, V>::load(w + i);
        } else {
            c = Chunk{};
        }
    }
    // The chunk's values: with kStore the residual is added, rounded and stored;
    // without it c.r is that sum.
    template <bool kStore>
    __device__ __forceinline__ void values(Chunk &c, int i, float (&h)[V]) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            h[j] = XT::get(c.x[j]);
            if constexpr (kRes) {
                if constexpr (kStore) c.r[j] = RT::put(h[j] + RT::get(c.r[j]));
                h[j] = RT::get(c.r[j]);
            }
        }
        if constexpr (kRes && kStore) {
            if (i < end) Pack<rbits, V>::store(ro + i, c.r);
        }
    }
    __device__ __forceinline__ double product(const Chunk &c, const float (&h)[V], int j) const {
        if constexpr (kNorm) return static_cast<double>(h[j]) * static_cast<double>(c.w[j]);
        return static_cast<double>(h[j]);
    }
    __device__ __forceinline__ float product32(const Chunk &c, const float (&h)[V], int j) const {
        if constexpr (kNorm) return h[j] * c.w[j];
        return h[j];
    }
    // What the chunk adds to the row's largest product (binary32) and sum of squares
    // (binary64, which costs nothing beside the loads: 32768 x 2048 bf16 with a
    // residual 86 us, squares added in pairs in binary32 85; 10000 x 6001 f16 110 and 134).
    __device__ __forceinline__ void narrow(const Chunk &c, const float (&h)[V], uint32_t &m, double &ss) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            m = max(m, magnitude(product32(c, h, j)));
            if constexpr (kNorm) ss = fma(static_cast<double>(h[j]), static_cast<double>(h[j]), ss);
        }
    }
    // The exact largest of the products that round to magnitude m, joined into
    // *slot (positive binary64 values order as integers).
    __device__ __forceinline__ void settle(const Chunk &c, const float (&h)[V], uint32_t m,
                                           unsigned long long *slot) const {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (magnitude(product32(c, h, j)) == m)
                atomicMax(slot, __builtin_bit_cast(unsigned long long, fabs(product(c, h, j))));
    }
    // The same in binary64; a product that is not finite makes the sum NaN.
    __device__ __forceinline__ void wide(const Chunk &c, const float (&h)[V], double &top, double &ss) const {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double p = product(c, h, j);
            if constexpr (kNorm) ss = fma(static_cast<double>(h[j]), static_cast<double>(h[j]), ss);
            ss = fma(p, 0.0, ss);
            top = fmax(top, fabs(p));
        }
    }
    __device__ __forceinline__ void put(const uint32_t (&b)[V], int i) const {
        if (i >= end) return;
        if constexpr (V == 1) {
            q[i] = static_cast<int8_t>(b[0]);
        } else {
            typename Pack<uint32_t, V / 4>::vec v;
#pragma unroll
            for (int j = 0; j < V / 4; ++j)
                v[j] = (b[4 * j] & 255u) | (b[4 * j + 1] & 255u) << 8 | (b[4 * j + 2] & 255u) << 16 |
                       b[4 * j + 3] << 24;
            typedef uint32_t any __attribute__((ext_vector_type(V / 4), aligned(1)));
            *reinterpret_cast<any *>(q + i) = v;
        }
    }
    __device__ __forceinline__ void codes(const Chunk &c, const float (&h)[V], int i, double inv,
                                          double top) const {
        uint32_t b[V];
#pragma unroll
        for (int j = 0; j < V; ++j) b[j] = inv == 0.0 ? 0u : code<kNorm>(product(c, h, j), inv, top);
        put(b, i);
    }
    // The same codes from binary32: product, top, reciprocal and the last product
    // each round, so t is within 127 * 4 * 2^-24 = 3.1e-5 of 127 g / G; what lies
    // within 4e-5 of a border is settled in binary64.
    __device__ __forceinline__ void codes32(const Chunk &c, const float (&h)[V], int i, float inv,
                                            double top) const {
        uint32_t b[V];
        uint32_t near = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float t = product32(c, h, j) * inv;
            const float s = t + kRound32;
            near |= fabsf(t - (s - kRound32)) > 0.5f - 4e-5f ? 1u << j : 0u;
            b[j] = __builtin_bit_cast(uint32_t, s);
        }
        while (near) {                                    // seldom: one element at a time
            const int k = __ffs(near) - 1;
            near &= near - 1;
            double g = 0.0;
#pragma unroll
            for (int j = 0; j < V; ++j) g = j == k ? product(c, h, j) : g;
            const uint32_t e = settled<kNorm>(g, top);
#pragma unroll
            for (int j = 0; j < V; ++j) b[j] = j == k ? e : b[j];
        }
        put(b, i);
    }
};

// T threads per row (R rows a workgroup, so R = 1 or T = 16 or 64), the row in
// registers: CH chunks a thread.  512 threads are held to four waves a SIMD, so
// that a compute unit holds two rows (10000 x 4100 f32: 66 us against 113).  Rows of ordinary magnitude are worked in
// binary32 where that is exact enough and in binary64 where it is not: binary64
// throughout is right too, but 20 such operations an element bound the kernel
// (32768 x 2048 bf16 with a residual: 129 us against 86).
template <typename XT, typename RT, bool kNorm, int T, int CH, int R>
__global__ __launch_bounds__(T * R, T == 512 ? 4 : 1) void k_quant_row(QuantArgs a) {
    constexpr int V = chunk_of<XT, RT>();
    typedef RowOf<XT, RT, kNorm, V> Row;
    typedef RowOf<XT, RT, kNorm, 1> One;
    static_assert(R == 1 || T == 64 || T == 16, "");
    constexpr int W = (T + 63) / 64;                      // a row's waves
    __shared__ uint32_t red_m[W];
    __shared__ double red_s[W], red_t[W], red_u[W];
    __shared__ unsigned long long exact[R];
    const int tid = threadIdx.x % T;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / T;
    if (id >= a.rows) return;                             // whole rows of lanes; no barrier if R > 1
    if (kNorm && tid == 0) exact[threadIdx.x / T] = 0;    // joined behind the first reduction's barrier
    const Row row(a, id);
    // the elements past the last whole chunk, one a thread
    const One one(a, id);
    const bool odd = row.end < one.end;
    const int o = row.end + tid;
    typename Row::Chunk c[CH];
    typename One::Chunk oc = {};
    float h[CH][V], oh[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < CH; ++k) row.load(c[k], (k * T + tid) * V);
    uint32_t m = 0;
    double ss = 0.0;
    if (odd) {
        one.load(oc, o);
        one.template values<true>(oc, o, oh);
        one.narrow(oc, oh, m, ss);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        row.template values<true>(c[k], (k * T + tid) * V, h[k]);
        row.narrow(c[k], h[k], m, ss);
    }
    m = reduce<T>(m, red_m, [](uint32_t x, uint32_t y) { return max(x, y); });
    if constexpr (kNorm) ss = reduce<T>(ss, red_s, plus);
    // 2^-60 <= the largest product < 2^126: no binary32 product over- or underflowed
    // where it counts, and none is infinite or NaN (those have the largest magnitudes)
    const bool plain = m >= 0x21800000u && m < 0x7e800000u;
    double top;
    if (plain) {
        top = static_cast<double>(__builtin_bit_cast(float, m));
        if constexpr (kNorm) {
            unsigned long long *slot = &exact[threadIdx.x / T];
#pragma unroll
            for (int k = 0; k < CH; ++k) row.settle(c[k], h[k], m, slot);
            if (odd) one.settle(oc, oh, m, slot);
            if constexpr (T > 64) __syncthreads();
            else __threadfence_block();
            top = __builtin_bit_cast(double, *static_cast<volatile unsigned long long *>(slot));
        }
        const float inv = 127.0f / static_cast<float>(top);
#pragma unroll
        for (int k = 0; k < CH; ++k) row.codes32(c[k], h[k], (k * T + tid) * V, inv, top);
        if (odd) one.codes32(oc, oh, o, inv, top);
    } else {
        top = ss = 0.0;
#pragma unroll
        for (int k = 0; k < CH; ++k) row.wide(c[k], h[k], top, ss);
        if (odd) one.wide(oc, oh, top, ss);
        top = reduce<T>(top, red_t, larger);
        ss = reduce<T>(ss, red_u, plus);
        const double inv = inverse(top, ss);
#pragma unroll
        for (int k = 0; k < CH; ++k) row.codes(c[k], h[k], (k * T + tid) * V, inv, top);
        if (odd) one.codes(oc, oh, o, inv, top);
    }
    if (tid == 0) a.scale[id] = scale_of<kNorm>(a, top, ss);
}

// Rows too long for registers: two passes in binary64, the second over what the
// first stored (or over x), which is still in the caches.
template <typename XT, typename RT, bool kNorm>
__global__ __launch_bounds__(1024) void k_quant_long(QuantArgs a) {
    constexpr int V = chunk_of<XT, RT>();
    typedef RowOf<XT, RT, kNorm, V> Row;
    typedef RowOf<XT, RT, kNorm, 1> One;
    __shared__ double red_t[16], red_s[16];
    const int tid = threadIdx.x;
    Row row(a, blockIdx.x);
    const One one(a, blockIdx.x);
    const int o = row.end + tid;
    typename Row::Chunk c;
    typename One::Chunk oc;
    float h[V], oh[1];
    double top = 0.0, ss = 0.0;
    one.load(oc, o);
    one.template values<true>(oc, o, oh);
    one.wide(oc, oh, top, ss);
    for (int i = tid * V; i < row.end; i += 1024 * V) {
        row.load(c, i);
        row.template values<true>(c, i, h);
        row.wide(c, h, top, ss);
    }
    top = reduce<1024>(top, red_t, larger);
    ss = reduce<1024>(ss, red_s, plus);
    const double inv = inverse(top, ss);
    if (tid == 0) a.scale[blockIdx.x] = scale_of<kNorm>(a, top, ss);
    one.codes(oc, oh, o, inv, top);
    row.r = row.ro;                                       // this thread's own stores
    for (int i = tid * V; i < row.end; i += 1024 * V) {
        row.load(c, i);
        row.template values<false>(c, i, h);
        row.codes(c, h, i, inv, top);
    }
}

template <typename XT, typename RT, bool kNorm>
hipError_t launch(const QuantArgs &a, hipStream_t s) {
    // Threads a row by its length alone, so a row's bits do not depend on how many
    // there are; 8 or 16 elements a thread, 32 in long rows without a norm (1600 x
    // 16000 bf16 22 us for 26; with a norm their registers leave too few waves: 10000
    // x 6001 f16 with a residual 131 us for 110, 3000 x 12000 bf16 288 for 66).  us on
    // 100000 rows: 16 lanes a row 23 at 100 bf16 with a residual and 36 at 256, a
    // wave a row 65 and 60; 116 at 512 f32, 256 threads a row 197.  On 32768 x 2048
    // bf16 with a residual: 256 threads 86, a wave a row 196.
    const unsigned rows = static_cast<unsigned>(a.rows);
    constexpr int V = chunk_of<XT, RT>(), C8 = 8 / V, C16 = 16 / V;
    const int body = a.n - a.n % V;
    if (body <= 128)
        k_quant_row<XT, RT, kNorm, 16, C8, 16><<<dim3((rows + 15) / 16), dim3(256), 0, s>>>(a);
    else if (body <= 256)
        k_quant_row<XT, RT, kNorm, 16, C16, 16><<<dim3((rows + 15) / 16), dim3(256), 0, s>>>(a);
    else if (body <= 512)
        k_quant_row<XT, RT, kNorm, 64, C8, 4><<<dim3((rows + 3) / 4), dim3(256), 0, s>>>(a);
    else if (body <= 1024)
        k_quant_row<XT, RT, kNorm, 64, C16, 4><<<dim3((rows + 3) / 4), dim3(256), 0, s>>>(a);
    else if (body <= 2048)
        k_quant_row<XT, RT, kNorm, 256, C8, 1><<<dim3(rows), dim3(256), 0, s>>>(a);
    else if (body <= 4096)
        k_quant_row<XT, RT, kNorm, 256, C16, 1><<<dim3(rows), dim3(256), 0, s>>>(a);
    else if (body <= 8192)
        k_quant_row<XT, RT, kNorm, kNorm ? 512 : 256, kNorm ? C16 : 2 * C16, 1>
            <<<dim3(rows), dim3(kNorm ? 512 : 256), 0, s>>>(a);
    else if (body <= 16384)
        k_quant_row<XT, RT, kNorm, kNorm ? 1024 : 512, kNorm ? C16 : 2 * C16, 1>
            <<<dim3(rows), dim3(kNorm ? 1024 : 512), 0, s>>>(a);
    else
        k_quant_long<XT, RT, kNorm><<<dim3(rows), dim3(1024), 0, s>>>(a);
    return hipGetLastError();
}

template <typename XT>
hipError_t launch_x(const QuantArgs &a, hipStream_t s) {
    if (!a.norm_w) return launch<XT, NoType, false>(a, s);
    switch (a.residual_type) {
    case GDN_F32: return launch<XT, F32, true>(a, s);
    case GDN_BF16: return launch<XT, BF16, true>(a, s);
    case GDN_F16: return launch<XT, F16, true>(a, s);
    case GDN_NONE: return launch<XT, NoType, true>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_quant(const QuantArgs &a, hipStream_t s) {
    switch (a.x_type) {
    case GDN_F32: return launch_x<F32>(a, s);
    case GDN_BF16: return launch_x<BF16>(a, s);
    case GDN_F16: return launch_x<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
