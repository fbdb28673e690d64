// gdn_quant.hip - gdn_add_rmsnorm_q8 and gdn_quantize_q8: residual addition,
// RMS norm and 8-bit codes of a row, in one pass over memory.
//
// Mathematics.  With h the (summed) row, g_i = h_i w_i, G = max|g_i| and
// r = 1 / sqrt(mean(h^2) + eps), the normed row is y_i = r g_i and its codes
// are rint(127 y_i / max|y|).  r cancels: q_i = rint(127 g_i / G), and only the
// scale r G / 127 needs it.  h and w are binary32, so g_i is exact in binary64
// and a code depends on nothing but the row's own products; the quotient is
// formed as g_i * (127 / G), at most 4e-14 off, and a value that close to a
// border is divided out (so ties are those of the formula).  The sum of
// squares is kept in binary64 too.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_serve.hpp"

namespace gdn {
namespace {

// One code: t = g * (127 / G) is within 4e-14 of 127 g / G.
__device__ __forceinline__ int code(double g, double inv, double top) {
    const double t = g * inv;
    double c = rint(t);
    if (fabs(fabs(t - c) - 0.5) < 1e-12) c = rint(127.0 * g / top);
    return static_cast<int>(c);
}

struct NoType {
    typedef uint32_t bits;
};

// One workgroup of T threads per row; the row is held in registers when it
// fits, CH vectors of V elements a thread, and read again otherwise.
template <typename XT, typename RT, bool kNorm, int T>
__global__ __launch_bounds__(T) void k_quant(QuantArgs a) {
    constexpr bool kRes = !__is_same(RT, NoType);
    constexpr int NW = T / 64;
    __shared__ double red[3][NW];
    const int64_t row = blockIdx.x;
    const int n = a.n;
    const typename XT::bits *x = static_cast<const typename XT::bits *>(a.x) + row * n;
    const typename RT::bits *r = static_cast<const typename RT::bits *>(a.residual) + row * n;
    typename RT::bits *ro = static_cast<typename RT::bits *>(a.residual_out) + row * n;

    double top = 0.0, ss = 0.0;
    for (int i = threadIdx.x; i < n; i += T) {
        float h = XT::get(x[i]);
        if constexpr (kRes) {
            const typename RT::bits b = RT::put(h + RT::get(r[i]));
            ro[i] = b;
            h = RT::get(b);
        }
        const double g = kNorm ? static_cast<double>(h) * static_cast<double>(a.norm_w[i])
                               : static_cast<double>(h);
        top = fmax(top, fabs(g));
        ss = fma(g, 0.0, ss);               // NaN once any product is not finite
        if constexpr (kNorm) ss = fma(static_cast<double>(h), static_cast<double>(h), ss);
    }
    top = wave_max(top);
    ss = wave_sum(ss);
    if ((threadIdx.x & 63) == 0) {
        red[0][threadIdx.x >> 6] = top;
        red[1][threadIdx.x >> 6] = ss;
    }
    __syncthreads();
    top = red[0][0];
    ss = red[1][0];
    for (int w = 1; w < NW; ++w) {
        top = fmax(top, red[0][w]);
        ss += red[1][w];
    }
    const bool bad = !(ss <= 1.7976931348623157e308);     // NaN or infinite
    const double inv = top > 0.0 && !bad ? 127.0 / top : 0.0;
    int8_t *q = a.q + row * n;
    for (int i = threadIdx.x; i < n; i += T) {
        float h;
        if constexpr (kRes)
            h = RT::get(ro[i]);
        else
            h = XT::get(x[i]);
        const double g = kNorm ? static_cast<double>(h) * static_cast<double>(a.norm_w[i])
                               : static_cast<double>(h);
        q[i] = inv == 0.0 ? 0 : static_cast<int8_t>(code(g, inv, top));
    }
    if (threadIdx.x == 0) {
        double scale = top / 127.0;
        if constexpr (kNorm)
            scale = scale / sqrt(ss / static_cast<double>(n) + static_cast<double>(a.eps));
        if (top == 0.0) scale = 0.0;
        if (bad) scale = __builtin_nan("");
        a.scale[row] = static_cast<float>(scale);
    }
}

template <typename XT, typename RT, bool kNorm>
hipError_t launch(const QuantArgs &a, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.rows));
    k_quant<XT, RT, kNorm, 256><<<grid, dim3(256), 0, s>>>(a);
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
