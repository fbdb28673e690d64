// gdn_decode.hip - gdn_decode: the delta rule token by token over packed
// sequences of a few tokens each, float32, bfloat16 or float16, with the states
// anywhere in a pool.
#include "gdn.h"
#include "gdn_device.hpp"
#include "gdn_elem.hpp"
#include "gdn_packed.hpp"

namespace gdn {
namespace {

template <typename ET>
__device__ __forceinline__ void load_typed(VecSlice &v, const typename ET::bits *src, int c) {
#pragma unroll
    for (int i = 0; i < kF4PerLane; ++i) {
        const auto x = Pack<typename ET::bits, 4>::load(src + 4 * (kLanesPerRow * i + c));
        v.x[i] = f4{ET::get(x[0]), ET::get(x[1]), ET::get(x[2]), ET::get(x[3])};
    }
}

// One wave per tile of 8 state rows; the arithmetic of gdn_step (row_token).  Memory
// bounds it: 256 sequences of one bf16 token 184 us (5.9 TB/s), of four 239; one
// sequence 3.3 us, a launch.  Two tiles through LDS in workgroups of 512, as gdn_step
// streams them, took 204 us: there the 16-bit vectors wait behind the tile.
template <typename ET>
__global__ __launch_bounds__(64) void k_decode(DecodeArgs a) {
    typedef typename ET::bits bits;
    const int lane = threadIdx.x, grp = lane >> 3, c = lane & 7;
    const int Hv = a.s.Hv, Hk = a.s.Hk;
    const int head = blockIdx.x / kTilesPerHead;
    const int row = (blockIdx.x % kTilesPerHead) * kRowsPerTile + grp;
    const int b = head / Hv, h = head - b * Hv, kh = h % Hk;
    const int slot = slot_of(a.s, b);
    if (slot < 0) return;
    const Span sp = span_of(a.s, b);
    const int64_t at = (static_cast<int64_t>(slot) * Hv + h) * (D * D) + row * D;
    if (sp.len == 0 && a.state == a.state_out) return;
    RowSlice m;
    load_row<true>(m, a.state + at, c);
    for (int t = 0; t < sp.len; ++t) {
        const int64_t tok = sp.first + t, hp = tok * Hv + h;
        VecSlice k, q;
        load_typed<ET>(k, static_cast<const bits *>(a.k) + (tok * Hk + kh) * D, c);
        load_typed<ET>(q, static_cast<const bits *>(a.q) + (tok * Hk + kh) * D, c);
        const float o = row_token(m, k, q, expf(a.gate[hp]), a.beta[hp],
                                  ET::get(static_cast<const bits *>(a.v)[hp * D + row]));
        if (c == 0) static_cast<bits *>(a.out)[hp * D + row] = ET::put(o);
    }
    store_row<true>(a.state_out + at, m, c);
}

template <typename ET>
hipError_t launch(const DecodeArgs &a, hipStream_t s) {
    const unsigned wgs = static_cast<unsigned>(static_cast<int64_t>(a.s.B) * a.s.Hv * kTilesPerHead);
    k_decode<ET><<<dim3(wgs), dim3(64), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const DecodeArgs &a, hipStream_t s) {
    switch (a.s.type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
