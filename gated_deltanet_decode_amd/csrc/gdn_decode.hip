// gdn_decode.hip - gdn_decode: the delta rule token by token over packed
// sequences of a few tokens each, float32, bfloat16 or float16, with the states
// anywhere in a pool.
#include "gdn.h"
#include "gdn_device.hpp"
#include "gdn_elem.hpp"
#include "gdn_packed.hpp"

namespace gdn {
namespace {

// A lane's share of a vector, as it is in memory.
template <typename ET>
struct Raw {
    typedef Pack<typename ET::bits, 4> P;
    typename P::vec x[kF4PerLane];
    __device__ __forceinline__ void load(const typename ET::bits *src, int c) {
#pragma unroll
        for (int i = 0; i < kF4PerLane; ++i) x[i] = P::load(src + 4 * (kLanesPerRow * i + c));
    }
    __device__ __forceinline__ VecSlice get() const {
        VecSlice v;
#pragma unroll
        for (int i = 0; i < kF4PerLane; ++i) v.x[i] = f4{ET::get(x[i][0]), ET::get(x[i][1]), ET::get(x[i][2]), ET::get(x[i][3])};
        return v;
    }
};

// One wave per tile of 8 state rows; the arithmetic of gdn_step (row_token).  Memory
// bounds it: 256 sequences of one bf16 token 179 us (6.0 TB/s), of four 245; one
// sequence 3.3 us, a launch.  Each token's vectors fetched when it is its turn, in fewer
// registers: 183 and 240 us, float32 186 for 178.  Two tiles through LDS in workgroups of
// 512, as gdn_step streams them, took 204 us: there the 16-bit vectors wait behind the
// tile.
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
    if (sp.len > 0) {
        Raw<ET> k, q;
        float gate, beta;
        bits v;
        const auto fetch = [&](int t) {
            const int64_t tok = sp.first + t, hp = tok * Hv + h;
            k.load(static_cast<const bits *>(a.k) + (tok * Hk + kh) * D, c);
            q.load(static_cast<const bits *>(a.q) + (tok * Hk + kh) * D, c);
            gate = a.gate[hp];
            beta = a.beta[hp];
            v = static_cast<const bits *>(a.v)[hp * D + row];
        };
        fetch(0);
        for (int t = 0; t < sp.len; ++t) {
            const VecSlice kv = k.get(), qv = q.get();
            const float e = expf(gate), bt = beta, vj = ET::get(v);
            if (t + 1 < sp.len) fetch(t + 1);             // the next token's, while this one is worked on
            const float o = row_token(m, kv, qv, e, bt, vj);
            if (c == 0) static_cast<bits *>(a.out)[((sp.first + t) * static_cast<int64_t>(Hv) + h) * D + row] = ET::put(o);
        }
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
