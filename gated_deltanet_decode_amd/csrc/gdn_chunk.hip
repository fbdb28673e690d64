// gdn_chunk.hip - gdn_chunk: the delta rule over packed sequences in chunks of
// 64 tokens, on the matrix cores: k_prep over all chunks at once, then k_walk
// along the sequences.
#include "gdn.h"
#include "gdn_walk.hpp"

namespace gdn {
namespace {

template <typename ET, int NP, int NO, int S>
hipError_t launch(const ChunkArgs &a, hipStream_t s) {
    PrepArgs p{};
    p.s = a.s;
    p.q = a.q;
    p.k = a.k;
    p.beta = a.beta;
    p.gate = a.gate;
    p.within = a.within;
    p.kq = a.kq;
    const hipError_t e = launch_prep<ET, NP, NO, false>(p, s);
    if (e != hipSuccess) return e;
    return launch_walk<ET, NP, NO, S, false>(a, s);
}

}  // namespace

hipError_t launch_chunk(const ChunkArgs &a, hipStream_t s) {
    switch (a.s.type) {
    case GDN_F32: return launch<F32, 3, 3, 1>(a, s);
    case GDN_BF16: return launch<BF16, 1, 2, 2>(a, s);
    case GDN_F16: return launch<F16, 2, 2, 1>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
