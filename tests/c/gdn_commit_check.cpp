// gdn_commit_check.cpp - what gdn_pair_commit hands to its launcher when one
// sequence's state passes 2^31 float4s, on the host alone, under
// AddressSanitizer and UndefinedBehaviorSanitizer, with a recording stub in
// place of the launch.  Device buffers are stand-in addresses that nothing
// reads through.  Test infrastructure.

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "gdn.h"
#include "gdn_serve.hpp"

namespace {
int launches = 0, failures = 0;
gdn::CommitArgs commit;
}  // namespace

namespace gdn {
hipError_t launch_quant(const QuantArgs &, hipStream_t) { return hipErrorLaunchFailure; }
hipError_t launch_linear(const LinearArgs &, hipStream_t) { return hipErrorLaunchFailure; }
hipError_t launch_verify(const VerifyArgs &, hipStream_t) { return hipErrorLaunchFailure; }
hipError_t launch_commit(const CommitArgs &a, hipStream_t) {
    commit = a;
    ++launches;
    return hipSuccess;
}
}  // namespace gdn

namespace {

void expect(bool ok, const char *what, int32_t heads) {
    if (ok) return;
    std::fprintf(stderr, "%d heads: expected %s (last error \"%s\")\n", heads, what, gdn_last_error());
    ++failures;
}

float *F(int i) { return reinterpret_cast<float *>(static_cast<uintptr_t>(i) << 44); }

int call(int32_t heads, int32_t B, int32_t conv_floats) {
    const gdn_dims d = {heads, 1, 128, 128};
    return gdn_pair_commit(&d, 1, B, reinterpret_cast<int32_t *>(F(1)), F(2), F(3), conv_floats,
                           conv_floats ? F(4) : nullptr, conv_floats ? F(5) : nullptr, nullptr);
}

// A call that passes hands over all of a sequence's state, 4096 float4s a head,
// in as many workgroups as the grid holds.
void accepted(int32_t heads, int32_t B, int32_t conv_floats) {
    const int before = launches;
    expect(call(heads, B, conv_floats) == GDN_OK && launches == before + 1, "GDN_OK and one launch", heads);
    expect(static_cast<int64_t>(commit.state_f4) == static_cast<int64_t>(heads) * 4096, "4096 float4s a head",
           heads);
    expect(commit.B == B && commit.ring_f4 == conv_floats / 4, "B and the ring", heads);
    expect(gdn::commit_blocks(commit.state_f4) == 2 * static_cast<int64_t>(heads), "two workgroups a head", heads);
}

}  // namespace

int main() {
    for (const int32_t heads : {1, 32, 524287, 524288, 524289, 1048575, 1048576, 1048577, 1048608, 8388607}) {
        accepted(heads, 1, 0);
        if (heads < 8388607) accepted(heads, 1, 24576);
        if (heads < 4194304) accepted(heads, 2, 0);
    }
    const int before = launches;
    for (const int32_t heads : {8388608, 134213631})
        expect(call(heads, 1, 0) == GDN_ERR_SHAPE && std::strstr(gdn_last_error(), "too large"), "GDN_ERR_SHAPE",
               heads);
    expect(call(8388607, 1, 24576) == GDN_ERR_SHAPE, "GDN_ERR_SHAPE with a ring", 8388607);
    expect(launches == before, "no launch", 0);
    if (failures) {
        std::printf("commit host check: %d failed\n", failures);
        return 1;
    }
    std::printf("commit host check ok\n");
    return 0;
}
