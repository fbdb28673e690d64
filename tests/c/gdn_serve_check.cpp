// gdn_serve_check.cpp - the C-ABI layer of the operators around the recurrent
// branch (gdn_serve_api.cpp) on the host alone, under AddressSanitizer and
// UndefinedBehaviorSanitizer, with recording stubs in place of the kernel
// launchers: size limits at and one past their boundary, overlaps to the
// byte, and what a call that passes hands to its launcher.  Device buffers
// are stand-in addresses that nothing reads through.  Test infrastructure.

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "gdn.h"
#include "gdn_serve.hpp"

namespace {
int launches = 0, failures = 0, checks = 0;
bool fail_next = false;
gdn::QuantArgs quant;
gdn::LinearArgs linear;
gdn::VerifyArgs verify;
gdn::CommitArgs commit;
hipStream_t last_stream;

hipError_t seen(hipStream_t s) {
    ++launches;
    last_stream = s;
    const bool f = fail_next;
    fail_next = false;
    return f ? hipErrorLaunchFailure : hipSuccess;
}
}  // namespace

namespace gdn {
hipError_t launch_quant(const QuantArgs &a, hipStream_t s) { quant = a; return seen(s); }
hipError_t launch_linear(const LinearArgs &a, hipStream_t s) { linear = a; return seen(s); }
hipError_t launch_verify(const VerifyArgs &a, hipStream_t s) { verify = a; return seen(s); }
hipError_t launch_commit(const CommitArgs &a, hipStream_t s) { commit = a; return seen(s); }
}  // namespace gdn

namespace {

void expect(bool ok, const char *what, int line) {
    ++checks;
    if (!ok) {
        std::fprintf(stderr, "line %d: expected %s (last error \"%s\")\n", line, what,
                     gdn_last_error());
        ++failures;
    }
}
#define EXPECT(c) expect((c), #c, __LINE__)

// The call must fail with `code` and a message holding `needle`, launching nothing.
template <typename F>
void refused(int code, const char *needle, int line, F f) {
    const int before = launches;
    const int rc = f();
    expect(rc == code && std::strstr(gdn_last_error(), needle) && launches == before, needle, line);
}
#define REFUSED(code, needle, call) refused(code, needle, __LINE__, [&] { return call; })
#define ACCEPTED(call)                                             \
    do {                                                           \
        const int before__ = launches;                             \
        EXPECT((call) == GDN_OK && launches == before__ + 1);      \
        EXPECT(gdn_last_error()[0] == '\0' && last_stream == S);   \
    } while (0)

char *slot(int i) { return reinterpret_cast<char *>(static_cast<uintptr_t>(i + 1) << 44); }
float *F(int i) { return reinterpret_cast<float *>(slot(i)); }
int8_t *C(int i) { return reinterpret_cast<int8_t *>(slot(i)); }
int32_t *I(int i) { return reinterpret_cast<int32_t *>(slot(i)); }
const hipStream_t S = reinterpret_cast<hipStream_t>(0x5eed0);

void check_quant() {
    ACCEPTED(gdn_add_rmsnorm_q8(3, 5, GDN_BF16, slot(0), GDN_F32, slot(1), slot(2), F(3), 0.5f,
                                C(4), F(5), S));
    EXPECT(quant.rows == 3 && quant.n == 5 && quant.x_type == GDN_BF16 &&
           quant.residual_type == GDN_F32 && quant.eps == 0.5f && quant.norm_w == F(3) &&
           quant.residual == slot(1) && quant.residual_out == slot(2));
    // in place; neighbours that touch but do not overlap: 15 codes, then scales
    ACCEPTED(gdn_add_rmsnorm_q8(3, 5, GDN_BF16, slot(0), GDN_F32, slot(1), slot(1), F(3), 0.f, C(4),
                                reinterpret_cast<float *>(slot(4) + 16), S));
    REFUSED(GDN_ERR_ALIAS, "q", gdn_add_rmsnorm_q8(3, 5, GDN_BF16, slot(0), GDN_F32, slot(1),
            slot(1), F(3), 0.f, C(4), reinterpret_cast<float *>(slot(4) + 12), S));
    ACCEPTED(gdn_add_rmsnorm_q8(4194303, 1073741823, GDN_F32, slot(0), GDN_NONE, nullptr, nullptr,
                                reinterpret_cast<float *>(uintptr_t(1) << 60), 0.f,
                                reinterpret_cast<int8_t *>(uintptr_t(1) << 61), F(5000), S));
    EXPECT(quant.residual == nullptr && quant.residual_out == nullptr);
    REFUSED(GDN_ERR_SHAPE, "n must", gdn_quantize_q8(1, 1073741824, GDN_F32, slot(0), C(1), F(2), S));
    REFUSED(GDN_ERR_SHAPE, "rows", gdn_quantize_q8(4194304, 8, GDN_F32, slot(0), C(1), F(2), S));
    ACCEPTED(gdn_quantize_q8(4194303, 8, GDN_F16, slot(0), C(1), F(2), S));
    EXPECT(quant.norm_w == nullptr && quant.x_type == GDN_F16 && quant.residual_type == GDN_NONE);
    fail_next = true;
    EXPECT(gdn_quantize_q8(1, 8, GDN_F16, slot(0), C(1), F(2), S) == GDN_ERR_HIP &&
           std::strstr(gdn_last_error(), "gdn_quantize_q8 launch"));
    ACCEPTED(gdn_quantize_q8(1, 8, GDN_F16, slot(0), C(1), F(2), S));
}

void check_linear() {
    const gdn_linear_out outs[4] = {{slot(5), 3}, {slot(6), 4}, {slot(7), 5}, {slot(8), 6}};
    for (int n = 1; n <= 4; ++n) {
        ACCEPTED(gdn_linear_q8(2, 7, C(0), F(1), C(2), F(3), n & 1 ? F(4) : nullptr, GDN_F16, outs,
                               n, S));
        int end = 0;
        for (int i = 0; i < 4; ++i) {
            if (i < n) end += outs[i].n;
            EXPECT(linear.end[i] == end && linear.out[i] == (i < n ? outs[i].out : nullptr));
        }
        EXPECT(linear.N == end && linear.M == 2 && linear.K == 7 &&
               linear.bias == (n & 1 ? F(4) : nullptr));
    }
    REFUSED(GDN_ERR_SHAPE, "n_outs", gdn_linear_q8(2, 7, C(0), F(1), C(2), F(3), nullptr, GDN_F16,
            outs, 5, S));
    ACCEPTED(gdn_linear_q8(2, 131071, C(0), F(1), C(2), F(3), nullptr, GDN_F16, outs, 1, S));
    REFUSED(GDN_ERR_SHAPE, "K must", gdn_linear_q8(2, 131072, C(0), F(1), C(2), F(3), nullptr,
            GDN_F16, outs, 1, S));
    const gdn_linear_out wide[2] = {{slot(500), (1 << 27) - 2}, {slot(600), 1}};
    ACCEPTED(gdn_linear_q8(64, 1, C(0), F(100), C(200), F(300), nullptr, GDN_F32, wide, 2, S));
    EXPECT(linear.N == (1 << 27) - 1);
    const gdn_linear_out wider[2] = {{slot(500), (1 << 27) - 2}, {slot(600), 2}};
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_linear_q8(64, 1, C(0), F(100), C(200), F(300), nullptr,
            GDN_F32, wider, 2, S));
    const gdn_linear_out one[1] = {{slot(500), 64}};
    ACCEPTED(gdn_linear_q8(64 * 4194303, 1, C(0), F(100), C(200), F(300), nullptr, GDN_F32, one, 1, S));
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_linear_q8(64 * 4194303 + 1, 1, C(0), F(100), C(200),
            F(300), nullptr, GDN_F32, one, 1, S));
    const gdn_linear_out two[1] = {{slot(500), 65}};
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_linear_q8(64 * 4194303, 1, C(0), F(100), C(200), F(300),
            nullptr, GDN_F32, two, 1, S));
    // outputs that touch: [2][4] of two bytes ends where the next may begin
    const gdn_linear_out touch[2] = {{slot(5), 4}, {slot(5) + 16, 4}};
    ACCEPTED(gdn_linear_q8(2, 7, C(0), F(1), C(2), F(3), nullptr, GDN_BF16, touch, 2, S));
    REFUSED(GDN_ERR_ALIAS, "outs[", gdn_linear_q8(2, 7, C(0), F(1), C(2), F(3), nullptr, GDN_F32,
            touch, 2, S));
    fail_next = true;
    EXPECT(gdn_linear_q8(2, 7, C(0), F(1), C(2), F(3), nullptr, GDN_F16, outs, 2, S) == GDN_ERR_HIP);
}

void check_verify() {
    const size_t need = gdn_verify_workspace_bytes(3, 5000);
    ACCEPTED(gdn_verify(3, 2, 5000, GDN_BF16, slot(0), slot(1), I(2), I(3), F(4), F(5), I(6), I(7),
                        slot(8), need, S));
    EXPECT(verify.B == 3 && verify.K == 2 && verify.V == 5000 && verify.n_draft == I(3) &&
           verify.partial == reinterpret_cast<double *>(slot(8)) && verify.draft == slot(1) &&
           reinterpret_cast<char *>(verify.rows) + 3 * 16 == slot(8) + need);
    ACCEPTED(gdn_verify(3, 2, 5000, GDN_BF16, slot(0), nullptr, I(2), nullptr, F(4), F(5), I(6),
                        I(7), slot(8), need, S));
    EXPECT(verify.draft == nullptr && verify.n_draft == nullptr);
    REFUSED(GDN_ERR_WORKSPACE, "needed", gdn_verify(3, 2, 5000, GDN_BF16, slot(0), slot(1), I(2),
            I(3), F(4), F(5), I(6), I(7), slot(8), need - 1, S));
    // accepted [3] ends 12 bytes on; tokens may begin there
    ACCEPTED(gdn_verify(3, 2, 5000, GDN_F32, slot(0), slot(1), I(2), I(3), F(4), F(5), I(6),
                        I(6) + 3, slot(8), need, S));
    REFUSED(GDN_ERR_ALIAS, "accepted", gdn_verify(3, 2, 5000, GDN_F32, slot(0), slot(1), I(2), I(3),
            F(4), F(5), I(6), I(6) + 2, slot(8), need, S));
    // [3][3][5000] of 4 bytes: the workspace may begin right behind the target
    ACCEPTED(gdn_verify(3, 2, 5000, GDN_F32, slot(0), slot(1), I(2), I(3), F(4), F(5), I(6), I(7),
                        slot(0) + 180000, need, S));
    REFUSED(GDN_ERR_ALIAS, "target", gdn_verify(3, 2, 5000, GDN_F32, slot(0), slot(1), I(2), I(3),
            F(4), F(5), I(6), I(7), slot(0) + 179984, need, S));
    const size_t most = gdn_verify_workspace_bytes(65535, 2147483647);
    EXPECT(most > 0);
    ACCEPTED(gdn_verify(65535, 1024, 2147483647, GDN_F16, slot(0), nullptr, I(50000), nullptr,
                        F(50001), F(50002), I(50003), I(50004), slot(60000), most, S));
    REFUSED(GDN_ERR_SHAPE, "B must", gdn_verify(65536, 1, 5, GDN_F16, slot(0), slot(1), I(2), I(3),
            F(4), F(5), I(6), I(7), slot(8), most, S));
    REFUSED(GDN_ERR_SHAPE, "K must", gdn_verify(1, 1025, 5, GDN_F16, slot(0), slot(1), I(2), I(3),
            F(4), F(5), I(6), I(7), slot(8), most, S));
}

void check_commit() {
    const gdn_dims page = {32, 16, 128, 128};
    ACCEPTED(gdn_pair_commit(&page, 2, 3, I(0), F(1), F(2), 24576, F(3), F(4), S));
    EXPECT(commit.layers == 2 && commit.B == 3 && commit.state_f4 == 32 * 4096 &&
           commit.ring_f4 == 6144 && commit.ring == F(3) && commit.ring_next == F(4));
    ACCEPTED(gdn_pair_commit(&page, 1, 3, I(0), F(1), F(2), 0, nullptr, nullptr, S));
    EXPECT(commit.ring == nullptr && commit.ring_f4 == 0);
    REFUSED(GDN_ERR_SHAPE, "conv_floats", gdn_pair_commit(&page, 1, 3, I(0), F(1), F(2), 0, F(3),
            F(4), S));
    REFUSED(GDN_ERR_NULL, "conv_state", gdn_pair_commit(&page, 1, 3, I(0), F(1), F(2), 8, nullptr,
            F(4), S));
    // 64 blocks a sequence: 262143 of them, and one more
    const int most = 16777215 / 64;
    ACCEPTED(gdn_pair_commit(&page, 1, most, I(0), F(1000), F(2000), 0, nullptr, nullptr, S));
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_pair_commit(&page, 1, most + 1, I(0), F(1000), F(2000),
            0, nullptr, nullptr, S));
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_pair_commit(&page, 1, most, I(0), F(1000), F(2000), 4,
            F(3000), F(4000), S));
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_pair_commit(&page, 2147483647, 2147483, I(0), F(1000),
            F(2000), 0, nullptr, nullptr, S));
    const gdn_dims one = {1, 1, 128, 128};
    ACCEPTED(gdn_pair_commit(&one, 1, 8388607, I(0), F(1000), F(2000), 0, nullptr, nullptr, S));
    ACCEPTED(gdn_pair_commit(&one, 1, 8, I(0), F(1000), F(2000), 2147483644, F(3000), F(4000), S));
    REFUSED(GDN_ERR_SHAPE, "too large", gdn_pair_commit(&one, 1, 64, I(0), F(1000), F(2000),
            2147483644, F(3000), F(4000), S));
}

}  // namespace

int main() {
    check_quant();
    check_linear();
    check_verify();
    check_commit();
    if (failures) {
        std::printf("serve ABI host check: %d of %d checks failed\n", failures, checks);
        return 1;
    }
    std::printf("serve ABI host check ok (%d checks)\n", checks);
    return 0;
}
