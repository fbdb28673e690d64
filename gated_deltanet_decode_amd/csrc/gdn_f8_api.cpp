// gdn_f8_api.cpp - the C ABI of the 8-bit floating point operators
// (gdn_quantize_f8, gdn_linear_f8): argument validation and dispatch, as in
// gdn_api.cpp.

#include "gdn.h"

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "gdn_check.hpp"
#include "gdn_f8.hpp"

namespace {

using gdn::Buf;
using gdn::check_alias;
using gdn::check_ptrs;
using gdn::check_type;
using gdn::clear_error;
using gdn::fail;
using gdn::hip_status;
using gdn::type_bytes;

int64_t blocks_of(int64_t n) { return (n + gdn::kF8Block - 1) / gdn::kF8Block; }

}  // namespace

extern "C" {

int gdn_quantize_f8(int32_t rows, int32_t n, int32_t block_rows, int32_t x_type, const void *x, uint8_t *q,
                    float *scale, void *stream) {
    clear_error();
    GDN_TRY(check_type(x_type, "x_type"));
    if (block_rows != 1 && block_rows != gdn::kF8Block)
        return fail(GDN_ERR_SHAPE, "block_rows must be 1 or %d (got %d)", gdn::kF8Block, block_rows);
    if (rows < 1) return fail(GDN_ERR_SHAPE, "rows must be >= 1 (got %d)", rows);
    // the kernels' element index stays clear of 2^31
    if (n < 1 || n > (1 << 30) - 1)
        return fail(GDN_ERR_SHAPE, "n must be in [1, 1073741823] (got %d)", n);
    // eight work-items a block of a row, 256 a square one
    const int64_t tall = block_rows == 1 ? rows : blocks_of(rows);
    const int64_t scales = tall * blocks_of(n), most = block_rows == 1 ? (1 << 29) - 32 : (1 << 24) - 1;
    if (scales > most)
        return fail(GDN_ERR_SHAPE, "rows = %d, n = %d: %lld scales, at most %lld", rows, n, (long long)scales,
                    (long long)most);
    const size_t e = static_cast<size_t>(rows) * n;
    const Buf vec[] = {{"x", x, e * type_bytes(x_type)}, {"q", q, e}};
    const Buf sc[] = {{"scale", scale, static_cast<size_t>(scales) * sizeof(float)}};
    GDN_TRY(check_ptrs(vec, 2, 16));
    GDN_TRY(check_ptrs(sc, 1, 4));
    const Buf all[] = {vec[0], vec[1], sc[0]};
    const Buf outs[] = {vec[1], sc[0]};
    GDN_TRY(check_alias(outs, 2, all, 3));

    gdn::QuantF8Args a{};
    a.x = x;
    a.q = q;
    a.scale = scale;
    a.rows = rows;
    a.n = n;
    a.block_rows = block_rows;
    a.x_type = x_type;
    (void)hipGetLastError();
    return hip_status(gdn::launch_quant_f8(a, static_cast<hipStream_t>(stream)), "gdn_quantize_f8 launch");
}

int gdn_linear_f8(int32_t M, int32_t K, const uint8_t *a, const float *a_scale, const uint8_t *w,
                  const float *w_scale, const float *bias, int32_t out_type, const gdn_linear_out *outs,
                  int32_t n_outs, void *stream) {
    static_assert(GDN_LINEAR_MAX_OUTS == gdn::kLinearMaxOuts, "");
    clear_error();
    GDN_TRY(check_type(out_type, "out_type"));
    if (M < 1) return fail(GDN_ERR_SHAPE, "M must be >= 1 (got %d)", M);
    // an offset into a tile's 256 rows stays below 2^31
    if (K < 1 || K > gdn::kTileMaxK)
        return fail(GDN_ERR_SHAPE, "K must be in [1, %d] (got %d)", gdn::kTileMaxK, K);
    if (n_outs < 1 || n_outs > GDN_LINEAR_MAX_OUTS)
        return fail(GDN_ERR_SHAPE, "n_outs must be in [1, %d] (got %d)", GDN_LINEAR_MAX_OUTS, n_outs);
    if (!outs) return fail(GDN_ERR_NULL, "outs is NULL");
    int64_t N = 0;
    for (int i = 0; i < n_outs; ++i) {
        if (outs[i].n < 1)
            return fail(GDN_ERR_SHAPE, "outs[%d].n must be >= 1 (got %d)", i, outs[i].n);
        N += outs[i].n;
    }
    const int64_t tiles = ((static_cast<int64_t>(M) + 63) / 64) * ((N + 63) / 64);
    if (N > (1 << 27) - 1 || tiles > 4194303)
        return fail(GDN_ERR_SHAPE, "M = %d, N = %lld is too large", M, (long long)N);

    static const char *const kOut[] = {"outs[0]", "outs[1]", "outs[2]", "outs[3]"};
    Buf vec[2 + GDN_LINEAR_MAX_OUTS] = {{"a", a, static_cast<size_t>(M) * K}, {"w", w, static_cast<size_t>(N) * K}};
    for (int i = 0; i < n_outs; ++i)
        vec[2 + i] = {kOut[i], outs[i].out, static_cast<size_t>(M) * outs[i].n * type_bytes(out_type)};
    const size_t kb = static_cast<size_t>(blocks_of(K)) * sizeof(float);
    const Buf sc[] = {{"a_scale", a_scale, M * kb},
                      {"w_scale", w_scale, static_cast<size_t>(blocks_of(N)) * kb},
                      {"bias", bias, static_cast<size_t>(N) * sizeof(float)}};
    const int n_sc = bias ? 3 : 2;
    GDN_TRY(check_ptrs(vec, 2 + n_outs, 16));
    GDN_TRY(check_ptrs(sc, n_sc, 4));
    Buf all[5 + GDN_LINEAR_MAX_OUTS];
    int n_all = 0;
    for (int i = 0; i < 2 + n_outs; ++i) all[n_all++] = vec[i];
    for (int i = 0; i < n_sc; ++i) all[n_all++] = sc[i];
    GDN_TRY(check_alias(vec + 2, n_outs, all, n_all));

    gdn::LinearF8Args l{};
    l.a = reinterpret_cast<const int8_t *>(a);
    l.a_scale = a_scale;
    l.w = reinterpret_cast<const int8_t *>(w);
    l.w_scale = w_scale;
    l.bias = bias;
    int32_t end = 0;
    for (int i = 0; i < gdn::kLinearMaxOuts; ++i) {
        // unused groups are empty and lie behind the last channel
        if (i < n_outs) end += outs[i].n;
        l.out[i] = i < n_outs ? outs[i].out : nullptr;
        l.end[i] = end;
    }
    l.M = M;
    l.N = static_cast<int32_t>(N);
    l.K = K;
    l.out_type = out_type;
    (void)hipGetLastError();
    return hip_status(gdn::launch_linear_f8(l, static_cast<hipStream_t>(stream)), "gdn_linear_f8 launch");
}

}  // extern "C"
