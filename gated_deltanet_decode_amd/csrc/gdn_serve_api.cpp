// gdn_serve_api.cpp - the C ABI of the operators around the recurrent branch
// (gdn_add_rmsnorm_q8, gdn_quantize_q8, gdn_linear_q8, gdn_verify,
// gdn_pair_commit): argument validation and dispatch, as in gdn_api.cpp.

#include "gdn.h"

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "gdn_check.hpp"
#include "gdn_launch.hpp"
#include "gdn_serve.hpp"

namespace {

using gdn::Buf;
using gdn::check_alias;
using gdn::check_ptrs;
using gdn::clear_error;
using gdn::fail;
using gdn::hip_status;

// Bytes of an element type, 0 for an unknown code.
size_t type_bytes(int32_t type) {
    switch (type) {
    case GDN_F32: return 4;
    case GDN_BF16:
    case GDN_F16: return 2;
    default: return 0;
    }
}

int check_type(int32_t type, const char *what) {
    if (type_bytes(type) == 0)
        return fail(GDN_ERR_SHAPE, "unknown %s %d (GDN_F32, GDN_BF16 or GDN_F16)", what, type);
    return GDN_OK;
}

int check_rows(int32_t rows, int32_t n) {
    const int64_t most = UINT32_MAX / gdn::kQuantMaxThreads;   // one workgroup per row
    if (rows < 1 || rows > most)
        return fail(GDN_ERR_SHAPE, "rows must be in [1, %lld] (got %d)", (long long)most, rows);
    // the kernels' element index stays clear of 2^31
    if (n < 1 || n > (1 << 30) - 1)
        return fail(GDN_ERR_SHAPE, "n must be in [1, 1073741823] (got %d)", n);
    return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_add_rmsnorm_q8(int32_t rows, int32_t n, int32_t x_type, const void *x,
                       int32_t residual_type, const void *residual, void *residual_out,
                       const float *norm_w, float eps, int8_t *q, float *scale, void *stream) {
    clear_error();
    GDN_TRY(check_rows(rows, n));
    GDN_TRY(check_type(x_type, "x_type"));
    const bool has = residual_type != GDN_NONE;
    if (has) GDN_TRY(check_type(residual_type, "residual_type"));
    if (!has && (residual || residual_out))
        return fail(GDN_ERR_SHAPE, "residual_type is GDN_NONE, but a residual is given");
    if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(GDN_ERR_SHAPE, "eps must be finite and >= 0");
    const size_t e = static_cast<size_t>(rows) * n;
    const size_t rb = has ? e * type_bytes(residual_type) : 0;
    Buf vec[4] = {{"x", x, e * type_bytes(x_type)}, {"q", q, e}};
    int n_vec = 2;
    if (has) {
        vec[n_vec++] = {"residual", residual, rb};
        vec[n_vec++] = {"residual_out", residual_out, rb};
    }
    const Buf sc[] = {{"norm_w", norm_w, static_cast<size_t>(n) * sizeof(float)},
                      {"scale", scale, static_cast<size_t>(rows) * sizeof(float)}};
    GDN_TRY(check_ptrs(vec, n_vec, 16));
    GDN_TRY(check_ptrs(sc, 2, 4));
    Buf all[6] = {vec[0], vec[1], sc[0], sc[1]};
    Buf outs[3] = {vec[1], sc[1]};
    int n_all = 4, n_out = 2;
    if (has) {
        all[n_all++] = vec[3];
        outs[n_out++] = vec[3];
        // in place is one buffer under two names
        if (residual != residual_out) all[n_all++] = vec[2];
    }
    GDN_TRY(check_alias(outs, n_out, all, n_all));

    gdn::QuantArgs a{};
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.norm_w = norm_w;
    a.q = q;
    a.scale = scale;
    a.eps = eps;
    a.rows = rows;
    a.n = n;
    a.x_type = x_type;
    a.residual_type = residual_type;
    (void)hipGetLastError();
    return hip_status(gdn::launch_quant(a, static_cast<hipStream_t>(stream)),
                      "gdn_add_rmsnorm_q8 launch");
}

int gdn_quantize_q8(int32_t rows, int32_t n, int32_t x_type, const void *x, int8_t *q,
                    float *scale, void *stream) {
    clear_error();
    GDN_TRY(check_rows(rows, n));
    GDN_TRY(check_type(x_type, "x_type"));
    const size_t e = static_cast<size_t>(rows) * n;
    const Buf vec[] = {{"x", x, e * type_bytes(x_type)}, {"q", q, e}};
    const Buf sc[] = {{"scale", scale, static_cast<size_t>(rows) * sizeof(float)}};
    GDN_TRY(check_ptrs(vec, 2, 16));
    GDN_TRY(check_ptrs(sc, 1, 4));
    const Buf all[] = {vec[0], vec[1], sc[0]};
    const Buf outs[] = {vec[1], sc[0]};
    GDN_TRY(check_alias(outs, 2, all, 3));

    gdn::QuantArgs a{};
    a.x = x;
    a.q = q;
    a.scale = scale;
    a.rows = rows;
    a.n = n;
    a.x_type = x_type;
    a.residual_type = GDN_NONE;
    (void)hipGetLastError();
    return hip_status(gdn::launch_quant(a, static_cast<hipStream_t>(stream)),
                      "gdn_quantize_q8 launch");
}

int gdn_linear_q8(int32_t M, int32_t K, const int8_t *a, const float *a_scale, const int8_t *w,
                  const float *w_scale, const float *bias, int32_t out_type,
                  const gdn_linear_out *outs, int32_t n_outs, void *stream) {
    static_assert(GDN_LINEAR_MAX_OUTS == gdn::kLinearMaxOuts, "");
    clear_error();
    GDN_TRY(check_type(out_type, "out_type"));
    if (M < 1) return fail(GDN_ERR_SHAPE, "M must be >= 1 (got %d)", M);
    // |a w| <= 2^14, so the sum of 131071 products stays below 2^31
    if (K < 1 || K > 131071)
        return fail(GDN_ERR_SHAPE, "K must be in [1, 131071] (got %d)", K);
    if (n_outs < 1 || n_outs > GDN_LINEAR_MAX_OUTS)
        return fail(GDN_ERR_SHAPE, "n_outs must be in [1, %d] (got %d)", GDN_LINEAR_MAX_OUTS,
                    n_outs);
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
    Buf vec[2 + GDN_LINEAR_MAX_OUTS] = {{"a", a, static_cast<size_t>(M) * K},
                                        {"w", w, static_cast<size_t>(N) * K}};
    for (int i = 0; i < n_outs; ++i)
        vec[2 + i] = {kOut[i], outs[i].out,
                      static_cast<size_t>(M) * outs[i].n * type_bytes(out_type)};
    const Buf sc[] = {{"a_scale", a_scale, static_cast<size_t>(M) * sizeof(float)},
                      {"w_scale", w_scale, static_cast<size_t>(N) * sizeof(float)},
                      {"bias", bias, static_cast<size_t>(N) * sizeof(float)}};
    const int n_sc = bias ? 3 : 2;
    GDN_TRY(check_ptrs(vec, 2 + n_outs, 16));
    GDN_TRY(check_ptrs(sc, n_sc, 4));
    Buf all[5 + GDN_LINEAR_MAX_OUTS];
    int n_all = 0;
    for (int i = 0; i < 2 + n_outs; ++i) all[n_all++] = vec[i];
    for (int i = 0; i < n_sc; ++i) all[n_all++] = sc[i];
    GDN_TRY(check_alias(vec + 2, n_outs, all, n_all));

    gdn::LinearArgs l{};
    l.a = a;
    l.a_scale = a_scale;
    l.w = w;
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
    return hip_status(gdn::launch_linear(l, static_cast<hipStream_t>(stream)),
                      "gdn_linear_q8 launch");
}

size_t gdn_verify_workspace_bytes(int32_t B, int32_t V) {
    if (B < 1 || B > 65535 || V < 1) return 0;
    return static_cast<size_t>(B) * gdn::kVerifyBytes;
}

int gdn_verify(int32_t B, int32_t K, int32_t V, int32_t prob_type, const void *target,
               const void *draft, const int32_t *draft_tokens, const int32_t *n_draft,
               const float *u_accept, const float *u_sample, int32_t *accepted, int32_t *tokens,
               void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    GDN_TRY(check_type(prob_type, "prob_type"));
    if (B < 1 || B > 65535) return fail(GDN_ERR_SHAPE, "B must be in [1, 65535] (got %d)", B);
    if (K < 1 || K > 1024) return fail(GDN_ERR_SHAPE, "K must be in [1, 1024] (got %d)", K);
    if (V < 1) return fail(GDN_ERR_SHAPE, "V must be >= 1 (got %d)", V);
    const size_t pb = type_bytes(prob_type);
    const size_t BK = static_cast<size_t>(B) * K;
    const size_t i4 = sizeof(int32_t), f = sizeof(float);
    Buf vec[2] = {{"target", target, (BK + B) * V * pb}, {"draft", draft, BK * V * pb}};
    const int n_vec = draft ? 2 : 1;
    Buf sc[6] = {{"draft_tokens", draft_tokens, BK * i4},
                 {"u_accept", u_accept, BK * f},
                 {"u_sample", u_sample, B * f},
                 {"accepted", accepted, B * i4},
                 {"tokens", tokens, (BK + B) * i4},
                 {"n_draft", n_draft, B * i4}};
    const int n_sc = n_draft ? 6 : 5;
    GDN_TRY(check_ptrs(vec, n_vec, 16));
    GDN_TRY(check_ptrs(sc, n_sc, 4));
    const size_t need = gdn_verify_workspace_bytes(B, V);
    if (!workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (!gdn::aligned(workspace, 16))
        return fail(GDN_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes,
                    need);
    Buf all[9];
    int n_all = 0;
    for (int i = 0; i < n_vec; ++i) all[n_all++] = vec[i];
    for (int i = 0; i < n_sc; ++i) all[n_all++] = sc[i];
    all[n_all++] = {"workspace", workspace, need};
    const Buf outs[] = {sc[3], sc[4], all[n_all - 1]};
    GDN_TRY(check_alias(outs, 3, all, n_all));

    gdn::VerifyArgs a{};
    a.target = target;
    a.draft = draft;
    a.draft_tokens = draft_tokens;
    a.n_draft = n_draft;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.accepted = accepted;
    a.tokens = tokens;
    a.partial = static_cast<double *>(workspace);
    a.rows = reinterpret_cast<int32_t *>(a.partial + static_cast<size_t>(B) * gdn::kVerifyUnits);
    a.B = B;
    a.K = K;
    a.V = V;
    a.prob_type = prob_type;
    (void)hipGetLastError();
    return hip_status(gdn::launch_verify(a, static_cast<hipStream_t>(stream)),
                      "gdn_verify launch");
}

int gdn_pair_commit(const gdn_dims *dims, int32_t layers, int32_t B, const int32_t *accepted,
                    float *state, const float *state_next, int32_t conv_floats, float *conv_state,
                    const float *conv_state_next, void *stream) {
    clear_error();
    GDN_TRY(gdn::check_dims(dims));
    if (layers < 1) return fail(GDN_ERR_SHAPE, "layers must be >= 1 (got %d)", layers);
    GDN_TRY(gdn::check_batch(dims, B, "B"));
    const int64_t LB = static_cast<int64_t>(layers) * B;
    const bool ring = conv_state || conv_state_next || conv_floats != 0;
    if (ring && (conv_floats < 4 || conv_floats % 4 != 0))
        return fail(GDN_ERR_SHAPE, "conv_floats must be a positive multiple of 4 (got %d)",
                    conv_floats);
    const size_t f = sizeof(float);
    const int64_t sf = static_cast<int64_t>(dims->n_v_heads) * dims->d_v * dims->d_k;
    // one launch for all of it: per_seq is at least 2 and at most 2^28 + 2^18
    const int64_t most = UINT32_MAX / gdn::kCommitThreads;
    const int64_t per_seq = gdn::commit_blocks(sf / 4) + gdn::commit_blocks(conv_floats / 4);
    if (LB > most || per_seq > most || LB * per_seq > most)
        return fail(GDN_ERR_SHAPE, "layers * B * (state + ring) is too large");
    const size_t ns = static_cast<size_t>(LB) * sf * f;
    const size_t nc = static_cast<size_t>(LB) * conv_floats * f;
    const Buf vec[] = {{"state", state, ns},
                       {"state_next", state_next, ns},
                       {"conv_state", conv_state, nc},
                       {"conv_state_next", conv_state_next, nc}};
    const Buf sc[] = {{"accepted", accepted, static_cast<size_t>(B) * sizeof(int32_t)}};
    const int n_vec = ring ? 4 : 2;
    GDN_TRY(check_ptrs(sc, 1, 4));
    GDN_TRY(check_ptrs(vec, n_vec, 16));
    Buf all[5] = {sc[0], vec[0], vec[1], vec[2], vec[3]};
    Buf outs[2] = {vec[0], vec[2]};
    GDN_TRY(check_alias(outs, ring ? 2 : 1, all, 1 + n_vec));

    gdn::CommitArgs a{};
    a.accepted = accepted;
    a.state = state;
    a.state_next = state_next;
    a.ring = conv_state;
    a.ring_next = conv_state_next;
    a.layers = layers;
    a.B = B;
    a.state_f4 = sf / 4;                  // past 2^31 from 524288 heads on
    a.ring_f4 = conv_floats / 4;
    (void)hipGetLastError();
    return hip_status(gdn::launch_commit(a, static_cast<hipStream_t>(stream)),
                      "gdn_pair_commit launch");
}

}  // extern "C"
