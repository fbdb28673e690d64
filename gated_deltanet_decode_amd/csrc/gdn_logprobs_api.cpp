// gdn_logprobs_api.cpp - the C ABI of gdn_logprobs: argument validation and
// dispatch, as in gdn_api.cpp.

#include "gdn.h"

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "gdn_check.hpp"
#include "gdn_logprobs.hpp"

namespace {

using gdn::Buf;
using gdn::check_type;
using gdn::clear_error;
using gdn::fail;

int check_sizes(int32_t rows, int32_t V, int32_t top) {
    // a workgroup of 256 per unit of a row, and an entry's index below 2^31
    if (rows < 1 || rows > 4194303)
        return fail(GDN_ERR_SHAPE, "rows must be in [1, 4194303] (got %d)", rows);
    if (V < 1 || V > (1 << 30)) return fail(GDN_ERR_SHAPE, "V must be in [1, 1073741824] (got %d)", V);
    if (top < 0 || top > GDN_LOGPROBS_MAX_TOP || top > V)
        return fail(GDN_ERR_SHAPE, "top must be in [0, %d] and at most V (got %d)", GDN_LOGPROBS_MAX_TOP, top);
    return GDN_OK;
}

size_t space(int32_t rows, int32_t V, int32_t top) {
    const int64_t units = gdn::logprobs_units(rows, V);
    return units == 1 ? 0 : static_cast<size_t>(rows) * units * (3 * sizeof(double) + top * sizeof(uint64_t));
}

}  // namespace

extern "C" {

size_t gdn_logprobs_workspace_bytes(int32_t rows, int32_t V, int32_t top) {
    const bool ok = check_sizes(rows, V, top) == GDN_OK;
    clear_error();
    return ok ? space(rows, V, top) : 0;
}

int gdn_logprobs(int32_t rows, int32_t V, int64_t ld, int32_t logit_type, const void *logits,
                 const int32_t *tokens, float *logprob, float *entropy, int32_t top, int32_t *top_ids,
                 float *top_logprobs, void *workspace, size_t workspace_bytes, void *stream) {
    static_assert(GDN_LOGPROBS_MAX_TOP == gdn::kLogprobsMaxTop, "");
    clear_error();
    GDN_TRY(check_type(logit_type, "logit_type"));
    GDN_TRY(check_sizes(rows, V, top));
    if (ld < V || ld > (INT64_C(1) << 40))
        return fail(GDN_ERR_SHAPE, "ld must be in [V, 2^40] (got %lld)", (long long)ld);
    if (!tokens != !logprob)
        return fail(GDN_ERR_NULL, "%s is NULL, but not %s", tokens ? "logprob" : "tokens", tokens ? "tokens" : "logprob");
    if (!tokens && !entropy && top == 0)
        return fail(GDN_ERR_NULL, "logprob is NULL, and nothing else is wanted");
    const size_t n = static_cast<size_t>(rows), w = sizeof(int32_t), need = space(rows, V, top);
    const size_t z = gdn::type_bytes(logit_type);
    // rows of a strided matrix: up to the last entry of the last one
    const Buf vec[] = {{"logits", logits, ((n - 1) * static_cast<size_t>(ld) + V) * z}};
    Buf all[7] = {vec[0]}, outs[5], sc[6];
    int n_sc = 0, n_out = 0, n_all = 1;
    if (tokens) {
        sc[n_sc++] = {"tokens", tokens, n * w};
        sc[n_sc++] = outs[n_out++] = {"logprob", logprob, n * w};
    }
    if (entropy) sc[n_sc++] = outs[n_out++] = {"entropy", entropy, n * w};
    if (top > 0) {
        sc[n_sc++] = outs[n_out++] = {"top_ids", top_ids, n * top * w};
        sc[n_sc++] = outs[n_out++] = {"top_logprobs", top_logprobs, n * top * w};
    }
    GDN_TRY(gdn::check_ptrs(vec, 1, z));
    GDN_TRY(gdn::check_ptrs(sc, n_sc, 4));
    for (int i = 0; i < n_sc; ++i) all[n_all++] = sc[i];
    if (need > 0) {
        if (!workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
        if (!gdn::aligned(workspace, 16)) return fail(GDN_ERR_ALIGN, "workspace is not 16-byte aligned");
        if (workspace_bytes < need)
            return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
        all[n_all++] = outs[n_out++] = {"workspace", workspace, need};
    }
    GDN_TRY(gdn::check_alias(outs, n_out, all, n_all));

    gdn::LogprobsArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.sums = static_cast<double *>(workspace);
    a.keys = reinterpret_cast<uint64_t *>(a.sums + n * gdn::logprobs_units(rows, V) * 3);
    a.rows = rows;
    a.V = V;
    a.top = top;
    a.type = logit_type;
    (void)hipGetLastError();
    return gdn::hip_status(gdn::launch_logprobs(a, static_cast<hipStream_t>(stream)), "gdn_logprobs launch");
}

}  // extern "C"
