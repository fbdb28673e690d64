// gdn_chunk_api.cpp - the C ABI of the delta rule over packed sequences
// (gdn_chunk, gdn_chunk_backward, gdn_decode): argument validation and dispatch,
// as in gdn_api.cpp.

#include "gdn.h"

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "gdn_check.hpp"
#include "gdn_chunk.hpp"

namespace {

using gdn::Buf;
using gdn::check_alias;
using gdn::check_ptrs;
using gdn::check_type;
using gdn::clear_error;
using gdn::fail;
using gdn::hip_status;
using gdn::type_bytes;

// Each launch has at most 1024 work-items a head (and as many for up to seven key
// heads' value heads more), or 512 a chunk place and head, and the dispatch counts them
// in 32 bits.
constexpr int64_t kMaxHeads = 3735551, kMaxPlaces = 8388607;

int check_packed(const gdn_dims *d, int32_t B, int32_t tokens, int32_t type, const int32_t *offsets) {
    GDN_TRY(gdn::check_dims(d));
    GDN_TRY(check_type(type, "type"));
    if (d->n_v_heads > 65535)
        return fail(GDN_ERR_SHAPE, "n_v_heads must be <= 65535 (got %d)", d->n_v_heads);
    if (B < 1) return fail(GDN_ERR_SHAPE, "B must be >= 1 (got %d)", B);
    if (tokens < 1) return fail(GDN_ERR_SHAPE, "tokens must be >= 1 (got %d)", tokens);
    if (static_cast<int64_t>(B) * d->n_v_heads > kMaxHeads)
        return fail(GDN_ERR_SHAPE, "B * n_v_heads = %lld exceeds %lld",
                    (long long)B * d->n_v_heads, (long long)kMaxHeads);
    if (!offsets && tokens % B != 0)
        return fail(GDN_ERR_SHAPE, "tokens = %d is not a multiple of B = %d, and offsets is NULL", tokens, B);
    return GDN_OK;
}

int check_places(const gdn_dims *d, int32_t B, int32_t tokens) {
    if (tokens > INT32_MAX - 64) return fail(GDN_ERR_SHAPE, "tokens = %d is too large", tokens);
    if (gdn::chunk_places(B, tokens) * d->n_v_heads > kMaxPlaces)
        return fail(GDN_ERR_SHAPE, "(tokens / 64 + B) * n_v_heads exceeds %lld", (long long)kMaxPlaces);
    return GDN_OK;
}

int check_slots(const int32_t *slots, int32_t n_slots, int32_t B) {
    if (n_slots < 1 || (!slots && n_slots != B))
        return fail(GDN_ERR_SHAPE, "n_slots = %d, but %s", n_slots,
                    slots ? "it must be >= 1" : "without slots it must be B");
    return GDN_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (!ws) return fail(GDN_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (!gdn::aligned(ws, 16)) return fail(GDN_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (bytes < need) return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, need);
    return GDN_OK;
}

// Do dims, B, tokens and type describe a call of gdn_chunk or its backward pass?
bool sizes_ok(const gdn_dims *d, int32_t B, int32_t tokens, int32_t type) {
    const int32_t any = 0;           // offsets decide what tokens may be, not the workspace
    const bool ok = check_packed(d, B, tokens, type, &any) == GDN_OK && check_places(d, B, tokens) == GDN_OK;
    clear_error();
    return ok;
}

// Where the parts of the workspace begin, each a multiple of 16 bytes.
struct ChunkSpace {
    size_t kq, bytes;                // the blocks first
    ChunkSpace(const gdn_dims *d, int32_t B, int32_t tokens, int32_t type) {
        const size_t places = static_cast<size_t>(gdn::chunk_places(B, tokens));
        const size_t pv = places * d->n_v_heads, pk = places * d->n_k_heads;
        kq = pv * gdn::within_bytes(gdn::planes_out(type));
        bytes = kq + (type == GDN_BF16 ? 0 : pk * 2 * gdn::planes_in(type) * gdn::kPlaneBytes);
    }
};
struct BackSpace {
    size_t kq, within, back, gsum, states, dstates, delta, r, od, du, bytes;
    BackSpace(const gdn_dims *d, int32_t B, int32_t tokens, int32_t type) {
        const size_t places = static_cast<size_t>(gdn::chunk_places(B, tokens));
        const size_t pv = places * d->n_v_heads, pk = places * d->n_k_heads;
        const size_t f = sizeof(float), D = gdn::kHeadDim, C = gdn::kChunk;
        size_t at = 0;
        const auto take = [&](size_t n) { const size_t x = at; at += n; return x; };
        gsum = take(pv * C * sizeof(double));
        states = take(pv * D * D * f);
        dstates = take(pv * D * D * f);
        delta = take(pv * C * D * f);
        r = take(pv * C * D * f);
        within = take(pv * gdn::within_bytes(3));
        back = take(pv * gdn::within_bytes(3));
        od = take(pv * 8 * C * f);
        du = take(pv * 8 * f);
        kq = take(type == GDN_BF16 ? 0 : pk * 2 * gdn::planes_in(type) * gdn::kPlaneBytes);
        bytes = at;
    }
};

gdn::Packed packed(const gdn_dims *d, int32_t B, int32_t tokens, int32_t type, const int32_t *offsets,
                   const int32_t *slots, int32_t n_slots) {
    gdn::Packed s{};
    s.offsets = offsets;
    s.slots = slots;
    s.B = B;
    s.tokens = tokens;
    s.n_slots = n_slots;
    s.Hv = d->n_v_heads;
    s.Hk = d->n_k_heads;
    s.type = type;
    return s;
}

// What gdn_chunk and gdn_decode share: the tensors, checked.
int check_tensors(const gdn_dims *d, int32_t B, int32_t tokens, int32_t type, const void *q, const void *k,
                  const void *v, const float *beta, const float *gate, const int32_t *offsets,
                  const int32_t *slots, int32_t n_slots, const float *state, float *state_out, void *out,
                  bool state_needed, const Buf *ws) {
    const size_t z = type_bytes(type), n = static_cast<size_t>(tokens), D = gdn::kHeadDim;
    const size_t nk = n * d->n_k_heads * D * z, nv = n * d->n_v_heads * D * z;
    const size_t ns = static_cast<size_t>(n_slots) * d->n_v_heads * D * D * sizeof(float);
    const size_t nb = n * d->n_v_heads * sizeof(float);
    const Buf st = {"state", state, ns}, so = {"state_out", state_out, ns};
    Buf vec[6] = {{"q", q, nk}, {"k", k, nk}, {"v", v, nv}, {"out", out, nv}};
    int n_vec = 4;
    if (state_needed || state) vec[n_vec++] = st;
    if (state_needed || state_out) vec[n_vec++] = so;
    Buf sc[4] = {{"beta", beta, nb}, {"gate", gate, nb}};
    int n_sc = 2;
    if (offsets) sc[n_sc++] = {"offsets", offsets, (static_cast<size_t>(B) + 1) * sizeof(int32_t)};
    if (slots) sc[n_sc++] = {"slots", slots, static_cast<size_t>(B) * sizeof(int32_t)};
    GDN_TRY(check_ptrs(vec, n_vec, 16));
    GDN_TRY(check_ptrs(sc, n_sc, 4));
    Buf all[11] = {vec[0], vec[1], vec[2], vec[3]}, outs[3] = {vec[3]};
    int n_all = 4, n_out = 1;
    for (int i = 0; i < n_sc; ++i) all[n_all++] = sc[i];
    if (state && state != state_out) all[n_all++] = st;   // in place is one buffer under two names
    if (state_out) all[n_all++] = outs[n_out++] = so;
    if (ws) all[n_all++] = outs[n_out++] = *ws;
    return check_alias(outs, n_out, all, n_all);
}

}  // namespace

extern "C" {

size_t gdn_chunk_workspace_bytes(const gdn_dims *dims, int32_t B, int32_t tokens, int32_t type) {
    return sizes_ok(dims, B, tokens, type) ? ChunkSpace(dims, B, tokens, type).bytes : 0;
}

int gdn_chunk(const gdn_dims *dims, int32_t B, int32_t tokens, int32_t type, const void *q, const void *k,
              const void *v, const float *beta, const float *gate, const int32_t *offsets,
              const int32_t *slots, int32_t n_slots, const float *state, float *state_out, void *out,
              void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    GDN_TRY(check_packed(dims, B, tokens, type, offsets));
    GDN_TRY(check_places(dims, B, tokens));
    GDN_TRY(check_slots(slots, n_slots, B));
    const ChunkSpace w(dims, B, tokens, type);
    GDN_TRY(check_workspace(workspace, workspace_bytes, w.bytes));
    const Buf ws = {"workspace", workspace, w.bytes};
    GDN_TRY(check_tensors(dims, B, tokens, type, q, k, v, beta, gate, offsets, slots, n_slots, state, state_out,
                          out, false, &ws));
    gdn::ChunkArgs a{};
    a.s = packed(dims, B, tokens, type, offsets, slots, n_slots);
    a.q = q;
    a.k = k;
    a.v = v;
    a.beta = beta;
    a.gate = gate;
    a.state = state;
    a.state_out = state_out;
    a.out = out;
    char *p = static_cast<char *>(workspace);
    a.within = p;
    a.kq = type == GDN_BF16 ? nullptr : p + w.kq;
    (void)hipGetLastError();
    return hip_status(gdn::launch_chunk(a, static_cast<hipStream_t>(stream)), "gdn_chunk launch");
}

size_t gdn_chunk_backward_workspace_bytes(const gdn_dims *dims, int32_t B, int32_t tokens, int32_t type) {
    return sizes_ok(dims, B, tokens, type) ? BackSpace(dims, B, tokens, type).bytes : 0;
}

int gdn_chunk_backward(const gdn_dims *dims, int32_t B, int32_t tokens, int32_t type, const void *q,
                       const void *k, const void *v, const float *beta, const float *gate,
                       const int32_t *offsets, const float *state, const void *d_out,
                       const float *d_state_out, void *dq, void *dk, void *dv, float *dbeta, float *dgate,
                       float *d_state, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    GDN_TRY(check_packed(dims, B, tokens, type, offsets));
    GDN_TRY(check_places(dims, B, tokens));
    const BackSpace w(dims, B, tokens, type);
    GDN_TRY(check_workspace(workspace, workspace_bytes, w.bytes));
    const size_t z = type_bytes(type), n = static_cast<size_t>(tokens), D = gdn::kHeadDim;
    const size_t nk = n * dims->n_k_heads * D * z, nv = n * dims->n_v_heads * D * z;
    const size_t ns = static_cast<size_t>(B) * dims->n_v_heads * D * D * sizeof(float);
    const size_t nb = n * dims->n_v_heads * sizeof(float);
    Buf vec[10] = {{"dq", dq, nk}, {"dk", dk, nk}, {"dv", dv, nv}, {"q", q, nk}, {"k", k, nk}, {"v", v, nv},
                   {"d_out", d_out, nv}};
    int n_vec = 7;
    if (state) vec[n_vec++] = {"state", state, ns};
    // in place is one buffer under two names
    if (d_state_out && d_state_out != d_state) vec[n_vec++] = {"d_state_out", d_state_out, ns};
    if (d_state) vec[n_vec++] = {"d_state", d_state, ns};
    const Buf sc[] = {{"dbeta", dbeta, nb}, {"dgate", dgate, nb}, {"beta", beta, nb}, {"gate", gate, nb},
                      {"offsets", offsets, (static_cast<size_t>(B) + 1) * sizeof(int32_t)}};
    const int n_sc = offsets ? 5 : 4;
    GDN_TRY(check_ptrs(vec, n_vec, 16));
    GDN_TRY(check_ptrs(sc, n_sc, 4));
    Buf all[16], outs[7] = {vec[0], vec[1], vec[2], sc[0], sc[1]};
    int n_all = 0, n_out = 5;
    for (int i = 0; i < n_vec; ++i) all[n_all++] = vec[i];
    for (int i = 0; i < n_sc; ++i) all[n_all++] = sc[i];
    all[n_all++] = outs[n_out++] = {"workspace", workspace, w.bytes};
    if (d_state) outs[n_out++] = vec[n_vec - 1];
    GDN_TRY(check_alias(outs, n_out, all, n_all));

    char *p = static_cast<char *>(workspace);
    const auto at = [&](size_t x) { return reinterpret_cast<float *>(p + x); };
    gdn::BackArgs a{};
    a.f.s = packed(dims, B, tokens, type, offsets, nullptr, B);
    a.f.q = q;
    a.f.k = k;
    a.f.v = v;
    a.f.beta = beta;
    a.f.gate = gate;
    a.f.state = state;
    a.f.d_out = d_out;
    a.f.within = p + w.within;
    a.f.kq = type == GDN_BF16 ? nullptr : p + w.kq;
    a.f.states = at(w.states);
    a.f.delta = at(w.delta);
    a.f.od = at(w.od);
    a.d_state_out = d_state_out;
    a.d_state = d_state;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dbeta = dbeta;
    a.dgate = dgate;
    a.back = p + w.back;
    a.gsum = reinterpret_cast<double *>(p + w.gsum);
    a.dstates = at(w.dstates);
    a.r = at(w.r);
    a.du = at(w.du);
    (void)hipGetLastError();
    return hip_status(gdn::launch_chunk_backward(a, static_cast<hipStream_t>(stream)),
                      "gdn_chunk_backward launch");
}

int gdn_decode(const gdn_dims *dims, int32_t B, int32_t tokens, int32_t type, const void *q, const void *k,
               const void *v, const float *beta, const float *gate, const int32_t *offsets,
               const int32_t *slots, int32_t n_slots, const float *state, float *state_out, void *out,
               void *stream) {
    clear_error();
    GDN_TRY(check_packed(dims, B, tokens, type, offsets));
    GDN_TRY(check_slots(slots, n_slots, B));
    GDN_TRY(check_tensors(dims, B, tokens, type, q, k, v, beta, gate, offsets, slots, n_slots, state, state_out,
                          out, true, nullptr));
    gdn::DecodeArgs a{};
    a.s = packed(dims, B, tokens, type, offsets, slots, n_slots);
    a.q = q;
    a.k = k;
    a.v = v;
    a.beta = beta;
    a.gate = gate;
    a.state = state;
    a.state_out = state_out;
    a.out = out;
    (void)hipGetLastError();
    return hip_status(gdn::launch_decode(a, static_cast<hipStream_t>(stream)), "gdn_decode launch");
}

}  // extern "C"
