// gdn_walk.hpp - k_walk, the delta rule along packed sequences in chunks of 64
// tokens, shared by the forward and the backward pass.  Included by kernel sources
// only.
//
// Mathematics.  Within a chunk that a state M (dv x dk) enters, with g the
// running sum of the gates (k_prep forms T and P):
//   X = V - diag(e^g) K M^T,   Delta = T diag(beta) X,
//   O = diag(e^g) Q M^T / sqrt(128) + P Delta,
//   M' = e^{g_64} M + (diag(e^{g_64 - g}) Delta)^T K:
// the recurrence's own corrections Delta, all tokens of the chunk at once.
//
// k_walk goes along a sequence's chunks with the state in registers.  Rows of M
// never exchange data: a wave has 16 of them, as the accumulators of 8 matrix
// tiles (dk x dv), and everything of a chunk that belongs to these rows (K M^T,
// X, Delta, O) stays in its registers as well, since a result's lane holds what
// an operand's lane needs (gdn_mma.hpp).  What all rows share (K, Q, T, P) comes
// through LDS once a workgroup.  The state and whatever feeds it are kept to
// binary32: three planes of M and Delta against the planes of K.
#pragma once

#include "gdn_prep.hpp"

namespace gdn {
namespace {

typedef __attribute__((address_space(3))) void *lds_t;

// 1 KiB straight into LDS: lane l's 16 bytes at off land at lds + 16 l.
__device__ __forceinline__ void fetch16(char *lds, const void *base, uint32_t bytes, int off, int more) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000), (lds_t)lds, 16, off,
        more, 0, 0);
}

// The k and q rows of a chunk (NP planes each, K's then Q's) on their way to LDS.
template <typename ET, int NP, int W>
__device__ __forceinline__ void fetch_rows(const ChunkArgs &a, char *K, char *Q, int64_t place, int token, int rows,
                                           int kh, int wave, int lane) {
    const int Hk = a.s.Hk;
    if constexpr (NP == 1) {                              // rows of the tensors, slots swizzled
        const int64_t at = (static_cast<int64_t>(token) * Hk + kh) * (kHeadDim * 2);
        const uint32_t bytes = ((rows - 1) * Hk + 1) * kHeadDim * 2;
#pragma unroll
        for (int i = 0; i < 16 / W; ++i) {
            const int rr = (i * W + wave) * 4 + (lane >> 4);
            const int off = rr * Hk * (kHeadDim * 2) + (((lane & 15) ^ (rr & 15)) << 4);
            fetch16(K + (i * W + wave) * 1024, static_cast<const char *>(a.k) + at, bytes, off, 0);
            fetch16(Q + (i * W + wave) * 1024, static_cast<const char *>(a.q) + at, bytes, off, 0);
        }
    } else {
        const char *kq = a.kq + (place * Hk + kh) * (2 * NP * kPlaneBytes);
        for (int i = wave; i < 2 * NP * 16; i += W)
            fetch16(K + i * 1024, kq, 2 * NP * kPlaneBytes, lane * 16, i * 1024);
    }
}

// Zeros for the rows that the last chunk of a sequence lacks (the planes in the
// workspace have them).  The whole workgroup calls it after its own fetches landed.
template <int NP, int W>
__device__ __forceinline__ void clear_rows(char *K, char *Q, int rows) {
    if (NP > 1 || rows == kChunk) return;
    meet();
    for (int i = threadIdx.x; i < (kChunk - rows) * 16; i += 64 * W) {
        *reinterpret_cast<u4 *>(K + rows * 256 + i * 16) = u4{0, 0, 0, 0};
        *reinterpret_cast<u4 *>(Q + rows * 256 + i * 16) = u4{0, 0, 0, 0};
    }
    wait_all<0>();
}

// Columns of a plane as operands: the tokens 32 half + 4 g + e and 16 more are k,
// and row (column) 4 c + i of tile t is dk 32 (t / 2) + 8 c + 4 (t % 2) + i, so that
// tiles 2 jj and 2 jj + 1 hold eight consecutive dk a lane.
__device__ __forceinline__ u4 columns_of(const char *plane, int half, int t, int r, int g) {
    const int tok = 32 * half + 4 * g + (r >> 2), chunk = 4 * (t / 2) + (r & 3);
    const u2 x = read_columns(plane + plane_at(tok, chunk) + 8 * (t % 2));
    const u2 y = read_columns(plane + plane_at(tok + 16, chunk) + 8 * (t % 2));
    return u4{x.x, x.y, y.x, y.y};
}

template <int NP, int NO>
struct Stage {
    static constexpr int kK = 0, kQ = NP * kPlaneBytes, kT = 2 * NP * kPlaneBytes, kP = kT + kTBytes,
                         kVec = kP + kPBlocks * 1024 * NO, kBytes = kVec + 1024;
};

// W waves, 16 rows of the state each.  NP planes of k and q, NO of what only the
// outputs see; S buffers of a chunk's operands.  For the backward pass (kBack) the
// states that enter each chunk and the corrections are kept, and the outputs
// only meet their gradient: od is the sum over the wave's rows of out * d_out.
template <typename ET, int NP, int NO, int W, int S, bool kBack>
__global__ __launch_bounds__(64 * W) void k_walk(ChunkArgs a, int parts) {
    typedef typename ET::bits bits;
    typedef Stage<NP, NO> L;
    __shared__ alignas(1024) char buf0[L::kBytes], buf1[S > 1 ? L::kBytes : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int Hv = a.s.Hv, Hk = a.s.Hk;
    // Each XCD (ids modulo 8) takes a run of neighbours: the parts of a head, then the
    // heads that share a key head.
    const int id = (blockIdx.x & 7) * static_cast<int>(gridDim.x >> 3) + (blockIdx.x >> 3);
    const int part = id % parts, hh = id / parts;
    const int b = hh / Hv;
    if (b >= a.s.B) return;
    const int kh = (hh - b * Hv) / (Hv / Hk), h = kh + (hh - b * Hv) % (Hv / Hk) * Hk;
    const int slot = slot_of(a.s, b);
    if (slot < 0) return;
    const Span sp = span_of(a.s, b);
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const int dv = (part * W + wave) * 16 + r;           // this lane's row of M

    // M[dv][32 jj + 8 g + 0..7] are the four of tile 2 jj and the four of 2 jj + 1
    f4 M[8];
    const int64_t row = ((static_cast<int64_t>(slot) * Hv + h) * kHeadDim + dv) * kHeadDim + 8 * g;
#pragma unroll
    for (int t = 0; t < 8; ++t)
        M[t] = a.state ? *reinterpret_cast<const f4 *>(a.state + row + 32 * (t / 2) + 4 * (t % 2)) : f4{0, 0, 0, 0};

    const int place0 = place_of(sp.first, b);
    auto fetch = [&](char *to, int c) {
        const int64_t place = place0 + c, ph = place * Hv + h;
        const int rows = min(kChunk, sp.len - c * kChunk);
        fetch_rows<ET, NP, W>(a, to + L::kK, to + L::kQ, place, sp.first + c * kChunk, rows, kh, wave, lane);
        const float *T = a.T + ph * (kTBlocks * 256);
        const char *P = a.P + ph * (kPBlocks * 1024 * NO);
        for (int i = wave; i < kTBlocks + kPBlocks * NO + 1; i += W) {
            if (i < kTBlocks)
                fetch16(to + L::kT + i * 1024, T, kTBytes, lane * 16, i * 1024);
            else if (i < kTBlocks + kPBlocks * NO)
                fetch16(to + L::kP + (i - kTBlocks) * 1024, P, kPBlocks * 1024 * NO, lane * 16, (i - kTBlocks) * 1024);
            else
                fetch16(to + L::kVec, a.vec + ph * kVecFloats, kVecFloats * 4, lane * 16, 0);
        }
    };
    const bits *vp = static_cast<const bits *>(a.v) + (static_cast<int64_t>(sp.first) * Hv + h) * kHeadDim + dv;
    bits *op = static_cast<bits *>(a.out) + (static_cast<int64_t>(sp.first) * Hv + h) * kHeadDim + dv - r + 4 * g;
    const bits *dop = static_cast<const bits *>(a.d_out) + (static_cast<int64_t>(sp.first) * Hv + h) * kHeadDim + dv - r + 4 * g;
    const int64_t vstride = static_cast<int64_t>(Hv) * kHeadDim;
    bits vn[16];                                          // v of the chunk to come
    auto load_v = [&](int c) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = c * kChunk + 16 * (i / 4) + 4 * g + i % 4;
            vn[i] = t < sp.len ? vp[t * vstride] : bits(0);
        }
    };

    auto chunk = [&](char *cur, char *nxt, int c) {
        const int64_t ph = (static_cast<int64_t>(place0) + c) * Hv + h;
        if constexpr (kBack) {
            float *to = a.states + ph * (kHeadDim * kHeadDim) + dv * kHeadDim + 8 * g;
#pragma unroll
            for (int t = 0; t < 8; ++t) *reinterpret_cast<f4 *>(to + 32 * (t / 2) + 4 * (t % 2)) = M[t];
        }
        if (S == 1) {
            meet();                                       // the buffer is read
            fetch(cur, c);
        }
        wait_all<0>();
        const int rows = min(kChunk, sp.len - c * kChunk);
        clear_rows<NP, W>(cur + L::kK, cur + L::kQ, rows);
        meet();                                           // cur has landed, nxt is read
        if (S > 1 && c + 1 < chunks) fetch(nxt, c + 1);
        f4 Y[4] = {}, Z[4] = {};
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            u4 m3[3], mo[NO];
            planes_of<3>(M[2 * jj], M[2 * jj + 1], m3);
#pragma unroll
            for (int p = 0; p < NO; ++p) mo[p] = m3[p];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                u4 kf[NP], qf[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const int at = p * kPlaneBytes + plane_at(jt * 16 + r, 4 * jj + g);
                    kf[p] = *reinterpret_cast<const u4 *>(cur + L::kK + at);
                    qf[p] = *reinterpret_cast<const u4 *>(cur + L::kQ + at);
                }
                Y[jt] = mma_planes<2>(kf, m3, Y[jt]);                 // token 4 g + e, row dv
                Z[jt] = mma_planes<NO - 1>(mo, qf, Z[jt]);            // dv 4 g + e, token r
            }
        }
        const float *vec = reinterpret_cast<const float *>(cur + L::kVec);
        f4 X[4], E[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            const f4 rise = *reinterpret_cast<const f4 *>(vec + 16 * jt + 4 * g);
            const f4 beta = *reinterpret_cast<const f4 *>(vec + 2 * kChunk + 16 * jt + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                X[jt][e] = beta[e] * fmaf(-rise[e], Y[jt][e], ET::get(vn[4 * jt + e]));
        }
        if (c + 1 < chunks) load_v(c + 1);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            f4 d = {0, 0, 0, 0};
#pragma unroll
            for (int jt = 0; jt <= it; ++jt)
                d = mma32(*reinterpret_cast<const f4 *>(cur + L::kT + block_of(it, jt) * 1024 + lane * 16), X[jt], d);
            E[it] = d;                                    // Delta: token 4 g + e, row dv
            if constexpr (kBack) {
                float *to = a.delta + (ph * kChunk + 16 * it + 4 * g) * kHeadDim + dv;
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e * kHeadDim] = d[e];
            }
        }
        // outputs
        u4 dp[2][NO];
        planes_of<NO>(E[0], E[1], dp[0]);
        planes_of<NO>(E[2], E[3], dp[1]);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            f4 o = Z[it] * (kReadScale * vec[16 * it + r]);
#pragma unroll
            for (int half = 0; half <= it / 2; ++half) {
                u4 pf[NO];
#pragma unroll
                for (int m = 0; m < NO; ++m)
                    pf[m] = *reinterpret_cast<const u4 *>(cur + L::kP + (m * kPBlocks + pblock_of(it, half)) * 1024 +
                                                          lane * 16);
                o = mma_planes<NO - 1>(dp[half], pf, o);
            }
            const int t = c * kChunk + 16 * it + r;
            if constexpr (kBack) {
                float s = 0.0f;
                if (t < sp.len) {
                    const auto w = Pack<bits, 4>::load(dop + t * vstride);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s = fmaf(o[e], ET::get(w[e]), s);
                }
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (g == 0) a.od[(ph * 8 + part * W + wave) * kChunk + 16 * it + r] = s;
            } else if (t < sp.len) {
                typename Pack<bits, 4>::vec w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = ET::put(o[e]);
                Pack<bits, 4>::store(op + t * vstride, w);
            }
        }
        // the state
        const float all = vec[kChunk - 1];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) E[jt] *= *reinterpret_cast<const f4 *>(vec + kChunk + 16 * jt + 4 * g);
#pragma unroll
        for (int t = 0; t < 8; ++t) M[t] *= all;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u4 ep[3];
            planes_of<3>(E[2 * half], E[2 * half + 1], ep);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                u4 kt[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) kt[p] = columns_of(cur + L::kK + p * kPlaneBytes, half, t, r, g);
                M[t] = mma_planes<2>(kt, ep, M[t]);
            }
        }
    };
    if (chunks > 0) {
        load_v(0);
        if (S > 1) fetch(buf0, 0);
        int c = 0;
        if constexpr (S > 1) {
            for (; c + 2 <= chunks; c += 2) {
                chunk(buf0, buf1, c);
                chunk(buf1, buf0, c + 1);
            }
            if (c < chunks) chunk(buf0, buf1, c);
        } else {
            for (; c < chunks; ++c) chunk(buf0, buf0, c);
        }
    }
    if (a.state_out) {
#pragma unroll
        for (int t = 0; t < 8; ++t) *reinterpret_cast<f4 *>(a.state_out + row + 32 * (t / 2) + 4 * (t % 2)) = M[t];
    }
}

template <typename ET, int NP, int NO, int S, bool kBack>
hipError_t launch_walk(const ChunkArgs &a, hipStream_t s) {
    constexpr int W = 8;
    const int parts = 8 / W;
    const int64_t wgs = static_cast<int64_t>(a.s.B) * a.s.Hv * parts;
    k_walk<ET, NP, NO, W, S, kBack><<<dim3(static_cast<unsigned>((wgs + 7) / 8 * 8)), dim3(64 * W), 0, s>>>(a, parts);
    return hipGetLastError();
}

}  // namespace
}  // namespace gdn
