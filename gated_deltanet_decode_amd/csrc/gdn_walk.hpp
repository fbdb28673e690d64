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
//
// The chain of products a chunk bounds it, K M^T to X to Delta to M', each waiting for
// the one before: 8 x 4096 tokens bf16, 32 value heads, 470 us with the matrix units 49 %
// and the vector units 50 % busy, which overlap little (clock 1.55 GHz); 1 x 4096 about 230 us, 3.6 us a chunk.  Waiting for every
// fetch and store at a chunk's end, and without the swizzle of columns: 640 us.
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
            const int off = rr * Hk * (kHeadDim * 2) + (((lane & 15) ^ turn(rr)) << 4);
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

// A chunk's operands in LDS: K and Q (NP planes each), and a block of k_prep.
template <int NP, int NO>
struct Stage {
    static constexpr int kK = 0, kQ = NP * kPlaneBytes, kT = 2 * NP * kPlaneBytes, kP = kT + kTBytes,
                         kVec = kP + kPBlocks * 1024 * NO, kBytes = kT + (within_bytes(NO) + 8191) / 8192 * 8192;
};

// The planes of operand `block` of T or P.
template <int N>
__device__ __forceinline__ void operand_at(const char *at, int block, int lane, u4 (&p)[N]) {
#pragma unroll
    for (int m = 0; m < N; ++m) p[m] = *reinterpret_cast<const u4 *>(at + (m * kPBlocks + block) * 1024 + lane * 16);
}

// `bytes` of a block on its way to LDS; each wave takes the same number of kilobytes,
// and those past the end come as they may.
template <int kBytes, int W>
__device__ __forceinline__ void fetch_block(const char *block, char *to, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < (kBytes / 1024 + W - 1) / W; ++i)
        fetch16(to + (i * W + wave) * 1024, block, kBytes, (i * W + wave) * 1024 + lane * 16, 0);
}

// A workgroup's sequence, heads and part of its head's rows.  The workgroups of a key
// head are neighbours on one XCD (ids modulo 8), the key heads of a sequence spread
// over all: 8 x 4096 tokens bf16 554 us for the whole of gdn_chunk, with a sequence on
// one XCD 577.
__device__ __forceinline__ bool workgroup_at(const Packed &s, int parts, int &b, int &kh, int &h, int &part) {
    const int per = parts * (s.Hv / s.Hk), at = static_cast<int>(blockIdx.x >> 3) % per;
    const int unit = static_cast<int>(blockIdx.x >> 3) / per * 8 + (blockIdx.x & 7);
    b = unit / s.Hk;
    kh = unit - b * s.Hk;
    part = at % parts;
    h = kh + at / parts * s.Hk;
    return b < s.B;
}
inline unsigned walk_grid(const Packed &s, int parts) {
    const int64_t units = static_cast<int64_t>(s.B) * s.Hk;
    return static_cast<unsigned>((units + 7) / 8 * 8 * parts * (s.Hv / s.Hk));
}

// W waves, 16 rows of the state each.  NP planes of k and q, NO of what only the
// outputs see; S buffers of a chunk's operands.  For the backward pass (kBack) the
// states that enter each chunk and the corrections are kept, and the outputs
// only meet their gradient: od is the sum over the wave's rows of out * d_out.
template <typename ET, int NP, int NO, int W, int S, bool kBack>
__global__ __launch_bounds__(64 * W) void k_walk(ChunkArgs a, int parts) {
    typedef typename ET::bits bits;
    typedef Stage<NP, NO> L;
    constexpr int kAhead = NP == 1 ? 2 : 1;               // sets of K and Q operands in registers
    __shared__ alignas(1024) char buf0[L::kBytes], buf1[S > 1 ? L::kBytes : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int Hv = a.s.Hv;
    int b, kh, h, part;
    if (!workgroup_at(a.s, parts, b, kh, h, part)) return;
    const int slot = slot_of(a.s, b);
    if (slot < 0) return;
    const Span sp = span_of(a.s, b);
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const int dv0 = (part * W + wave) * 16, dv = dv0 + r;   // this lane's row of M

    // M[dv][32 jj + 8 g + 0..7] are the four of tile 2 jj and the four of 2 jj + 1
    f4 M[8];
    const int64_t row = ((static_cast<int64_t>(slot) * Hv + h) * kHeadDim + dv) * kHeadDim + 8 * g;
#pragma unroll
    for (int t = 0; t < 8; ++t)
        M[t] = a.state ? *reinterpret_cast<const f4 *>(a.state + row + 32 * (t / 2) + 4 * (t % 2)) : f4{0, 0, 0, 0};

    const int place0 = place_of(sp.first, b);
    auto fetch = [&](char *to, int c) {
        const int64_t place = place0 + c;
        const int rows = min(kChunk, sp.len - c * kChunk);
        fetch_rows<ET, NP, W>(a, to + L::kK, to + L::kQ, place, sp.first + c * kChunk, rows, kh, wave, lane);
        fetch_block<within_bytes(NO), W>(a.within + (place * Hv + h) * within_bytes(NO), to + L::kT, wave, lane);
        if constexpr (S > 1) in_order();                  // ahead of what is counted
    };
    auto rows_of = [&](const void *base, int c) {
        return Rows<ET>(base, static_cast<int64_t>(sp.first) + c * kChunk, min(kChunk, sp.len - c * kChunk), h, Hv);
    };
    bits vn[16];                                          // v of the chunk to come
    auto load_v = [&](int c) {
        const Rows<ET> v = rows_of(a.v, c);
#pragma unroll
        for (int i = 0; i < 16; ++i) vn[i] = v.load(16 * (i / 4) + 4 * g + i % 4, dv);
    };

    auto chunk = [&](char *cur, char *nxt, int c) {
        const int64_t ph = (static_cast<int64_t>(place0) + c) * Hv + h;
        const int rows = min(kChunk, sp.len - c * kChunk);
        if constexpr (kBack) {
            float *to = a.states + ph * (kHeadDim * kHeadDim) + dv * kHeadDim + 8 * g;
#pragma unroll
            for (int t = 0; t < 8; ++t) *reinterpret_cast<f4 *>(to + 32 * (t / 2) + 4 * (t % 2)) = M[t];
        }
        if (S == 1) {
            wait_lds();
            meet();                                       // the buffer is read
            fetch(cur, c);
            wait_all<0>();
        } else {
            // This chunk's fetches have landed; what came behind them may still be on
            // its way: the 16 loads of v at least, and for the backward pass 16 stores
            // of corrections.
            wait_all<kBack ? 32 : 16>();
        }
        clear_rows<NP, W>(cur + L::kK, cur + L::kQ, rows);
        meet();                                           // cur has landed, nxt is read
        if (S > 1 && c + 1 < chunks) fetch(nxt, c + 1);
        // K and Q against the state, 32 dk at a time, the next ones read ahead
        f4 Y[4] = {}, Z[4] = {};
        u4 kf[kAhead][4][NP], qf[kAhead][4][NP];
        auto read = [&](int jj) {
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const int at = p * kPlaneBytes + plane_at(jt * 16 + r, 4 * jj + g);
                    kf[jj % kAhead][jt][p] = *reinterpret_cast<const u4 *>(cur + L::kK + at);
                    qf[jj % kAhead][jt][p] = *reinterpret_cast<const u4 *>(cur + L::kQ + at);
                }
        };
        if (kAhead > 1) read(0);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            if (kAhead == 1) read(jj);
            else if (jj < 3) read(jj + 1);
            u4 m3[3], mo[NO];
            planes_of<3>(M[2 * jj], M[2 * jj + 1], m3);
#pragma unroll
            for (int p = 0; p < NO; ++p) mo[p] = m3[p];
            mma_planes<2, true>(kf[jj % kAhead], m3, Y);              // token 4 g + e, row dv
            mma_planes<NO - 1, false>(qf[jj % kAhead], mo, Z);        // dv 4 g + e, token r
        }
        const float *vec = reinterpret_cast<const float *>(cur + L::kVec);
        f4 X[4], E[4] = {};
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            const f4 rise = *reinterpret_cast<const f4 *>(vec + 16 * jt + 4 * g);
            const f4 beta = *reinterpret_cast<const f4 *>(vec + 2 * kChunk + 16 * jt + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                X[jt][e] = beta[e] * fmaf(-rise[e], Y[jt][e], ET::get(vn[4 * jt + e]));
        }
        if (c + 1 < chunks) load_v(c + 1);
        // Delta: token 4 g + e, row dv
        u4 tf[4][3], xp[3];
#pragma unroll
        for (int it = 0; it < 4; ++it) operand_at<3>(cur + L::kT, pblock_of(it, 0), lane, tf[it]);
        planes_of<3>(X[0], X[1], xp);
        mma_planes<2, true>(tf, xp, E);
        u4 te[2][3];
#pragma unroll
        for (int it = 0; it < 2; ++it) operand_at<3>(cur + L::kT, pblock_of(it + 2, 1), lane, te[it]);
        planes_of<3>(X[2], X[3], xp);
        f4 (&E2)[2] = *reinterpret_cast<f4 (*)[2]>(&E[2]);
        mma_planes<2, true>(te, xp, E2);
        if constexpr (kBack) {
            float *to = a.delta + (ph * kChunk + 4 * g) * kHeadDim + dv;
#pragma unroll
            for (int i = 0; i < 16; ++i) to[(16 * (i / 4) + i % 4) * kHeadDim] = E[i / 4][i % 4];
        }
        // outputs
        u4 dp[2][NO];
        planes_of<NO>(E[0], E[1], dp[0]);
        planes_of<NO>(E[2], E[3], dp[1]);
        const Rows<ET> out = rows_of(kBack ? a.d_out : a.out, c);
        f4 dout[4];
        if constexpr (kBack)
#pragma unroll
            for (int it = 0; it < 4; ++it) dout[it] = out.load4(16 * it + r, dv0 + 4 * g);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            f4 o = Z[it] * (kReadScale * vec[16 * it + r]);
#pragma unroll
            for (int half = 0; half <= it / 2; ++half) {
                u4 pf[NO];
                operand_at<NO>(cur + L::kP, pblock_of(it, half), lane, pf);
                o = mma_planes<NO - 1>(dp[half], pf, o);
            }
            if constexpr (kBack) {
                float s = 0.0f;                           // d_out is zero past the last token
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fmaf(o[e], dout[it][e], s);
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (g == 0) a.od[(ph * 8 + part * W + wave) * kChunk + 16 * it + r] = s;
            } else {
                out.store4(16 * it + r, dv0 + 4 * g, o);
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
            u4 ep[3], kt[8][NP];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int p = 0; p < NP; ++p) kt[t][p] = columns_of(cur + L::kK + p * kPlaneBytes, half, t, r, g);
            planes_of<3>(E[2 * half], E[2 * half + 1], ep);
            mma_planes<2, true>(kt, ep, M);
        }
    };
    if (chunks > 0) {
        if (S > 1) fetch(buf0, 0);
        load_v(0);
        wait_all<0>();
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

// Eight waves of 16 rows are a head; in two workgroups of four where that leaves each
// compute unit one: a wave alone on its SIMD goes through a chunk faster than two of
// them (2048 tokens, 32 heads a sequence, the whole of gdn_chunk, in two against one: 1
// sequence 138 against 175 us, 3 168 against 200, 4 191 against 214, 6 343 against
// 254; in four or eight never faster than in two by more than 1 %).
constexpr bool halves_heads(int64_t heads, int cus) { return 2 * heads <= cus; }

template <typename ET, int NP, int NO, int W, int S, bool kBack>
hipError_t launch_walk_of(const ChunkArgs &a, hipStream_t s) {
    const int parts = 8 / W;
    k_walk<ET, NP, NO, W, S, kBack><<<dim3(walk_grid(a.s, parts)), dim3(64 * W), 0, s>>>(a, parts);
    return hipGetLastError();
}
template <typename ET, int NP, int NO, int S, bool kBack>
hipError_t launch_walk(const ChunkArgs &a, hipStream_t s) {
    const bool halves = halves_heads(static_cast<int64_t>(a.s.B) * a.s.Hv, device_cus());
    return halves ? launch_walk_of<ET, NP, NO, 4, S, kBack>(a, s) : launch_walk_of<ET, NP, NO, 8, S, kBack>(a, s);
}

}  // namespace
}  // namespace gdn
