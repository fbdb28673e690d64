// gdn_chunk_back.hip - gdn_chunk_backward: the gradient of gdn_chunk.
//
// Mathematics, with the names of gdn_walk.hpp, G the gradient of the state that
// leaves a chunk, rise = e^g, fall = e^{g_64 - g} and s = 1 / sqrt(128):
//   U = K G^T,  dDelta = P^T dO + diag(fall) U,  R = T^T dDelta,  dV = diag(beta) R,
//   G' = e^{g_64} G + s dO^T diag(rise) Q - dV^T diag(rise) K        (k_back)
// for the chunk before, and then, chunk by chunk,                    (k_grad)
//   D_ij = e^{g_i - g_j},  F = s tril(dO Delta^T) o D,
//   E = -stril(R Delta^T) o (beta_i D),
//   dQ = s diag(rise) dO M + F K,
//   dK = -diag(beta rise) R M + diag(fall) Delta G + F^T Q + (E + E^T) K,
//   dbeta_i = R_i . Delta_i / beta_i.
// Everything that decays shares the running sums g, and the terms of their
// gradient meet: with c_i = dO_i . O_i - dV_i . V_i,
//   dgate_t = sum over the chunk's i >= t of c_i + <G, M'>,
//   <G, M'> = e^{g_64} <G, M> + sum_j fall_j Delta_j . U_j,
// a suffix sum of one chunk, kept in binary64.  dQ and dK of a key head are summed
// over the value heads that share it, in registers.
#include "gdn.h"
#include "gdn_walk.hpp"

namespace gdn {
namespace {

// Two of a token's planes as an operand: elements of tokens 4 g + e of tiles a and b.
template <typename ET, int NP>
__device__ __forceinline__ void planes_in(const typename ET::bits *x, u4 (&p)[NP]) {
    if constexpr (NP == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[0][i] = static_cast<uint32_t>(x[2 * i]) | static_cast<uint32_t>(x[2 * i + 1]) << 16;
    } else {
        planes_of<NP>(f4{ET::get(x[0]), ET::get(x[1]), ET::get(x[2]), ET::get(x[3])},
                      f4{ET::get(x[4]), ET::get(x[5]), ET::get(x[6]), ET::get(x[7])}, p);
    }
}

// Columns dk 16 t + r of a plane as an operand whose k are the tokens as in
// columns_of.  turn() is the same for rows 16 apart, so that a lane needs one place
// for each t.
__device__ __forceinline__ int plain_place(int r, int g) {
    return plane_at(4 * g + (r >> 2), r >> 1 & 1) + 8 * (r & 1);
}
__device__ __forceinline__ u4 plain_columns(const char *plane, int half, int t, int place) {
    const char *at = plane + (place ^ t << 5) + half * 32 * 256;
    const u2 x = read_columns(at), y = read_columns(at + 16 * 256);
    return u4{x.x, x.y, y.x, y.y};
}
// The same whose k are the rows 8 g + e of a slab of 32.
__device__ __forceinline__ int slab_place(int r, int g) {
    return plane_at(8 * g + (r >> 2), r >> 1 & 1) + 8 * (r & 1);
}
__device__ __forceinline__ u4 slab_columns(const char *plane, int t, int place) {
    const u2 x = read_columns(plane + (place ^ t << 5)), y = read_columns(plane + (place ^ (t << 5 | 16)) + 4 * 256);
    return u4{x.x, x.y, y.x, y.y};
}
// Keeps what is derived from x from being formed ahead of a loop and spilled there.
__device__ __forceinline__ int here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The planes of a chunk's k (which = 0) or q to LDS, zero past its n tokens.
template <typename ET, int NP, int kThreads>
__device__ __forceinline__ void load_planes(const ChunkArgs &a, int which, char *to, int place, int64_t t0, int n, int kh) {
    if constexpr (NP == 1) {
        const Rows<ET> rows(which ? a.q : a.k, t0, n, kh, a.s.Hk);
        for (int i = threadIdx.x; i < kPlaneBytes / 16; i += kThreads)
            *reinterpret_cast<u4 *>(to + plane_at(i >> 4, i & 15)) = rows.load8(i >> 4, 8 * (i & 15)).x[0];
    } else {
        const char *kq = a.kq + ((static_cast<int64_t>(place) * a.s.Hk + kh) * 2 + which) * (NP * kPlaneBytes);
        for (int i = threadIdx.x; i < NP * kPlaneBytes / 16; i += kThreads)
            *reinterpret_cast<u4 *>(to + i * 16) = *reinterpret_cast<const u4 *>(kq + i * 16);
    }
}

// Along the sequences in reverse, 16 rows of G a wave as k_walk has rows of M, and bound
// as that is: 8 ragged sequences of up to 4096 tokens bf16 632 us (19 thousand tokens; k_walk
// with what the backward pass keeps of it 596), 1 x 333 36 us.
template <typename ET, int NP, int W, int S>
__global__ __launch_bounds__(64 * W) void k_back(BackArgs a, int parts) {
    typedef typename ET::bits bits;
    typedef Stage<NP, 3> L;
    constexpr int kAhead = NP == 1 ? 2 : 1;
    __shared__ alignas(1024) char buf0[L::kBytes], buf1[S > 1 ? L::kBytes : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const Packed &s = a.f.s;
    const int Hv = s.Hv;
    int b, kh, h, part;
    if (!workgroup_at(s, parts, b, kh, h, part)) return;
    const Span sp = span_of(s, b);
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const int dv = (part * W + wave) * 16 + r;

    f4 G[8];
    const int64_t row = ((static_cast<int64_t>(b) * Hv + h) * kHeadDim + dv) * kHeadDim + 8 * g;
#pragma unroll
    for (int t = 0; t < 8; ++t)
        G[t] = a.d_state_out ? *reinterpret_cast<const f4 *>(a.d_state_out + row + 32 * (t / 2) + 4 * (t % 2))
                             : f4{0, 0, 0, 0};
    const int place0 = place_of(sp.first, b);
    auto fetch = [&](char *to, int c) {
        const int64_t place = place0 + c;
        const int rows = min(kChunk, sp.len - c * kChunk);
        fetch_rows<ET, NP, W>(a.f, to + L::kK, to + L::kQ, place, sp.first + c * kChunk, rows, kh, wave, lane);
        fetch_block<within_bytes(3), W>(a.back + (place * Hv + h) * within_bytes(3), to + L::kT, wave, lane);
    };
    auto rows_of = [&](const void *base, int c) {
        return Rows<ET>(base, static_cast<int64_t>(sp.first) + c * kChunk, min(kChunk, sp.len - c * kChunk), h, Hv);
    };
    bits on[16];                                          // d_out of the chunk to come
    auto load_o = [&](int c) {
        const Rows<ET> o = rows_of(a.f.d_out, c);
#pragma unroll
        for (int i = 0; i < 16; ++i) on[i] = o.load(16 * (i / 4) + 4 * g + i % 4, dv);
    };

    auto chunk = [&](char *cur, char *nxt, int c) {
        const int64_t ph = (static_cast<int64_t>(place0) + c) * Hv + h;
        float *keep = a.dstates + ph * (kHeadDim * kHeadDim) + dv * kHeadDim + 8 * g;
#pragma unroll
        for (int t = 0; t < 8; ++t) *reinterpret_cast<f4 *>(keep + 32 * (t / 2) + 4 * (t % 2)) = G[t];
        float dl[16];                                     // Delta, as U lies
#pragma unroll
        for (int i = 0; i < 16; ++i)
            dl[i] = a.f.delta[(ph * kChunk + 16 * (i / 4) + 4 * g + i % 4) * kHeadDim + dv];
        if (S == 1) {
            wait_lds();
            meet();                                       // the buffer is read
            fetch(cur, c);
            wait_all<0>();
        } else {
            // This chunk's fetches have landed; behind them came 32 stores of R and dV, 16
            // loads of d_out, 8 stores of G and 16 loads of Delta.
            wait_all<48>();
        }
        const int rows = min(kChunk, sp.len - c * kChunk);
        clear_rows<NP, W>(cur, cur + L::kQ, rows);
        meet();
        if (S > 1 && c > 0) fetch(nxt, c - 1);
        const float *vec = reinterpret_cast<const float *>(cur + L::kVec);
        f4 U[4] = {};
        u4 kf[kAhead][4][NP];
        auto read = [&](int jj) {
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    kf[jj % kAhead][jt][p] = *reinterpret_cast<const u4 *>(cur + L::kK + p * kPlaneBytes +
                                                                           plane_at(jt * 16 + r, 4 * jj + g));
        };
        if (kAhead > 1) read(0);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            if (kAhead == 1) read(jj);
            else if (jj < 3) read(jj + 1);
            u4 g3[3];
            planes_of<3>(G[2 * jj], G[2 * jj + 1], g3);
            mma_planes<2, true>(kf[jj % kAhead], g3, U);
        }
        u4 op[2][NP];
        planes_in<ET, NP>(on, op[0]);
        planes_in<ET, NP>(on + 8, op[1]);
        float du = 0.0f;
        f4 dd[4];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            const f4 fall = *reinterpret_cast<const f4 *>(vec + kChunk + 16 * jt + 4 * g);
            dd[jt] = fall * U[jt];
#pragma unroll
            for (int e = 0; e < 4; ++e) du = fmaf(dl[4 * jt + e], dd[jt][e], du);
#pragma unroll
            for (int half = jt / 2; half < 2; ++half) {
                u4 pf[3];
                operand_at<3>(cur + L::kP, pnblock_of(jt, half), lane, pf);
                dd[jt] = mma_planes<2>(pf, op[half], dd[jt]);
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) du += __shfl_xor(du, d);
        if (lane == 0) a.du[ph * 8 + part * W + wave] = du;
        f4 R[4] = {};
        u4 tf[4][3], xp[3];
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) operand_at<3>(cur + L::kT, pnblock_of(jt, 1), lane, tf[jt]);
        planes_of<3>(dd[2], dd[3], xp);
        mma_planes<2, true>(tf, xp, R);
        u4 te[2][3];
#pragma unroll
        for (int jt = 0; jt < 2; ++jt) operand_at<3>(cur + L::kT, pnblock_of(jt, 0), lane, te[jt]);
        planes_of<3>(dd[0], dd[1], xp);
        f4 (&R0)[2] = *reinterpret_cast<f4 (*)[2]>(&R[0]);
        mma_planes<2, true>(te, xp, R0);
        if constexpr (S > 1) in_order();                  // the next chunk's fetches are ahead of what is counted
        const Rows<ET> dvr = rows_of(a.dv, c);
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            const f4 beta = *reinterpret_cast<const f4 *>(vec + 2 * kChunk + 16 * jt + 4 * g);
            float *to = a.r + (ph * kChunk + 16 * jt + 4 * g) * kHeadDim + dv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                to[e * kHeadDim] = R[jt][e];
                R[jt][e] *= fabsf(beta[e]) <= kLeastBeta ? 0.0f : beta[e];
                dvr.store(16 * jt + 4 * g + e, dv, R[jt][e]);
            }
        }
        // the gradient of the state that enters the chunk
        const float all = vec[kChunk - 1];
#pragma unroll
        for (int t = 0; t < 8; ++t) G[t] *= all;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f4 xo[2], xv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f4 rise = *reinterpret_cast<const f4 *>(vec + 32 * half + 16 * i + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xo[i][e] = kReadScale * rise[e] * ET::get(on[8 * half + 4 * i + e]);
                    xv[i][e] = -rise[e] * R[2 * half + i][e];
                }
            }
            u4 po[3], pv[3];
            planes_of<3>(xo[0], xo[1], po);
            planes_of<3>(xv[0], xv[1], pv);
            u4 ct[8][NP];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int p = 0; p < NP; ++p) ct[t][p] = columns_of(cur + L::kQ + p * kPlaneBytes, half, t, r, g);
            mma_planes<2, true>(ct, po, G);
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int p = 0; p < NP; ++p) ct[t][p] = columns_of(cur + L::kK + p * kPlaneBytes, half, t, r, g);
            mma_planes<2, true>(ct, pv, G);
        }
        if (c > 0) load_o(c - 1);
    };
    if (chunks > 0) {
        if (S > 1) fetch(buf0, chunks - 1);
        load_o(chunks - 1);
        wait_all<0>();
        int c = chunks - 1;
        if constexpr (S > 1) {
            for (; c >= 1; c -= 2) {
                chunk(buf0, buf1, c);
                chunk(buf1, buf0, c - 1);
            }
            if (c == 0) chunk(buf0, buf1, 0);
        } else {
            for (; c >= 0; --c) chunk(buf0, buf0, c);
        }
    }
    if (a.d_state) {
#pragma unroll
        for (int t = 0; t < 8; ++t) *reinterpret_cast<f4 *>(a.d_state + row + 32 * (t / 2) + 4 * (t % 2)) = G[t];
    }
}

// ------------------------------------------------------------ chunk by chunk
// One workgroup of eight waves per chunk place and key head, the value heads that
// share the key head after each other.  Wave w + 4 p has the 16 tokens w as its
// rows, and half p of the dk columns of dQ and dK; of the products between tokens it
// forms F (p = 0) or E (p = 1), which change hands through LDS.  The products over
// dv run in slabs of 32: a wave's own rows of R, Delta and d_out come straight
// from memory as operands, and through LDS for the other waves; the slabs of M and G
// are cut into planes in LDS and read by columns; the next slab, of the next head too,
// is on its way meanwhile.  The vector units (cutting, 39 % busy), the matrix units (17 %)
// and waiting for memory and each other bound it; 8 ragged sequences of up to 4096 tokens, 32 value heads: 774 us
// (one buffer of slabs 806, four waves with whole rows of dk, products of rows scaled ahead: 1130).
// float32, three planes of everything, keeps 20 registers in scratch.
template <typename ET, int NP, int NO>
__global__ __launch_bounds__(512) void k_grad(BackArgs a) {
    constexpr int kRow = 64;                              // bytes of a token's slab of a plane
    constexpr int kTok = kChunk * kRow;                   // bytes of a plane of Delta, d_out or R
    constexpr int kMat = 32 * 256;                        // bytes of a plane of M or G
    // K and Q stay, the operands F and E take the slabs' place; f32 reads Q anew for each
    // head, to behind F and E.
    constexpr int kK = NP * kPlaneBytes, kSlab = 3 * NO * kTok + 2 * NO * kMat, kPass = 20 * NO * 1024;
    constexpr bool kStays = NP < 3;
    constexpr int kTurn = kStays ? 2 * kK : kK, kQ = kStays ? kK : kK + kPass;
    constexpr int kBuffers = NP == 1 ? 2 : 1;             // of slabs
    constexpr int kAll = kStays ? kTurn + kBuffers * (kSlab > kPass ? kSlab : kPass)
                                : kTurn + (kSlab > kPass + kK ? kSlab : kPass + kK);
    static_assert(kBuffers == 1 || kPass <= kSlab, "F and E fit the buffer that is not being read");
    __shared__ alignas(16) char lds[kAll];
    __shared__ double gs[kChunk], part[8];
    __shared__ float vec[kVecFloats], dots[2][kChunk], ods[8][kChunk], dus[8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, w = wave & 3, p = wave >> 2;
    char *const turn0 = lds + kTurn;
    const Packed &s = a.f.s;
    const int Hv = s.Hv, Hk = s.Hk;
    const int place = blockIdx.x / Hk, kh = blockIdx.x - place * Hk;
    const int b = sequence_at(s, place);
    const Span sp = span_of(s, b);
    const int c0 = (place - place_of(sp.first, b)) * kChunk;
    if (c0 < 0 || c0 >= sp.len) return;
    const int n = min(kChunk, sp.len - c0);
    const int64_t t0 = sp.first + c0;
    // 16 bytes of four k of eight each: chunk c of row t at c ^ (t >> 1 & 3), which
    // spreads 16 rows over the banks twice
    const auto tok_at = [](int t, int c) { return t * kRow + ((c ^ (t >> 1 & 3)) << 4); };
    // the planes of F to dQ, F to dK and E of a wave's tokens and one half of the others
    // (the halves that are there)
    const auto pass_at = [&](int lane, int which, int half, int m) {
        const int unit = which == 0 ? w + 2 * half : which == 1 ? 6 + w + 4 * (1 - half) : 12 + 2 * w + half;
        return turn0 + (unit * NO + m) * 1024 + lane * 16;
    };
    const auto decay = [](double x) { return exp_2(x); };

    f4 r0, r1, d0, d1, m0, m1, g0, g1;
    typename Rows<ET>::Eight o, v;
    double gx = 0.0;
    float vx = 0.0f, odx, dux = 0.0f;
    const auto load = [&](int h, int slab) {
        const int lane = here(threadIdx.x) & 63, r = lane & 15, g = lane >> 4, tok = w * 16 + r;
        const int64_t ph = static_cast<int64_t>(place) * Hv + h;
        const auto at = [](const float *base, int64_t first, unsigned lane_at, int i) {
            return *reinterpret_cast<const f4 *>(reinterpret_cast<const char *>(base + first) + lane_at + 16 * i);
        };
        const int64_t mat = ph * (kHeadDim * kHeadDim) + 32 * slab * kHeadDim, row = ph * (kChunk * kHeadDim) + 32 * slab;
        const unsigned mine = 32 * here(threadIdx.x), own = (tok * kHeadDim + 8 * g) * 4;
        m0 = at(a.f.states, mat, mine, 0);
        m1 = at(a.f.states, mat, mine, 1);
        g0 = at(a.dstates, mat, mine, 0);
        g1 = at(a.dstates, mat, mine, 1);
        r0 = at(a.r, row, own, 0);
        r1 = at(a.r, row, own, 1);
        d0 = at(a.f.delta, row, own, 0);
        d1 = at(a.f.delta, row, own, 1);
        // d_out and v past the last token read zero
        o = Rows<ET>(a.f.d_out, t0, n, h, Hv).load8(tok, 32 * slab + 8 * g);
        v = Rows<ET>(a.f.v, t0, n, h, Hv).load8(tok, 32 * slab + 8 * g);
    };
    const auto load_head = [&](int h) {
        const int64_t ph = static_cast<int64_t>(place) * Hv + h;
        const float *pvec = reinterpret_cast<const float *>(a.f.within + (ph + 1) * within_bytes(3) - 1024);
        if (threadIdx.x < kChunk) gx = a.gsum[ph * kChunk + threadIdx.x];
        if (threadIdx.x < kVecFloats) vx = pvec[threadIdx.x];
        odx = a.f.od[(ph * 8 + wave) * kChunk + lane];
        if (threadIdx.x < 8) dux = a.du[ph * 8 + threadIdx.x];
        load(h, 0);
    };
    load_head(kh);
    load_planes<ET, NP, 512>(a.f, 0, lds, place, t0, n, kh);
    if (kStays) load_planes<ET, NP, 512>(a.f, 1, lds + kQ, place, t0, n, kh);
    f4 dq[4] = {}, dk[4] = {};                            // rows 16 w + 4 g + e, column dk 16 (4 p + t) + r
#pragma unroll 1
    for (int h = kh; h < Hv; h += Hk) {
        // F or E between tiles of 16 tokens, lane: the own token, element: the other's;
        // with the tiles up to the own as the earlier ones, P[t], and from the own on as the
        // later ones, P[t + 1].
        f4 P[5] = {}, om[4] = {}, rm[4] = {}, dg[4] = {}; // and d_out M, R M and Delta G
        float dot = 0.0f, gm = 0.0f;
#pragma unroll 1
        for (int slab = 0; slab < 4; ++slab) {
            const int lane = here(threadIdx.x) & 63, r = lane & 15, g = lane >> 4, tok = w * 16 + r;
            u4 op[NO] = {}, rp[NO], dp[NO];
            // LDS of Delta, of d_out or R, which is the half's own, of M and of G
            char *const ld = turn0 + (kBuffers == 2 ? slab & 1 : 0) * kSlab, *const lx = ld + (1 + p) * NO * kTok,
                 *const lm = ld + 3 * NO * kTok, *const lg = lm + NO * kMat;
            if (kBuffers == 1 || slab == 0) {
                wait_lds();
                meet();                                   // the last slab, or F and E, is read
            }
            {
                const int mr = here(threadIdx.x) >> 4, mc = here(threadIdx.x) & 15;  // this thread's piece of M and G
                u4 mp[NO], gp[NO];
                planes_of<NO>(m0, m1, mp);
                planes_of<NO>(g0, g1, gp);
                planes_of<NO>(r0, r1, rp);
                planes_of<NO>(d0, d1, dp);
                if constexpr (NP == 1)
                    op[0] = o.x[0];
                else
                    planes_of<NO>(Rows<ET>::four(o, 0), Rows<ET>::four(o, 1), op);
#pragma unroll
                for (int m = 0; m < NO; ++m) {
                    *reinterpret_cast<u4 *>(lm + m * kMat + plane_at(mr, mc)) = mp[m];
                    *reinterpret_cast<u4 *>(lg + m * kMat + plane_at(mr, mc)) = gp[m];
                    *reinterpret_cast<u4 *>(lx + m * kTok + tok_at(tok, g)) = p == 0 ? op[m] : rp[m];
                    if (p == 0) *reinterpret_cast<u4 *>(ld + m * kTok + tok_at(tok, g)) = dp[m];
                }
                const f4 v0 = Rows<ET>::four(v, 0), v1 = Rows<ET>::four(v, 1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gm = fmaf(m0[e], g0[e], gm);
                    gm = fmaf(m1[e], g1[e], gm);
                    dot = fmaf(r0[e], p == 0 ? v0[e] : d0[e], dot);
                    dot = fmaf(r1[e], p == 0 ? v1[e] : d1[e], dot);
                }
                if (slab == 1) {                          // (the last head is done with them)
                    if (threadIdx.x < kChunk) gs[threadIdx.x] = gx;
                    if (threadIdx.x < kVecFloats) vec[threadIdx.x] = vx;
                    ods[wave][lane] = odx;
                    if (threadIdx.x < 8) dus[threadIdx.x] = dux;
                }
            }
            if (slab < 3)
                load(h, slab + 1);
            else if (h + Hk < Hv)
                load_head(h + Hk);
            wait_lds();
            meet();                                       // (the loads stay on their way)
#pragma unroll
            for (int u = 0; u < 5; ++u) {
                const bool to = u <= w;
                const char *other = to ? ld : lx;
                u4 oj[NO], ow[NO];
#pragma unroll
                for (int m = 0; m < NO; ++m) {
                    oj[m] = *reinterpret_cast<const u4 *>(other + m * kTok + tok_at((to ? u : u - 1) * 16 + r, g));
                    ow[m] = to ? (p == 0 ? op[m] : rp[m]) : dp[m];
                }
                P[u] = mma_planes<NO - 1>(oj, ow, P[u]);
            }
            // rows 8 g + e of the slab are an operand's k
            const int column = here(slab_place(r, g));
            u4 on[NP];
#pragma unroll
            for (int m = 0; m < NP; ++m) on[m] = op[m];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u4 mcol[NO], gcol[NO];
#pragma unroll
                for (int m = 0; m < NO; ++m) {
                    mcol[m] = slab_columns(lm + m * kMat, 4 * p + t, column);
                    gcol[m] = slab_columns(lg + m * kMat, 4 * p + t, column);
                }
                om[t] = mma_planes<NO - 1>(on, mcol, om[t]);
                rm[t] = mma_planes<NO - 1>(rp, mcol, rm[t]);
                dg[t] = mma_planes<NO - 1>(dp, gcol, dg[t]);
            }
        }
        const int lane = here(threadIdx.x) & 63, r = lane & 15, g = lane >> 4, tok = w * 16 + r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = w * 16 + 4 * g + e;
            const float rise = vec[row], fall = vec[kChunk + row], beta = vec[2 * kChunk + row];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                dq[t][e] = fmaf(kReadScale * rise, om[t][e], dq[t][e]);
                dk[t][e] = fmaf(fall, dg[t][e], fmaf(-beta * rise, rm[t][e], dk[t][e]));
            }
        }
        if (kBuffers == 1) {
            wait_lds();
            meet();                                       // the slabs are read: F and E take their place
        }
        if (!kStays) load_planes<ET, NP, 512>(a.f, 1, lds + kQ, place, t0, n, kh);
        // decays and masks
        const double gt = gs[tok];
        if (p == 0) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f4 early[2], late[2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = (2 * half + t) * 16 + 4 * g + e;
                        const double x = gt - gs[i];
                        const float d = kReadScale * decay(i <= tok ? x : -x);
                        early[t][e] = i <= tok ? d * P[2 * half + t][e] : 0.0f;
                        late[t][e] = i >= tok ? d * P[2 * half + t + 1][e] : 0.0f;
                    }
                u4 f[NO];
                if (2 * half <= w) {
                    planes_of<NO>(early[0], early[1], f);
#pragma unroll
                    for (int m = 0; m < NO; ++m) *reinterpret_cast<u4 *>(pass_at(lane, 0, half, m)) = f[m];
                }
                if (2 * half + 1 >= w) {
                    planes_of<NO>(late[0], late[1], f);
#pragma unroll
                    for (int m = 0; m < NO; ++m) *reinterpret_cast<u4 *>(pass_at(lane, 1, half, m)) = f[m];
                }
            }
        } else {
            const float beta = vec[2 * kChunk + tok];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f4 both[2];                               // E + E^T
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = (2 * half + t) * 16 + 4 * g + e;
                        const double x = gt - gs[i];
                        const float d = decay(i < tok ? x : -x);
                        const float y = i < tok ? beta * P[2 * half + t][e] : vec[2 * kChunk + i] * P[2 * half + t + 1][e];
                        both[t][e] = i == tok ? 0.0f : -d * y;
                    }
                u4 f[NO];
                planes_of<NO>(both[0], both[1], f);
#pragma unroll
                for (int m = 0; m < NO; ++m) *reinterpret_cast<u4 *>(pass_at(lane, 2, half, m)) = f[m];
            }
        }
        // per token: the sums over dv of its four lanes
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        double gd = gm;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) gd += __shfl_xor(gd, d);
        if (g == 0) dots[p][tok] = dot;
        if (lane == 0) part[wave] = gd;
        wait_lds();
        meet();
        if (wave == 0) {
            const float bl = vec[2 * kChunk + lane];
            double od = 0.0, du = 0.0, mg = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) od += ods[i][lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) mg += part[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) du += dus[i];
            const double end = du + static_cast<double>(vec[kChunk - 1]) * mg;
            double y = od - static_cast<double>(fabsf(bl) <= kLeastBeta ? 0.0f : bl) * dots[0][lane];
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const double z = __shfl_down(y, d);
                if (lane + d < 64) y += z;
            }
            if (lane < n) {
                a.dgate[(t0 + lane) * Hv + h] = static_cast<float>(y + end);
                a.dbeta[(t0 + lane) * Hv + h] = dots[1][lane] / bl;
            }
        }
        const int column = here(plain_place(r, g));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u4 f[NO], e[NO];
#pragma unroll
            for (int m = 0; m < NO; ++m) {
                f[m] = *reinterpret_cast<const u4 *>(pass_at(lane, 0, half, m));
                e[m] = *reinterpret_cast<const u4 *>(pass_at(lane, 2, half, m));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u4 kc[NP];
#pragma unroll
                for (int m = 0; m < NP; ++m) kc[m] = plain_columns(lds + m * kPlaneBytes, half, 4 * p + t, column);
                if (2 * half <= w) dq[t] = mma_planes<NO - 1>(f, kc, dq[t]);
                dk[t] = mma_planes<NO - 1>(e, kc, dk[t]);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
            if (2 * half + 1 >= w) {
                u4 f[NO];
#pragma unroll
                for (int m = 0; m < NO; ++m) f[m] = *reinterpret_cast<const u4 *>(pass_at(lane, 1, half, m));
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    u4 qc[NP];
#pragma unroll
                    for (int m = 0; m < NP; ++m) qc[m] = plain_columns(lds + kQ + m * kPlaneBytes, half, 4 * p + t, column);
                    dk[t] = mma_planes<NO - 1>(f, qc, dk[t]);
                }
            }
    }
    const Rows<ET> qo(a.dq, t0, n, kh, Hk), ko(a.dk, t0, n, kh, Hk);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            qo.store(w * 16 + 4 * g + e, 16 * (4 * p + t) + r, dq[t][e]);
            ko.store(w * 16 + 4 * g + e, 16 * (4 * p + t) + r, dk[t][e]);
        }
}

// Waves a workgroup as in launch_walk.
template <typename ET, int NP, int W, int S>
hipError_t launch_back_of(const BackArgs &a, hipStream_t s) {
    const int parts = 8 / W;
    k_back<ET, NP, W, S><<<dim3(walk_grid(a.f.s, parts)), dim3(64 * W), 0, s>>>(a, parts);
    return hipGetLastError();
}
template <typename ET, int NP, int S>
hipError_t launch_back(const BackArgs &a, hipStream_t s) {
    const bool halves = halves_heads(static_cast<int64_t>(a.f.s.B) * a.f.s.Hv, device_cus());
    return halves ? launch_back_of<ET, NP, 4, S>(a, s) : launch_back_of<ET, NP, 8, S>(a, s);
}

template <typename ET, int NP, int NO, int S>
hipError_t launch(const BackArgs &a, hipStream_t s) {
    PrepArgs p{};
    p.s = a.f.s;
    p.q = a.f.q;
    p.k = a.f.k;
    p.beta = a.f.beta;
    p.gate = a.f.gate;
    p.within = a.f.within;
    p.kq = a.f.kq;
    p.back = a.back;
    p.gsum = a.gsum;
    hipError_t e = launch_prep<ET, NP, 3, true>(p, s);
    if (e != hipSuccess) return e;
    e = launch_walk<ET, NP, 3, S, true>(a.f, s);
    if (e != hipSuccess) return e;
    e = launch_back<ET, NP, S>(a, s);
    if (e != hipSuccess) return e;
    const int64_t places = chunk_places(a.f.s.B, a.f.s.tokens) * a.f.s.Hk;
    k_grad<ET, NP, NO><<<dim3(static_cast<unsigned>(places)), dim3(512), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_backward(const BackArgs &a, hipStream_t s) {
    switch (a.f.s.type) {
    case GDN_F32: return launch<F32, 3, 3, 1>(a, s);
    case GDN_BF16: return launch<BF16, 1, 2, 2>(a, s);
    case GDN_F16: return launch<F16, 2, 2, 1>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
