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

// Columns dk 16 t + r of a plane as an operand: k are the tokens as in columns_of
// (plain_columns), or the rows 8 g + e of a slab of 32.
__device__ __forceinline__ u4 plain_columns(const char *plane, int half, int t, int r, int g) {
    const int tok = 32 * half + 4 * g + (r >> 2), chunk = 2 * t + (r >> 1 & 1);
    const u2 x = read_columns(plane + plane_at(tok, chunk) + 8 * (r & 1));
    const u2 y = read_columns(plane + plane_at(tok + 16, chunk) + 8 * (r & 1));
    return u4{x.x, x.y, y.x, y.y};
}
__device__ __forceinline__ u4 slab_columns(const char *plane, int t, int r, int g) {
    const int row = 8 * g + (r >> 2), chunk = 2 * t + (r >> 1 & 1);
    const u2 x = read_columns(plane + plane_at(row, chunk) + 8 * (r & 1));
    const u2 y = read_columns(plane + plane_at(row + 4, chunk) + 8 * (r & 1));
    return u4{x.x, x.y, y.x, y.y};
}

// The planes of a chunk's k, then q, to LDS, zero past its n tokens; ends with a
// barrier.
template <typename ET, int NP>
__device__ __forceinline__ void load_kq(const ChunkArgs &a, char *to, int place, int64_t t0, int n, int kh) {
    const char *kq = a.kq + (static_cast<int64_t>(place) * a.s.Hk + kh) * (2 * NP * kPlaneBytes);
    for (int i = threadIdx.x; i < 2 * NP * kPlaneBytes / 16; i += 256) {
        u4 x = {0, 0, 0, 0};
        int at = i * 16;
        if constexpr (NP == 1) {
            const int row = i >> 4 & 63, chunk = i & 15;
            at = (i >> 10) * kPlaneBytes + plane_at(row, chunk);
            if (row < n)
                x = *reinterpret_cast<const u4 *>(static_cast<const char *>(i < 1024 ? a.k : a.q) +
                                                  ((t0 + row) * a.s.Hk + kh) * (kHeadDim * 2) + chunk * 16);
        } else {
            x = *reinterpret_cast<const u4 *>(kq + at);
        }
        *reinterpret_cast<u4 *>(to + at) = x;
    }
    __syncthreads();
}

// Along the sequences in reverse, 16 rows of G a wave as k_walk has rows of M.
template <typename ET, int NP, int W, int S>
__global__ __launch_bounds__(64 * W) void k_back(BackArgs a, int parts) {
    typedef typename ET::bits bits;
    typedef Stage<NP, 3> L;
    constexpr int kAhead = NP == 1 ? 2 : 1;
    __shared__ alignas(1024) char buf0[L::kBytes], buf1[S > 1 ? L::kBytes : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const Packed &s = a.f.s;
    const int Hv = s.Hv, Hk = s.Hk;
    const int id = (blockIdx.x & 7) * static_cast<int>(gridDim.x >> 3) + (blockIdx.x >> 3);
    const int part = id % parts, hh = id / parts;
    const int b = hh / Hv;
    if (b >= s.B) return;
    const int kh = (hh - b * Hv) / (Hv / Hk), h = kh + (hh - b * Hv) % (Hv / Hk) * Hk;
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
            meet();
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
// One workgroup of four waves per chunk place and key head, 16 tokens a wave, the
// value heads that share the key head after each other.  The products over dv
// run in slabs of 32: a wave's own rows of R, Delta and d_out come straight from
// memory as operands, and through LDS for the other waves; the slabs of M and G
// are cut into planes in LDS and read by columns.
template <typename ET, int NP, int NO>
__global__ __launch_bounds__(256) void k_grad(BackArgs a) {
    typedef typename ET::bits bits;
    constexpr int kRow = 64;                              // bytes of a token's slab of a plane
    constexpr int kTok = kChunk * kRow;                   // bytes of a plane of R, Delta, d_out
    constexpr int kMat = 32 * 256;                        // bytes of a plane of M or G
    // the slabs, and after the last of them the planes of K and Q
    constexpr int kSlab = (2 * NO + NP) * kTok + 2 * NO * kMat, kKQ = 2 * NP * kPlaneBytes;
    __shared__ alignas(16) char lds[kSlab > kKQ ? kSlab : kKQ];
    __shared__ double gs[kChunk];
    __shared__ float vec[kVecFloats], dots[3][kChunk];
    __shared__ double part[4];
    char *const lr = lds, *const ld = lr + NO * kTok, *const lo = ld + NO * kTok, *const lm = lo + NP * kTok,
         *const lg = lm + NO * kMat;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const Packed &s = a.f.s;
    const int Hv = s.Hv, Hk = s.Hk;
    const int place = blockIdx.x / Hk, kh = blockIdx.x - place * Hk;
    const int b = sequence_at(s, place);
    const Span sp = span_of(s, b);
    const int c0 = (place - place_of(sp.first, b)) * kChunk;
    if (c0 < 0 || c0 >= sp.len) return;
    const int n = min(kChunk, sp.len - c0);
    const int64_t t0 = sp.first + c0;
    const int tok = wave * 16 + r;                        // this lane's token as a row or column
    // 16 bytes of four k of eight each: chunk c of row t at c ^ (t >> 1 & 3), which
    // spreads 16 rows over the banks twice
    const auto tok_at = [](int t, int c) { return t * kRow + ((c ^ (t >> 1 & 3)) << 4); };

    f4 dq[8] = {}, dk[8] = {};                            // rows 16 wave + 4 g + e, column dk 16 t + r
    for (int x = 0; x < Hv / Hk; ++x) {
        const int h = kh + x * Hk;
        const int64_t ph = static_cast<int64_t>(place) * Hv + h;
        if (x > 0) __syncthreads();                       // the last head is done with LDS
        if (threadIdx.x < kChunk) gs[threadIdx.x] = a.gsum[ph * kChunk + threadIdx.x];
        if (threadIdx.x < kVecFloats) vec[threadIdx.x] = reinterpret_cast<const float *>(
            a.f.within + (ph + 1) * within_bytes(3) - 1024)[threadIdx.x];
        f4 Z[8] = {}, Wm[8] = {}, H[8] = {};
        // lane: own token; elements: the other's.  F1, E1 of tiles up to the own, F2, E2
        // from it on.
        f4 F1[4] = {}, E1[4] = {}, F2[4] = {}, E2[4] = {};
        float rd = 0.0f, rv = 0.0f, gm = 0.0f;
        const float *pr = a.r + (ph * kChunk + tok) * kHeadDim + 8 * g;
        const float *pd = a.f.delta + (ph * kChunk + tok) * kHeadDim + 8 * g;
        const int64_t vat = ((t0 + tok) * Hv + h) * kHeadDim + 8 * g;
        for (int slab = 0; slab < 4; ++slab) {
            u4 rp[NO], dp[NO], op[NP] = {};
            {
                const f4 r0 = *reinterpret_cast<const f4 *>(pr + 32 * slab), r1 = *reinterpret_cast<const f4 *>(pr + 32 * slab + 4);
                const f4 d0 = *reinterpret_cast<const f4 *>(pd + 32 * slab), d1 = *reinterpret_cast<const f4 *>(pd + 32 * slab + 4);
                planes_of<NO>(r0, r1, rp);
                planes_of<NO>(d0, d1, dp);
                if (tok < n) {
                    load_planes<ET, NP>(a.f.d_out, vat + 32 * slab, op);
                    const auto v = Pack<bits, 8>::load(static_cast<const bits *>(a.f.v) + vat + 32 * slab);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        rd = fmaf(r0[e], d0[e], rd);
                        rd = fmaf(r1[e], d1[e], rd);
                        rv = fmaf(r0[e], ET::get(v[e]), rv);
                        rv = fmaf(r1[e], ET::get(v[4 + e]), rv);
                    }
                }
            }
            if (slab > 0) __syncthreads();                // the last slab is read
#pragma unroll
            for (int p = 0; p < NO; ++p) {
                *reinterpret_cast<u4 *>(lr + p * kTok + tok_at(tok, g)) = rp[p];
                *reinterpret_cast<u4 *>(ld + p * kTok + tok_at(tok, g)) = dp[p];
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<u4 *>(lo + p * kTok + tok_at(tok, g)) = op[p];
            // M and G: 32 rows of 16 chunks of eight
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = i * 256 + threadIdx.x, rr = at >> 4, ch = at & 15;
                const int64_t src = ph * (kHeadDim * kHeadDim) + (32 * slab + rr) * kHeadDim + 8 * ch;
                const f4 m0 = *reinterpret_cast<const f4 *>(a.f.states + src), m1 = *reinterpret_cast<const f4 *>(a.f.states + src + 4);
                const f4 g0 = *reinterpret_cast<const f4 *>(a.dstates + src), g1 = *reinterpret_cast<const f4 *>(a.dstates + src + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gm = fmaf(m0[e], g0[e], gm);
                    gm = fmaf(m1[e], g1[e], gm);
                }
                u4 mp[NO], gp[NO];
                planes_of<NO>(m0, m1, mp);
                planes_of<NO>(g0, g1, gp);
#pragma unroll
                for (int p = 0; p < NO; ++p) {
                    *reinterpret_cast<u4 *>(lm + p * kMat + plane_at(rr, ch)) = mp[p];
                    *reinterpret_cast<u4 *>(lg + p * kMat + plane_at(rr, ch)) = gp[p];
                }
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u4 rj[NO], dj[NO], oj[NP];
#pragma unroll
                for (int p = 0; p < NO; ++p) {
                    rj[p] = *reinterpret_cast<const u4 *>(lr + p * kTok + tok_at(t * 16 + r, g));
                    dj[p] = *reinterpret_cast<const u4 *>(ld + p * kTok + tok_at(t * 16 + r, g));
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) oj[p] = *reinterpret_cast<const u4 *>(lo + p * kTok + tok_at(t * 16 + r, g));
                if (t <= wave) {
                    F1[t] = mma_planes<NO - 1>(dj, op, F1[t]);
                    E1[t] = mma_planes<NO - 1>(dj, rp, E1[t]);
                }
                if (t >= wave) {
                    F2[t] = mma_planes<NO - 1>(oj, dp, F2[t]);
                    E2[t] = mma_planes<NO - 1>(rj, dp, E2[t]);
                }
            }
            // rows 8 g + e of the slab are an operand's k; column dk 16 t + r
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                u4 mc[NO], gc[NO];
#pragma unroll
                for (int p = 0; p < NO; ++p) {
                    mc[p] = slab_columns(lm + p * kMat, t, r, g);
                    gc[p] = slab_columns(lg + p * kMat, t, r, g);
                }
                Z[t] = mma_planes<NO - 1>(op, mc, Z[t]);
                Wm[t] = mma_planes<NO - 1>(rp, mc, Wm[t]);
                H[t] = mma_planes<NO - 1>(dp, gc, H[t]);
            }
        }
        __syncthreads();                                  // the slabs are read: K and Q take their place
        load_kq<ET, NP>(a.f, lds, place, t0, n, kh);
        // decays and masks; F1 and E1 are j <= i = tok, F2 and E2 i >= j = tok
        const double gt = gs[tok];
        const float bt = vec[2 * kChunk + tok];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int o = t * 16 + 4 * g + e;
                float e1 = 0.0f, e2 = 0.0f, f1 = 0.0f, f2 = 0.0f;
                if (o <= tok) {
                    const float d = expf(static_cast<float>(gt - gs[o]));
                    f1 = kReadScale * (d * F1[t][e]);
                    e1 = o < tok ? -bt * (d * E1[t][e]) : 0.0f;
                }
                if (o >= tok) {
                    const float d = expf(static_cast<float>(gs[o] - gt));
                    f2 = kReadScale * (d * F2[t][e]);
                    e2 = o > tok ? -vec[2 * kChunk + o] * (d * E2[t][e]) : 0.0f;
                }
                F1[t][e] = f1;
                F2[t][e] = f2;
                E1[t][e] = e1 + e2;
            }
        // per token: the sums over dv of its four lanes
        rd += __shfl_xor(rd, 16);
        rd += __shfl_xor(rd, 32);
        rv += __shfl_xor(rv, 16);
        rv += __shfl_xor(rv, 32);
        double gd = gm;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) gd += __shfl_xor(gd, d);
        if (g == 0) {
            dots[0][tok] = rd;
            dots[1][tok] = rv;
        }
        if (lane == 0) part[wave] = gd;
        __syncthreads();
        if (wave == 0) {
            const float beta = vec[2 * kChunk + lane];
            double od = 0.0, du = lane < 8 ? a.du[ph * 8 + lane] : 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) od += a.f.od[(ph * 8 + w) * kChunk + lane];
#pragma unroll
            for (int d = 1; d < 8; d *= 2) du += __shfl_xor(du, d);
            const double end = lane_of(du, 0) + static_cast<double>(vec[kChunk - 1]) * (part[0] + part[1] + part[2] + part[3]);
            double x = od - static_cast<double>(fabsf(beta) <= kLeastBeta ? 0.0f : beta) * dots[1][lane];
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const double y = __shfl_down(x, d);
                if (lane + d < 64) x += y;
            }
            if (lane < n) {
                a.dgate[(t0 + lane) * Hv + h] = static_cast<float>(x + end);
                a.dbeta[(t0 + lane) * Hv + h] = dots[0][lane] / beta;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = wave * 16 + 4 * g + e;
            const float rise = vec[i], fall = vec[kChunk + i], beta = vec[2 * kChunk + i];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                dq[t][e] = fmaf(kReadScale * rise, Z[t][e], dq[t][e]);
                dk[t][e] = fmaf(-beta * rise, Wm[t][e], fmaf(fall, H[t][e], dk[t][e]));
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u4 f1[NO], f2[NO], e1[NO];
            planes_of<NO>(F1[2 * half], F1[2 * half + 1], f1);
            planes_of<NO>(F2[2 * half], F2[2 * half + 1], f2);
            planes_of<NO>(E1[2 * half], E1[2 * half + 1], e1);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                u4 kc[NP], qc[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    kc[p] = plain_columns(lds + p * kPlaneBytes, half, t, r, g);
                    qc[p] = plain_columns(lds + (NP + p) * kPlaneBytes, half, t, r, g);
                }
                dq[t] = mma_planes<NO - 1>(f1, kc, dq[t]);
                dk[t] = mma_planes<NO - 1>(f2, qc, dk[t]);
                dk[t] = mma_planes<NO - 1>(e1, kc, dk[t]);
            }
        }
    }
    bits *qo = static_cast<bits *>(a.dq), *ko = static_cast<bits *>(a.dk);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = wave * 16 + 4 * g + e;
        if (i >= n) continue;
        const int64_t at = ((t0 + i) * Hk + kh) * kHeadDim + r;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            qo[at + 16 * t] = ET::put(dq[t][e]);
            ko[at + 16 * t] = ET::put(dk[t][e]);
        }
    }
}

// Waves a workgroup as in launch_walk.
template <typename ET, int NP, int W, int S>
hipError_t launch_back_of(const BackArgs &a, hipStream_t s) {
    const int parts = 8 / W;
    const int64_t wgs = static_cast<int64_t>(a.f.s.B) * a.f.s.Hv * parts;
    k_back<ET, NP, W, S><<<dim3(static_cast<unsigned>((wgs + 7) / 8 * 8)), dim3(64 * W), 0, s>>>(a, parts);
    return hipGetLastError();
}
template <typename ET, int NP, int S>
hipError_t launch_back(const BackArgs &a, hipStream_t s) {
    const int64_t heads = static_cast<int64_t>(a.f.s.B) * a.f.s.Hv;
    const int cus = device_cus();
    if (heads * 8 <= cus) return launch_back_of<ET, NP, 1, S>(a, s);
    if (heads * 4 <= cus) return launch_back_of<ET, NP, 2, S>(a, s);
    if (heads * 2 <= cus) return launch_back_of<ET, NP, 4, S>(a, s);
    return launch_back_of<ET, NP, 8, S>(a, s);
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
    k_grad<ET, NP, NO><<<dim3(static_cast<unsigned>(places)), dim3(256), 0, s>>>(a);
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
