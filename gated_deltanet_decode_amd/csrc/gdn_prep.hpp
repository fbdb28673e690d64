// gdn_prep.hpp - k_prep, the part of the delta rule in chunks that no state
// enters: one launch over all chunks, shared by the forward and backward pass.
// Included by kernel sources only.
//
// With g the running sum of the gates in a chunk (g_i - g_j is the log decay
// from token j to token i), for j <= i < 64:
//   A_ij = beta_i exp(g_i - g_j) k_i . k_j  (j < i),    T = (I + A)^-1,
//   P_ij = exp(g_i - g_j) q_i . k_j / sqrt(128).
// The differences are formed in binary64, so that a token with a strong decay
// costs the later ones no accuracy.  T is formed by blocks of 16: the diagonal
// ones by substitution, a column a lane, the others from them by float32
// matrix products, column of blocks by column.
//
// The vector units bound it (exponentials, cutting results into planes, the 16
// dependent steps of a substitution), then the 33 KB that it writes a chunk and value
// head: 8 x 4096 tokens bf16, 32 value heads, 162 us, 3.4 TB/s of blocks; the 4 chunks of
// 200 tokens 10 us.  T in float32, cut by each workgroup of the walk: the walk 10 %
// slower.
#pragma once

#include <hip/hip_runtime.h>

#include "gdn_elem.hpp"
#include "gdn_mma.hpp"
#include "gdn_packed.hpp"

namespace gdn {
namespace {

constexpr float kReadScale = 0.08838834764831845f;   // 1 / sqrt(128)

// The gates are summed as powers of two.  2^x by its whole and its broken part, so that
// a strong decay is right to float32 too; the hardware's exponential is right to one
// unit in the last place.
constexpr double kLog2e = 1.44269504088896340736;
__device__ __forceinline__ float exp_2(double x) {
    const double n = floor(x);        // (x less its fraction may lie just beside a whole number)
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(static_cast<float>(x - n)), static_cast<int>(n));
}

struct PrepArgs {
    Packed s;
    const void *q;
    const void *k;
    const float *beta;
    const float *gate;
    char *within;                    // a block per chunk place and value head
    char *kq;
    // the backward pass alone
    char *back;                      // the same with T and P transposed
    double *gsum;
};

// A row of a plane is 16 chunks of 16 bytes; chunk c of row r lies at slot c ^ turn(r).
// Sixteen rows at a chunk and four neighbouring rows at four neighbouring chunks
// (read_columns) both spread over all banks.
__device__ __forceinline__ int turn(int row) { return (row & 3) << 2 | (row >> 2 & 3); }
__device__ __forceinline__ int plane_at(int row, int chunk) { return row * 256 + ((chunk ^ turn(row)) << 4); }

constexpr int kABlocks = 10;
constexpr int block_of(int it, int jt) { return it * (it + 1) / 2 + jt; }
// Operand of 16 tokens it x 32 tokens of half h.
constexpr int pblock_of(int it, int h) { return it < 2 ? it : 2 + (it - 2) * 2 + h; }

// Transposed: operand of 16 tokens jt x the 32 tokens of half h, h >= jt / 2.
constexpr int pnblock_of(int jt, int h) { return jt < 2 ? jt * 2 + h : 4 + (jt - 2); }

// Eight elements from p as planes.
template <typename ET, int NP>
__device__ __forceinline__ void load_planes(const void *base, int64_t at, u4 (&p)[NP]) {
    typedef typename ET::bits bits;
    const bits *src = static_cast<const bits *>(base) + at;
    if constexpr (NP == 1) {
        p[0] = *reinterpret_cast<const u4 *>(src);
    } else {
        f4 x, y;
        const auto v = Pack<bits, 8>::load(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = ET::get(v[i]);
            y[i] = ET::get(v[4 + i]);
        }
        planes_of<NP>(x, y, p);
    }
}

// The log decay from j to i may pass any number of gates; one of less than -2^14
// counts as -2^14: no run of gates that float32 can raise again makes up for it
// (exp of either is 0), and sums stay finite.
__device__ __forceinline__ double gate_of(float x) { return x < -16384.0f ? -16384.0 : static_cast<double>(x); }

// The backward pass divides corrections by beta; one of (nearly) 0 counts there as
// 2^-60, whose corrections are below any rounding.
constexpr float kLeastBeta = 0x1p-60f;
template <bool kBack>
__device__ __forceinline__ float beta_of(float x) {
    return kBack && fabsf(x) < kLeastBeta ? kLeastBeta : x;
}

// One workgroup of four waves per chunk place and key head; wave w has the 16
// tokens w of the chunk as its rows.  The value heads of the key head go through
// two at a time.
template <typename ET, int NP, int NO, bool kBack>
__global__ __launch_bounds__(256, NP == 3 ? 1 : NP == 2 ? 2 : kBack ? 3 : 4) void k_prep(PrepArgs a) {
    constexpr int HB = 2;
    constexpr int kBlock = within_bytes(NO), kBackBlock = within_bytes(3);
    // the planes of k and q; after their products A's blocks and T's diagonal ones
    __shared__ alignas(16) char lds[2 * NP * kPlaneBytes];
    char (*const kp)[kPlaneBytes] = reinterpret_cast<char (*)[kPlaneBytes]>(lds), (*const qp)[kPlaneBytes] = kp + NP;
    float (*const As)[kABlocks][256] = reinterpret_cast<float (*)[kABlocks][256]>(lds);
    float (*const Td)[4][256] = reinterpret_cast<float (*)[4][256]>(lds + HB * kABlocks * 1024);
    static_assert(HB * (kABlocks * 1024 + 4096) <= sizeof(lds), "");
    __shared__ double gs[HB][kChunk];
    __shared__ float bs[HB][kChunk];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int place = blockIdx.x / a.s.Hk, kh = blockIdx.x - place * a.s.Hk;
    const int b = sequence_at(a.s, place);
    const Span sp = span_of(a.s, b);
    const int c0 = (place - place_of(sp.first, b)) * kChunk;
    if (c0 < 0 || c0 >= sp.len || slot_of(a.s, b) < 0) return;
    const int n = min(kChunk, sp.len - c0);            // tokens of this chunk
    const int64_t t0 = sp.first + c0;

    // rows past the last token are zero
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = i * 256 + threadIdx.x, row = at >> 4, chunk = at & 15;
        u4 pk[NP] = {}, pq[NP] = {};
        if (row < n) {
            const int64_t src = ((t0 + row) * a.s.Hk + kh) * kHeadDim + chunk * 8;
            load_planes<ET, NP>(a.k, src, pk);
            load_planes<ET, NP>(a.q, src, pq);
        }
        const int dst = plane_at(row, chunk);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            *reinterpret_cast<u4 *>(kp[p] + dst) = pk[p];
            *reinterpret_cast<u4 *>(qp[p] + dst) = pq[p];
        }
        if constexpr (NP > 1) {
            char *to = a.kq + (static_cast<int64_t>(place) * a.s.Hk + kh) * (2 * NP * kPlaneBytes) + dst;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                *reinterpret_cast<u4 *>(to + p * kPlaneBytes) = pk[p];
                *reinterpret_cast<u4 *>(to + (NP + p) * kPlaneBytes) = pq[p];
            }
        }
    }
    __syncthreads();
    // k_i . k_j and q_i . k_j: lane r has token i = 16 wave + r, elements j = 16 jt + 4 g..
    f4 kk[4] = {}, qk[4] = {}, kq[4] = {};                // kq: lane r token j, elements i
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
        u4 ki[NP], qi[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int at = plane_at(wave * 16 + r, 4 * jj + g);
            ki[p] = *reinterpret_cast<const u4 *>(kp[p] + at);
            qi[p] = *reinterpret_cast<const u4 *>(qp[p] + at);
        }
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
            if (jt <= wave) {
                u4 kj[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    kj[p] = *reinterpret_cast<const u4 *>(kp[p] + plane_at(jt * 16 + r, 4 * jj + g));
                kk[jt] = mma_planes<2>(kj, ki, kk[jt]);
                qk[jt] = mma_planes<2>(kj, qi, qk[jt]);
                if constexpr (kBack) kq[jt] = mma_planes<2>(qi, kj, kq[jt]);
            }
    }
    const int group = a.s.Hv / a.s.Hk;
    for (int h0 = 0; h0 < group; h0 += HB) {
        __syncthreads();                                // the planes, the last heads' columns are read
        if (wave < HB && h0 + wave < group) {           // running sums of the gates
            const int h = kh + (h0 + wave) * a.s.Hk;
            const int64_t at = (t0 + lane) * a.s.Hv + h;
            const float beta = lane < n ? beta_of<kBack>(a.beta[at]) : 0.0f;
            double x = lane < n ? gate_of(a.gate[at]) * kLog2e : 0.0;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const double y = __shfl_up(x, d);
                if (lane >= d) x += y;
            }
            gs[wave][lane] = x;
            bs[wave][lane] = beta;
            const double last = lane_of(x, 63);
            const int64_t ph = static_cast<int64_t>(place) * a.s.Hv + h;
            const auto put = [&](char *block) {
                float *vec = reinterpret_cast<float *>(block);
                vec[lane] = exp_2(x);
                vec[kChunk + lane] = exp_2(last - x);
                vec[2 * kChunk + lane] = beta;
            };
            put(a.within + ph * kBlock + kBlock - 1024);
            if constexpr (kBack) {
                put(a.back + ph * kBackBlock + kBackBlock - 1024);
                a.gsum[ph * kChunk + lane] = x;
            }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < HB; ++x) {
            if (h0 + x >= group) break;
            const int h = kh + (h0 + x) * a.s.Hk;
            const int64_t ph = static_cast<int64_t>(place) * a.s.Hv + h;
            const int i = wave * 16 + r;
            const double gi = gs[x][i];
            const float bi = bs[x][i];
            f4 pv[4] = {};
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
                if (jt <= wave) {
                    f4 av;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = jt * 16 + 4 * g + e;
                        const float d = exp_2(gi - gs[x][j]);
                        av[e] = j < i ? bi * (d * kk[jt][e]) : 0.0f;
                        pv[jt][e] = j <= i ? kReadScale * (d * qk[jt][e]) : 0.0f;
                    }
                    *reinterpret_cast<f4 *>(&As[x][block_of(wave, jt)][r * 16 + 4 * g]) = av;
                }
            char *P = a.within + ph * kBlock + kTBytes + lane * 16;
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half <= wave / 2) {
                    u4 p[NO];
                    planes_of<NO>(pv[2 * half], pv[2 * half + 1], p);
#pragma unroll
                    for (int m = 0; m < NO; ++m)
                        *reinterpret_cast<u4 *>(P + (m * kPBlocks + pblock_of(wave, half)) * 1024) = p[m];
                }
            if constexpr (kBack) {
                // operand (jt, half): lane r token j, eight tokens i of the tiles 2 half
                // and 2 half + 1; this wave's four of them.  Operands whose tiles lie
                // all above the diagonal do not exist.
                char *Pn = a.back + ph * kBackBlock + kTBytes + lane * 16 + 8 * (wave & 1);
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) {
                    if (jt / 2 > wave / 2) continue;
                    f4 pv = {0, 0, 0, 0};
                    if (jt <= wave) {
                        const int j = jt * 16 + r;
                        const double gj = gs[x][j];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = wave * 16 + 4 * g + e;
                            const float d = exp_2(gs[x][i] - gj);
                            pv[e] = j <= i ? kReadScale * (d * kq[jt][e]) : 0.0f;
                        }
                    }
                    u4 p[3];
                    planes_of<3>(pv, pv, p);
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        *reinterpret_cast<u2 *>(Pn + (m * kPBlocks + pnblock_of(jt, wave / 2)) * 1024) = u2{p[m].x, p[m].y};
                }
            }
        }
        __syncthreads();
        if (wave < HB && h0 + wave < group) {           // column r of diagonal block g
            const float *A = As[wave][block_of(g, g)];
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == r ? 1.0f : 0.0f;
#pragma unroll
                for (int j = 0; j < i; ++j) s = fmaf(-A[i * 16 + j], x[j], s);
                x[i] = s;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) Td[wave][g][i * 16 + r] = x[i];
        }
        __syncthreads();
        // Columns of blocks: wave 0 and 1 have the first of a head each, 2 and 3 the
        // other three.
        const int x = wave % HB;
        if (h0 + x < group) {
            const int h = kh + (h0 + x) * a.s.Hk;
            const int64_t ph = static_cast<int64_t>(place) * a.s.Hv + h;
            char *const T = a.within + ph * kBlock + lane * 16;
            // rows: T_ij with lane r row r, elements columns 4 g..: the half (j & 1) of an
            // operand of row tile i
            const auto put_rows = [&](int i, int j, f4 rows) {
                u4 p[3];
                planes_of<3>(rows, rows, p);
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    *reinterpret_cast<u2 *>(T + (m * kPBlocks + pblock_of(i, j / 2)) * 1024 + 8 * (j & 1)) = u2{p[m].x, p[m].y};
            };
            const int j0 = wave < HB ? 0 : 1, j1 = wave < HB ? 1 : 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j < j0 || j >= j1) continue;
                f4 col[4] = {};                         // T_ij, lane r column r, rows 4 g..
#pragma unroll
                for (int e = 0; e < 4; ++e) col[j][e] = Td[x][j][(4 * g + e) * 16 + r];
                put_rows(j, j, *reinterpret_cast<const f4 *>(&Td[x][j][r * 16 + 4 * g]));
                if (j & 1) put_rows(j - 1, j, f4{0, 0, 0, 0});
#pragma unroll
                for (int i = j + 1; i < 4; ++i) {
                    f4 s = {0, 0, 0, 0};
#pragma unroll
                    for (int m = j; m < i; ++m)
                        s = mma32(*reinterpret_cast<const f4 *>(&As[x][block_of(i, m)][r * 16 + 4 * g]), col[m], s);
                    s = -s;
                    const f4 diag = *reinterpret_cast<const f4 *>(&Td[x][i][r * 16 + 4 * g]);
                    col[i] = mma32(diag, s, f4{0, 0, 0, 0});
                    put_rows(i, j, mma32(s, diag, f4{0, 0, 0, 0}));
                }
                if constexpr (kBack) {
                    char *const Tn = a.back + ph * kBackBlock + lane * 16;
#pragma unroll
                    for (int half = j / 2; half < 2; ++half) {
                        u4 p[3];
                        planes_of<3>(col[2 * half], col[2 * half + 1], p);
#pragma unroll
                        for (int m = 0; m < 3; ++m)
                            *reinterpret_cast<u4 *>(Tn + (m * kPBlocks + pnblock_of(j, half)) * 1024) = p[m];
                    }
                }
            }
        }
    }
}

template <typename ET, int NP, int NO, bool kBack>
hipError_t launch_prep(const PrepArgs &a, hipStream_t s) {
    const int64_t wgs = chunk_places(a.s.B, a.s.tokens) * a.s.Hk;
    k_prep<ET, NP, NO, kBack><<<dim3(static_cast<unsigned>(wgs)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace gdn
