// gdn_linear_f8.hip - gdn_linear_f8: e4m3 rows times e4m3 weights on the matrix
// cores, with a scale for each block of 128 k of a row and of 128 channels by 128
// k of the weights.
//
// Mathematics.  y[m][c] = sum over blocks b of a_scale[m][b] w_scale[c / 128][b]
// (sum_{k in b} a[m][k] w[c][k]) + bias[c].  A block's sum comes out of one matrix
// instruction of 16 x 16 x 128 and joins the running sum by one fused step with
// the product of the scales, in float32.
//
// The 8-bit instructions align the 32 products that they add at a time and drop
// what lies about 2^-16 below the largest (measured: 1.5e-5 of a sum of normally
// distributed codes, 5e-5 of random ones).  That is far below the rounding of
// 16-bit outputs (bf16 1.7e-3, fp16 2.1e-4), but not of float32 ones: for those
// (kWide) the codes are widened to fp16, which is exact, and multiplied by the fp16
// instructions, at half the rate (their sums are right to float32).
//
// Lane r + 16 g supplies 32 k of row r (channels from w as the first operand,
// tokens from a as the second): the chunks g and g + 4 of 16 bytes, in any order
// that both operands share; it receives channels 4 g..4 g+3 of token r.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_f8.hpp"
#include "gdn_launch.hpp"
#include "gdn_tile.hpp"

namespace gdn {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
struct Codes {                               // one lane's 32 codes of a row's block
    i4 lo, hi;
};
struct Halfs {                               // the same as fp16
    i4 x[4];
};

__device__ __forceinline__ f4 mul(const Codes &w, const Codes &x) {
    typedef int32_t i8 __attribute__((ext_vector_type(8)));
    const i8 a = {w.lo[0], w.lo[1], w.lo[2], w.lo[3], w.hi[0], w.hi[1], w.hi[2], w.hi[3]};
    const i8 b = {x.lo[0], x.lo[1], x.lo[2], x.lo[3], x.hi[0], x.hi[1], x.hi[2], x.hi[3]};
    constexpr int one = 0x7f7f7f7f;          // the instruction's own scales: 2^0
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f4{0, 0, 0, 0}, 0, 0, 0, one, 0, one);
}
__device__ __forceinline__ i4 widen(int a, int b) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return i4{__builtin_bit_cast(int, h2(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false))),
              __builtin_bit_cast(int, h2(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true))),
              __builtin_bit_cast(int, h2(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false))),
              __builtin_bit_cast(int, h2(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true)))};
}
__device__ __forceinline__ Halfs widen(const Codes &c) {
    return Halfs{{widen(c.lo[0], c.lo[1]), widen(c.lo[2], c.lo[3]), widen(c.hi[0], c.hi[1]), widen(c.hi[2], c.hi[3])}};
}
__device__ __forceinline__ f4 mul(const Halfs &w, const Halfs &x) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    f4 c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w.x[i]), __builtin_bit_cast(h8, x.x[i]), c, 0, 0, 0);
    return c;
}

// All TN x TM tiles of a wave over one block of k; s: the scales' product per token
// tile.
template <bool kWide, int TN, int TM>
__device__ __forceinline__ void mul_block(const Codes (&w)[TN], const Codes (&x)[TM], const float (&s)[TM], f4 (&acc)[TN][TM]) {
    if constexpr (kWide) {
        Halfs xh[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) xh[j] = widen(x[j]);
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const Halfs wh = widen(w[i]);
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const f4 p = mul(wh, xh[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s[j], acc[i][j][e]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const f4 p = mul(w[i], x[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s[j], acc[i][j][e]);
            }
    }
}

// Four consecutive channels c.. of token m.
template <typename OT>
__device__ __forceinline__ void put4(const LinearF8Args &a, int c, int m, f4 y) {
    typedef typename OT::bits bits;
    if (c >= a.N || m >= a.M) return;
    int first;
    const int s = group_of(a, c, first);
    const int n = a.end[s] - first;
    typename Pack<bits, 4>::vec v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = OT::put(y[i] + (a.bias ? a.bias[min(c + i, a.N - 1)] : 0.0f));
    if (c + 4 <= a.end[s]) {
        Pack<bits, 4>::store(static_cast<bits *>(a.out[s]) + static_cast<int64_t>(m) * n + c - first, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {                         // the four straddle a group's end
        const int s2 = group_of(a, c + i, first);
        if (c + i < a.N)
            static_cast<bits *>(a.out[s2])[static_cast<int64_t>(m) * (a.end[s2] - first) + c + i - first] = v[i];
    }
}
__device__ __forceinline__ void put4(const LinearF8Args &a, int c, int m, f4 y) {
    if (a.out_type == GDN_F32)
        put4<F32>(a, c, m, y);
    else if (a.out_type == GDN_BF16)
        put4<BF16>(a, c, m, y);
    else
        put4<F16>(a, c, m, y);
}

// The token scales of a wave's tiles, block by block.
template <int TM>
struct Scales {
    const float *p[TM];
    __device__ __forceinline__ Scales(const LinearF8Args &a, int m0, int blocks) {
        const int r = threadIdx.x & 15;
#pragma unroll
        for (int j = 0; j < TM; ++j) p[j] = a.a_scale + static_cast<int64_t>(min(m0 + 16 * j + r, a.M - 1)) * blocks;
    }
    __device__ __forceinline__ void at(int b, float sw, float (&s)[TM]) const {
#pragma unroll
        for (int j = 0; j < TM; ++j) s[j] = p[j][b] * sw;
    }
};

// ------------------------------------------------------------- split product
// For few tokens: a workgroup's WK waves share one tile of 16 TN channels x 16 TM
// tokens and split the blocks of k among them, each with a ring of S blocks of
// its own in LDS.  The partial sums meet in LDS.
template <int TN, int TM, int WK, int S, bool kVec, bool kWide>
__global__ __launch_bounds__(64 * WK) void k_f8_ring(LinearF8Args a, int tiles_n, int tiles_m) {
    constexpr int L = 2 * (TN + TM);
    constexpr int kPiece = L * 1024;
    static_assert(TN * TM * 1024 <= S * kPiece, "the sums fit a wave's ring");
    __shared__ alignas(1024) int8_t ring[WK][S][kPiece];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    int tn, tm;
    tile_of(blockIdx.x, tiles_n, tiles_m, tn, tm);
    if (tn >= tiles_n) return;
    const int c0 = tn * TN * 16, m0 = tm * TM * 16;
    const int blocks = (a.K + kBK - 1) / kBK;
    const int n = (blocks - wave + WK - 1) / WK;          // this wave's: wave, wave + WK, ..
    const int8_t *pw = a.w + static_cast<int64_t>(c0) * a.K, *px = a.a + static_cast<int64_t>(m0) * a.K;
    const int8_t *we = a.w + static_cast<int64_t>(a.N) * a.K, *xe = a.a + static_cast<int64_t>(a.M) * a.K;
    const uint32_t nw = span(a.N - c0, a.K), nx = span(a.M - m0, a.K);
    int off[L], at[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        int row = j * 8 + (lane >> 3) - (j < 2 * TN ? 0 : 16 * TN);
        at[j] = 16 * ((lane & 7) ^ swz(row));
        if (!kVec) row = min(row, j < 2 * TN ? a.N - 1 - c0 : a.M - 1 - m0);
        off[j] = row * a.K + (kVec ? at[j] : 0);
    }
    const int rd[2] = {r * kBK + 16 * (g ^ swz(r)), r * kBK + 16 * ((4 + g) ^ swz(r))};
    const Scales<TM> sc(a, m0, blocks);
    const float *sw = a.w_scale + static_cast<int64_t>(c0 / kF8Block) * blocks;
    f4 acc[TN][TM] = {};
    Codes w[TN], x[TM];
    auto read = [&](const int8_t *piece) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
            w[i] = Codes{*reinterpret_cast<const i4 *>(piece + i * 2048 + rd[0]), *reinterpret_cast<const i4 *>(piece + i * 2048 + rd[1])};
#pragma unroll
        for (int j = 0; j < TM; ++j)
            x[j] = Codes{*reinterpret_cast<const i4 *>(piece + (TN + j) * 2048 + rd[0]),
                         *reinterpret_cast<const i4 *>(piece + (TN + j) * 2048 + rd[1])};
    };
    // Codes past the last k are zero in both operands (a stray one could be a NaN).
    auto mask = [&](int left) {
        const bool lo = 16 * g < left, hi = 64 + 16 * g < left;
        const i4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < TN; ++i) w[i] = Codes{lo ? w[i].lo : zero, hi ? w[i].hi : zero};
#pragma unroll
        for (int j = 0; j < TM; ++j) x[j] = Codes{lo ? x[j].lo : zero, hi ? x[j].hi : zero};
    };
    float s[TM];
    if constexpr (kVec) {
        auto fetch = [&](int slot, int i) {               // past the end: the last block again
            const int k0 = (wave + min(i, n - 1) * WK) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j)
                fetch16(ring[wave][slot] + j * 1024, j < 2 * TN ? pw : px, j < 2 * TN ? nw : nx, off[j], k0);
        };
        auto step = [&](int slot, int i) {
            const int b = wave + i * WK;
            sc.at(b, sw[b], s);
            wait_mem<0, false>();
            read(ring[wave][slot]);
            wait_mem<63, true>();
            fetch(slot, i + S);
            if ((b + 1) * kBK > a.K) mask(a.K - b * kBK);
            mul_block<kWide>(w, x, s, acc);
        };
        if (n > 0) {
            for (int i = 0; i < S; ++i) fetch(i, i);
            for (int i = 0, slot = 0; i < n; ++i, slot = slot + 1 == S ? 0 : slot + 1) step(slot, i);
        }
        wait_mem<0, true>();
    } else {
        i4 v[L];
        auto load = [&](int i) {
            const int k0 = (wave + i * WK) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j)
                v[j] = (k0 + kBK <= a.K) ? any16((j < 2 * TN ? pw : px) + off[j] + k0 + at[j])
                                         : load16((j < 2 * TN ? pw : px) + off[j], k0 + at[j], a.K, j < 2 * TN ? we : xe);
        };
        if (n > 0) load(0);
        for (int i = 0; i < n; ++i) {
#pragma unroll
            for (int j = 0; j < L; ++j) *reinterpret_cast<i4 *>(ring[wave][0] + j * 1024 + lane * 16) = v[j];
            const int b = wave + i * WK;
            sc.at(b, sw[b], s);
            if (i + 1 < n) load(i + 1);
            read(ring[wave][0]);
            mul_block<kWide>(w, x, s, acc);
        }
    }
    // a wave's sums lie in its own ring, in its own lanes' order
    int8_t *const mine = ring[wave][0];
#pragma unroll
    for (int t = 0; t < TN * TM; ++t) *reinterpret_cast<f4 *>(mine + t * 1024 + lane * 16) = acc[t / TM][t % TM];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (TN * TM + WK - 1) / WK; ++i) {
        const int t = wave + i * WK;
        if (t >= TN * TM) break;
        f4 y = *reinterpret_cast<const f4 *>(ring[0][0] + t * 1024 + lane * 16);
#pragma unroll
        for (int k = 1; k < WK; ++k) y += *reinterpret_cast<const f4 *>(ring[k][0] + t * 1024 + lane * 16);
        put4(a, c0 + 16 * (t / TM) + 4 * g, m0 + 16 * (t % TM) + r, y);
    }
}

// ------------------------------------------------------- one tile a workgroup
// BN channels x BM tokens a workgroup, its waves in a WN x WM grid over them, a ring
// of S blocks in LDS.  While a block is multiplied the next one is read from
// LDS; one barrier a block hands its buffer back to the fetches.
template <typename OT, int BN, int BM, int WN, int WM, int S, bool kVec, bool kWide>
__global__ __launch_bounds__(64 * WN * WM) void k_f8_block(LinearF8Args a, int tiles_n, int tiles_m) {
    constexpr int NW = WN * WM;
    constexpr int TN = BN / WN / 16, TM = BM / WM / 16;
    constexpr int L = (BN + BM) / 8 / NW, LN = BN / 8 / NW;
    constexpr int kBytes = (BN + BM) * kBK;
    static_assert(kF8Block % (16 * TN) == 0, "a wave's channels share a scale");
    __shared__ alignas(1024) int8_t ring[S][kBytes];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;
    int tn, tm;
    tile_of(blockIdx.x, tiles_n, tiles_m, tn, tm);
    if (tn >= tiles_n) return;
    const int c0 = tn * BN, m0 = tm * BM;
    const int blocks = (a.K + kBK - 1) / kBK;
    const int8_t *pw = a.w + static_cast<int64_t>(c0) * a.K, *px = a.a + static_cast<int64_t>(m0) * a.K;
    const int8_t *we = a.w + static_cast<int64_t>(a.N) * a.K, *xe = a.a + static_cast<int64_t>(a.M) * a.K;
    const uint32_t nw = span(a.N - c0, a.K), nx = span(a.M - m0, a.K);
    int off[L], at[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        int row = ((j < LN ? j : j - LN) * NW + wave) * 8 + (lane >> 3);
        at[j] = 16 * ((lane & 7) ^ swz(row));
        if (!kVec) row = min(row, j < LN ? a.N - 1 - c0 : a.M - 1 - m0);
        off[j] = row * a.K + (kVec ? at[j] : 0);
    }
    // piece j of this wave in a buffer
    auto piece = [&](int j) { return (j < LN ? 0 : BN * kBK) + ((j < LN ? j : j - LN) * NW + wave) * 1024; };
    const int rd[2] = {r * kBK + 16 * (g ^ swz(r)), r * kBK + 16 * ((4 + g) ^ swz(r))};
    const int cw = c0 + wn * TN * 16, mw = m0 + wm * TM * 16;
    const Scales<TM> sc(a, mw, blocks);
    // (a tile's last waves may lie past the last channel)
    const float *sw = a.w_scale + static_cast<int64_t>(min(cw, a.N - 1) / kF8Block) * blocks;
    f4 acc[TN][TM] = {};
    auto read = [&](const int8_t *buf, int b, Codes (&w)[TN], Codes (&x)[TM], float (&s)[TM]) {
        sc.at(b, sw[b], s);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int8_t *p = buf + (BN + (wm * TM + j) * 16) * kBK;
            x[j] = Codes{*reinterpret_cast<const i4 *>(p + rd[0]), *reinterpret_cast<const i4 *>(p + rd[1])};
        }
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int8_t *p = buf + (wn * TN + i) * 16 * kBK;
            w[i] = Codes{*reinterpret_cast<const i4 *>(p + rd[0]), *reinterpret_cast<const i4 *>(p + rd[1])};
        }
        if (kVec && (b + 1) * kBK > a.K) {                // zeros past the last k, in both operands
            const int left = a.K - b * kBK;
            const bool lo = 16 * g < left, hi = 64 + 16 * g < left;
            const i4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < TN; ++i) w[i] = Codes{lo ? w[i].lo : zero, hi ? w[i].hi : zero};
#pragma unroll
            for (int j = 0; j < TM; ++j) x[j] = Codes{lo ? x[j].lo : zero, hi ? x[j].hi : zero};
        }
    };
    i4 v[kVec ? 1 : L];
    auto load = [&](int b) {                              // past the end: the last block again
        const int k0 = min(b, blocks - 1) * kBK;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int8_t *row = (j < LN ? pw : px) + off[j];
            v[kVec ? 0 : j] = k0 + kBK <= a.K ? any16(row + k0 + at[j]) : load16(row, k0 + at[j], a.K, j < LN ? we : xe);
        }
    };
    // block b on its way to its buffer; without 16-byte rows it waits in registers
    auto fetch = [&](int8_t *buf, int b) {
        if constexpr (kVec) {
            const int k0 = min(b, blocks - 1) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j) fetch16(buf + piece(j), j < LN ? pw : px, j < LN ? nw : nx, off[j], k0);
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) *reinterpret_cast<i4 *>(buf + piece(j) + lane * 16) = v[j];
            load(b + 1);
        }
    };
    Codes w0[TN], x0[TM], w1[TN], x1[TM];
    float s0[TM], s1[TM];
    if (!kVec) load(0);
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(ring[i], i);
    wait_mem<0, true>();
    barrier();
    read(ring[0], 0, w0, x0, s0);
    int slot = 0;
    for (int b = 0; b < blocks; b += 2) {
        int next = slot + 1 == S ? 0 : slot + 1;
        wait_mem<kVec ? (S - 2) * L : 0, true>();         // block b + 1 has landed, block b is read
        barrier();
        if (b + 1 < blocks) read(ring[next], b + 1, w1, x1, s1);
        fetch(ring[slot], b + S);
        mul_block<kWide>(w0, x0, s0, acc);
        if (b + 1 >= blocks) break;
        slot = next;
        next = slot + 1 == S ? 0 : slot + 1;
        wait_mem<kVec ? (S - 2) * L : 0, true>();
        barrier();
        if (b + 2 < blocks) read(ring[next], b + 2, w0, x0, s0);
        fetch(ring[slot], b + 1 + S);
        mul_block<kWide>(w1, x1, s1, acc);
        slot = next;
    }
    wait_mem<0, true>();                                  // nothing lands in LDS after the end
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) put4<OT>(a, cw + 16 * i + 4 * g, mw + 16 * j + r, acc[i][j]);
}

// ------------------------------------------------------------------- dispatch
template <typename OT, int TN, int TM, int WK, int S>
hipError_t launch_ring(const LinearF8Args &a, hipStream_t s) {
    constexpr bool kWide = __is_same(OT, F32);
    const int tn = static_cast<int>(tiles(a.N, 16 * TN)), tm = static_cast<int>(tiles(a.M, 16 * TM));
    if (a.K % 16 == 0)
        k_f8_ring<TN, TM, WK, S, true, kWide><<<tile_grid(tn, tm), dim3(64 * WK), 0, s>>>(a, tn, tm);
    else
        k_f8_ring<TN, TM, WK, S, false, kWide><<<tile_grid(tn, tm), dim3(64 * WK), 0, s>>>(a, tn, tm);
    return hipGetLastError();
}

template <typename OT, int BN, int BM, int WN, int WM, int S>
hipError_t launch_block(const LinearF8Args &a, hipStream_t s) {
    constexpr bool kWide = __is_same(OT, F32);
    const int tn = static_cast<int>(tiles(a.N, BN)), tm = static_cast<int>(tiles(a.M, BM));
    const dim3 block(64 * WN * WM);
    if (a.K % 16 == 0)
        k_f8_block<OT, BN, BM, WN, WM, S, true, kWide><<<tile_grid(tn, tm), block, 0, s>>>(a, tn, tm);
    else
        k_f8_block<OT, BN, BM, WN, WM, 2, false, kWide><<<tile_grid(tn, tm), block, 0, s>>>(a, tn, tm);
    return hipGetLastError();
}

template <typename OT>
hipError_t launch(const LinearF8Args &a, hipStream_t s) {
    const int cus = device_cus();
    const auto fits = [&](int bn, int bm) {
        return (bn <= 64 || bn < 2 * a.N) && (bm <= 16 || bm < 2 * a.M) &&
               2 * tiles(a.N, bn) * tiles(a.M, bm) > static_cast<int64_t>(cus);
    };
    if (fits(256, 128)) return launch_block<OT, 256, 128, 4, 2, 3>(a, s);
    if (fits(128, 128)) return launch_block<OT, 128, 128, 2, 4, 4>(a, s);
    if (fits(64, 128)) return launch_block<OT, 64, 128, 2, 2, 4>(a, s);
    if (fits(64, 64)) return launch_ring<OT, 4, 4, 4, 2>(a, s);
    if (fits(32, 64)) return launch_ring<OT, 2, 4, 4, 3>(a, s);
    if (fits(64, 32)) return launch_ring<OT, 4, 2, 4, 3>(a, s);
    if (fits(32, 32)) return launch_ring<OT, 2, 2, 4, 4>(a, s);
    if (fits(64, 16)) return launch_ring<OT, 4, 1, 4, 3>(a, s);
    return launch_ring<OT, 1, 1, 8, 2>(a, s);
}

}  // namespace

hipError_t launch_linear_f8(const LinearF8Args &a, hipStream_t s) {
    switch (a.out_type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
