// gdn_linear.hip - gdn_linear_q8: int8 rows times int8 weights on the matrix
// cores, scaled by row and channel and written to up to four output tensors.
//
// Mathematics.  y[m][c] = (sum_k a[m][k] w[c][k]) a_scale[m] w_scale[c] + bias[c].
// The integer sum is exact in 32 bits, so neither the order of k nor a split
// of it over waves changes a result: every kernel here gives the same bits.
//
// Matrix instructions of 16 x 16 x 64: lane r + 16 g supplies 16 consecutive k
// of row r (channels from w as the first operand, tokens from a as the second)
// and receives channels 4 g..4 g+3 of token r.
//
// Kernels, by how many tiles the product has (launch() says which):
//   k_linear_ring   a workgroup's waves split k over one small tile
//   k_linear_block  one tile a workgroup, its waves share the operands in LDS
//   k_linear_tile   persistent workgroups over 256 x 256 tiles
// All of them move 128-byte lines into LDS eight rows at a time.  Loads in the
// operands' own shape (sixteen rows, 64 bytes of each) cost the vector cache a
// cycle per row and were half as fast from 64 tokens on.
#include "gdn.h"
#include "gdn_elem.hpp"
#include "gdn_launch.hpp"
#include "gdn_serve.hpp"
#include "gdn_tile.hpp"

namespace gdn {
namespace {

// ------------------------------------------------------------------- results
// Four consecutive channels c.. that a lane scales and writes.
struct Channels {
    void *out;          // the first's group, its first row at channel c
    int32_t n;          // channels of that group (a row's length)
    int32_t live;       // how many of the four belong to it
    float scale[4], bias[4];

    Channels() = default;
    __device__ __forceinline__ Channels(const LinearArgs &a, int c, size_t bytes) {
        int first;
        const int s = group_of(a, c, first);
        n = a.end[s] - first;
        live = max(0, min(4, a.end[s] - c));
        out = static_cast<char *>(a.out[s]) + (c - first) * bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = min(c + i, a.N - 1);
            scale[i] = a.w_scale[ch];
            bias[i] = a.bias ? a.bias[ch] : 0.0f;
        }
    }
};

// The scaled sum: the integer and the two products each round to binary32, the
// last together with the bias.
__device__ __forceinline__ float scaled(int32_t acc, float sa, float sw, float bias) {
    return fmaf(static_cast<float>(acc) * sa, sw, bias);
}

// Writes four consecutive channels of token m, whose scale is sa.
template <typename OT>
__device__ __forceinline__ void put4(const LinearArgs &a, const Channels &ch, int c, int m, float sa,
                                     i4 acc) {
    typedef typename OT::bits bits;
    typename Pack<bits, 4>::vec v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = OT::put(scaled(acc[i], sa, ch.scale[i], ch.bias[i]));
    bits *p = static_cast<bits *>(ch.out) + static_cast<int64_t>(m) * ch.n;
    if (ch.live == 4) {
        Pack<bits, 4>::store(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {                         // the four straddle a group's end
        int first;
        const int s = group_of(a, c + i, first);
        if (c + i < a.N)
            static_cast<bits *>(a.out[s])[static_cast<int64_t>(m) * (a.end[s] - first) + c + i - first] =
                v[i];
    }
}

__device__ __forceinline__ int type_bytes(const LinearArgs &a) { return a.out_type == GDN_F32 ? 4 : 2; }
__device__ __forceinline__ void put4(const LinearArgs &a, const Channels &ch, int c, int m, float sa,
                                     i4 acc) {
    if (a.out_type == GDN_F32)
        put4<F32>(a, ch, c, m, sa, acc);
    else if (a.out_type == GDN_BF16)
        put4<BF16>(a, ch, c, m, sa, acc);
    else
        put4<F16>(a, ch, c, m, sa, acc);
}

// Writes a wave's TN x TM matrix tiles.  Where all its channels belong to one
// group they pass through the wave's own piece of LDS, so that a store covers
// whole lines of a token's row instead of 8 or 16 bytes of sixteen rows
// (256 x 256 tiles at 32768 tokens x 12352 channels, k = 2048, bf16: 0.88 ms
// against 1.20).
constexpr int kStageBytes = 4096;
template <typename OT, int TN, int TM>
__device__ __forceinline__ void write_tile(const LinearArgs &a, int c0, int m0, int lane, int8_t *stage,
                                           const i4 (&acc)[TN][TM]) {
    typedef typename OT::bits bits;
    typedef float f4 __attribute__((ext_vector_type(4)));
    const int r = lane & 15, g = lane >> 4;
    int first;
    const int s = group_of(a, c0, first);
    float sa[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) sa[j] = a.a_scale[min(m0 + j * 16 + r, a.M - 1)];
    if (c0 + TN * 16 > a.end[s]) {                        // several groups, or the last channels
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int c = c0 + i * 16 + 4 * g;
            if (c < a.N) {
                const Channels ch(a, c, sizeof(bits));
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    if (m0 + j * 16 + r < a.M) put4<OT>(a, ch, c, m0 + j * 16 + r, sa[j], acc[i][j]);
            }
        }
        return;
    }
    const int n = a.end[s] - first;
    bits *out = static_cast<bits *>(a.out[s]) + static_cast<int64_t>(m0) * n + (c0 - first);
    f4 sw[TN], bias[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        sw[i] = Pack<float, 4>::load(a.w_scale + c0 + i * 16 + 4 * g);
        bias[i] = a.bias ? Pack<float, 4>::load(a.bias + c0 + i * 16 + 4 * g) : f4{0, 0, 0, 0};
    }
    constexpr int kRow = TN * 16 * sizeof(bits);          // bytes of a token's channels
    constexpr int kTok = 16 * kRow <= kStageBytes / 2 && TM % 2 == 0 ? 2 : 1;
    constexpr int kLanes = kRow / 16;                     // lanes that store a token's row
    static_assert(16 * kRow * kTok <= kStageBytes && (kLanes & (kLanes - 1)) == 0 && kLanes >= 4, "stage");
    // chunk c (16 bytes) of row i lies at c ^ (i modulo the chunks)
#pragma unroll
    for (int j0 = 0; j0 < TM; j0 += kTok) {
#pragma unroll
        for (int j = 0; j < kTok; ++j)
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                typename Pack<bits, 4>::vec v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = OT::put(scaled(acc[i][j0 + j][e], sa[j0 + j], sw[i][e], bias[i][e]));
                const int at = (i * 16 + 4 * g) * sizeof(bits);
                *reinterpret_cast<typename Pack<bits, 4>::vec *>(
                    stage + (j * 16 + r) * kRow + (((at >> 4) ^ (r & (kLanes - 1))) << 4) + (at & 15)) = v;
            }
#pragma unroll
        for (int p = 0; p < 16 * kTok * kLanes / 64; ++p) {
            const int row = p * (64 / kLanes) + lane / kLanes, col = lane % kLanes;
            const i4 v = *reinterpret_cast<const i4 *>(stage + row * kRow + 16 * (col ^ (row & (kLanes - 1))));
            const int m = j0 * 16 + row;
            if (m0 + m < a.M)
                Pack<bits, 16 / sizeof(bits)>::store(
                    out + static_cast<int64_t>(m) * n + col * (16 / sizeof(bits)),
                    __builtin_bit_cast(typename Pack<bits, 16 / sizeof(bits)>::vec, v));
        }
    }
}

// ------------------------------------------------------------- split product
// For few tokens, where the weights' bytes or the latency of a long k bound the
// product: a workgroup's WK waves share one tile of 16 TN channels x 16 TM
// tokens and split k among them in blocks.  Each wave has a ring of S blocks of
// its own in LDS (no barrier, only its own counter); the partial sums meet in
// LDS.  kVec: rows are 16-byte aligned and go straight to LDS; others pass
// through registers, one block ahead, into a single piece.
template <int TN, int TM, int WK, int S, bool kVec>
__global__ __launch_bounds__(64 * WK) void k_linear_ring(LinearArgs a, int tiles_n, int tiles_m) {
    constexpr int L = 2 * (TN + TM);                      // fetches of a block, 8 rows each
    constexpr int kPiece = L * 1024;
    static_assert(S >= 2 && S <= 4 && (S - 1) * L < 60, "");
    __shared__ alignas(1024) int8_t r0[WK * kPiece], r1[WK * kPiece], r2[kVec && S > 2 ? WK * kPiece : 16],
        r3[kVec && S > 3 ? WK * kPiece : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    int tn, tm;
    tile_of(blockIdx.x, tiles_n, tiles_m, tn, tm);
    if (tn >= tiles_n) return;
    const int c0 = tn * TN * 16, m0 = tm * TM * 16;

    // what the wave scales and writes in the end, fetched while the sums run
    const int mine = min(wave, TN * TM - 1);
    const int c = c0 + 16 * (mine / TM) + 4 * g, m = m0 + 16 * (mine % TM) + r;
    const Channels ch(a, min(c, a.N - 1), type_bytes(a));
    const float sa = a.a_scale[min(m, a.M - 1)];

    const int full = a.K / kBK;                           // whole blocks
    const int n = (full - wave + WK - 1) / WK;            // this wave's: wave, wave + WK, ..
    const int8_t *pw = a.w + static_cast<int64_t>(c0) * a.K, *px = a.a + static_cast<int64_t>(m0) * a.K;
    const uint32_t nw = span(a.N - c0, a.K), nx = span(a.M - m0, a.K);
    int off[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        int row = j * 8 + (lane >> 3) - (j < 2 * TN ? 0 : 16 * TN);
        const int slot = 16 * ((lane & 7) ^ swz(row));
        // a load to registers stays in the matrix: rows past the last are the last
        if (!kVec) row = min(row, j < 2 * TN ? a.N - 1 - c0 : a.M - 1 - m0);
        off[j] = row * a.K + slot;
    }
    const int rd[2] = {r * kBK + 16 * (g ^ swz(r)), r * kBK + 16 * ((4 + g) ^ swz(r))};
    i4 acc[TN][TM] = {};
    i4 wf[2][TN], xf[2][TM];
    auto read = [&](const int8_t *piece) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < TN; ++i) wf[h][i] = *reinterpret_cast<const i4 *>(piece + i * 2048 + rd[h]);
#pragma unroll
            for (int j = 0; j < TM; ++j)
                xf[h][j] = *reinterpret_cast<const i4 *>(piece + (TN + j) * 2048 + rd[h]);
        }
    };
    // Weights past the last k are zero; `left` of k from this lane's chunk on.
    auto mask = [&](int left) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TN; ++i) wf[h][i] = 64 * h < left ? wf[h][i] : i4{0, 0, 0, 0};
    };
    auto mul = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[h][i], xf[h][j], acc[i][j], 0, 0, 0);
    };
    int8_t *const p0 = r0 + wave * kPiece, *const p1 = r1 + wave * kPiece;
    if constexpr (kVec) {
        int8_t *const p2 = S > 2 ? r2 + wave * kPiece : nullptr, *const p3 = S > 3 ? r3 + wave * kPiece : nullptr;
        // the block past the whole ones, if there is one and it is this wave's
        const bool part = full * kBK < a.K && wave == full % WK;
        const int all = n + (part ? 1 : 0);
        auto fetch = [&](int8_t *piece, int i) {          // past the end: the last block again
            const int k0 = (wave + min(i, all - 1) * WK) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j)
                fetch16(piece + j * 1024, j < 2 * TN ? pw : px, j < 2 * TN ? nw : nx, off[j], k0);
        };
        auto step = [&](int8_t *piece, int i) {
            wait_mem<(S - 1) * L, false>();               // block i has landed
            read(piece);
            wait_mem<63, true>();                         // and is in registers: its piece is free
            fetch(piece, i + S);
            mul();
        };
        if (all > 0) {
            fetch(p0, 0);
            fetch(p1, 1);
            if constexpr (S > 2) fetch(p2, 2);
            if constexpr (S > 3) fetch(p3, 3);
            // whole rounds of the ring, then what is left (a branch out of a round
            // would make the compiler wait for every fetch where the paths meet)
            int i = 0;
            for (; i + S <= n; i += S) {
                step(p0, i);
                step(p1, i + 1);
                if constexpr (S > 2) step(p2, i + 2);
                if constexpr (S > 3) step(p3, i + 3);
            }
            if (i < n) {
                step(p0, i);
                if constexpr (S > 2)
                    if (i + 1 < n) {
                        step(p1, i + 1);
                        if constexpr (S > 3)
                            if (i + 2 < n) step(p2, i + 2);
                    }
            }
        }
        // the last fetches have landed before LDS takes the sums or ends
        wait_mem<0, true>();
        if (part) {
            const int slot = n % S;
            read(slot == 0 ? p0 : slot == 1 ? p1 : slot == 2 ? p2 : p3);
            mask(a.K - full * kBK - 16 * g);
            mul();
        }
    } else {
        i4 v[L];
        auto load = [&](int i) {
            const int k0 = (wave + i * WK) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j) v[j] = any16((j < 2 * TN ? pw : px) + off[j] + k0);
        };
        if (n > 0) load(0);
        for (int i = 0; i < n; ++i) {
#pragma unroll
            for (int j = 0; j < L; ++j) *reinterpret_cast<i4 *>(p0 + j * 1024 + lane * 16) = v[j];
            if (i + 1 < n) load(i + 1);
            read(p0);
            mul();
        }
    }
    if (!kVec && full * kBK < a.K && wave == full % WK) { // the bytes past the last whole block
        const int8_t *const we = a.w + static_cast<int64_t>(a.N) * a.K, *const xe = a.a + static_cast<int64_t>(a.M) * a.K;
        for (int k = full * kBK; k < a.K; k += 64) {
#pragma unroll
            for (int i = 0; i < TN; ++i)
                wf[0][i] = load16(a.w + static_cast<int64_t>(min(c0 + 16 * i + r, a.N - 1)) * a.K, k + 16 * g, a.K, we);
#pragma unroll
            for (int j = 0; j < TM; ++j)
                xf[0][j] = load16(a.a + static_cast<int64_t>(min(m0 + 16 * j + r, a.M - 1)) * a.K, k + 16 * g, a.K, xe);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[0][i], xf[0][j], acc[i][j], 0, 0, 0);
        }
    }
    __syncthreads();
    // tile t of a wave lies in its piece of r0 as far as that reaches, then in r1's
    constexpr int kIn0 = L;
    static_assert(TN * TM <= 2 * L, "the sums fit two pieces");
#pragma unroll
    for (int t = 0; t < TN * TM; ++t)
        *reinterpret_cast<i4 *>((t < kIn0 ? p0 + t * 1024 : p1 + (t - kIn0) * 1024) + lane * 16) =
            acc[t / TM][t % TM];
    constexpr int NT = (TN * TM + WK - 1) / WK;           // tiles a wave sums and writes: wave, wave + WK, ..
    Channels chs[NT];
    float sas[NT];
    chs[0] = ch;
    sas[0] = sa;
#pragma unroll
    for (int i = 1; i < NT; ++i) {
        const int t = min(wave + i * WK, TN * TM - 1);
        chs[i] = Channels(a, min(c0 + 16 * (t / TM) + 4 * g, a.N - 1), type_bytes(a));
        sas[i] = a.a_scale[min(m0 + 16 * (t % TM) + r, a.M - 1)];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t = wave + i * WK;
        if (t >= TN * TM) break;
        const int8_t *p = t < kIn0 ? r0 + t * 1024 : r1 + (t - kIn0) * 1024;
        i4 s = *reinterpret_cast<const i4 *>(p + lane * 16);
#pragma unroll
        for (int k = 1; k < WK; ++k) s += *reinterpret_cast<const i4 *>(p + k * kPiece + lane * 16);
        const int ct = c0 + 16 * (t / TM) + 4 * g, mt = m0 + 16 * (t % TM) + r;
        if (ct < a.N && mt < a.M) put4(a, chs[i], ct, mt, sas[i], s);
    }
}

// ------------------------------------------------------- one tile a workgroup
// BN channels x BM tokens a workgroup, its waves in a WN x WM grid over them,
// with a ring of S blocks in LDS that hides the latency of the fetches where
// the chip holds a workgroup a compute unit.  A block is multiplied in halves
// of 64 k: while one half is multiplied the next is read from LDS, and one
// barrier a block hands its buffer back to the fetches.  Rows that are not
// 16-byte aligned (kVec false) pass through registers instead, into two
// buffers.
template <typename OT, int BN, int BM, int WN, int WM, int S, bool kVec>
__global__ __launch_bounds__(64 * WN * WM) void k_linear_block(LinearArgs a, int tiles_n, int tiles_m) {
    constexpr int NW = WN * WM;
    constexpr int TN = BN / WN / 16, TM = BM / WM / 16;
    constexpr int L = (BN + BM) / 8 / NW, LN = BN / 8 / NW;
    constexpr int kBytes = (BN + BM) * kBK;
    static_assert(S >= 2 && S <= 4 && (kVec || S == 2), "");
    static_assert(NW * kStageBytes <= kBytes, "the waves' pieces for the stores fit a block");
    __shared__ alignas(1024) int8_t r0[kBytes], r1[kBytes], r2[S > 2 ? kBytes : 16], r3[S > 3 ? kBytes : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;
    int tn, tm;
    tile_of(blockIdx.x, tiles_n, tiles_m, tn, tm);
    if (tn >= tiles_n) return;
    const int c0 = tn * BN, m0 = tm * BM;
    const int8_t *pw = a.w + static_cast<int64_t>(c0) * a.K, *px = a.a + static_cast<int64_t>(m0) * a.K;
    const uint32_t nw = span(a.N - c0, a.K), nx = span(a.M - m0, a.K);
    int off[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        int row = ((j < LN ? j : j - LN) * NW + wave) * 8 + (lane >> 3);
        const int slot = 16 * ((lane & 7) ^ swz(row));
        if (!kVec) row = min(row, j < LN ? a.N - 1 - c0 : a.M - 1 - m0);
        off[j] = row * a.K + slot;
    }
    const int rd[2] = {r * kBK + 16 * (g ^ swz(r)), r * kBK + 16 * ((4 + g) ^ swz(r))};
    i4 acc[TN][TM] = {};
    i4 wf[2][TN], xf[2][TM];
    auto read = [&](const int8_t *buf, int half) {
#pragma unroll
        for (int j = 0; j < TM; ++j)
            xf[half][j] = *reinterpret_cast<const i4 *>(buf + (BN + (wm * TM + j) * 16) * kBK + rd[half]);
#pragma unroll
        for (int i = 0; i < TN; ++i)
            wf[half][i] = *reinterpret_cast<const i4 *>(buf + (wn * TN + i) * 16 * kBK + rd[half]);
    };
    auto mul = [&](int half) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[half][i], xf[half][j], acc[i][j], 0, 0, 0);
    };
    const int n = a.K / kBK;                              // whole blocks
    // piece j of this wave in a buffer
    auto at = [&](int j) { return (j < LN ? 0 : BN * kBK) + ((j < LN ? j : j - LN) * NW + wave) * 1024; };
    if constexpr (kVec) {
        const int all = (a.K + kBK - 1) / kBK;            // with the block past the whole ones
        auto fetch = [&](int8_t *buf, int i) {            // past the end: the last block again
            const int k0 = min(i, all - 1) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j) fetch16(buf + at(j), j < LN ? pw : px, j < LN ? nw : nx, off[j], k0);
        };
        // block i is in cur, its first half in registers
        auto step = [&](int8_t *cur, int8_t *nxt, int i) {
            read(cur, 1);
            mul(0);
            wait_mem<(S - 2) * L, true>();                // block i + 1 has landed, cur is read
            barrier();
            fetch(cur, i + S);
            read(nxt, 0);
            mul(1);
        };
        fetch(r0, 0);
        fetch(r1, 1);
        if constexpr (S > 2) fetch(r2, 2);
        if constexpr (S > 3) fetch(r3, 3);
        if (n > 0) {
            wait_mem<(S - 1) * L, true>();
            barrier();
            read(r0, 0);
            // whole rounds of the ring, then what is left, as in k_linear_ring
            int b = 0;
            for (; b + S <= n; b += S) {
                step(r0, r1, b);
                if constexpr (S == 2) step(r1, r0, b + 1);
                if constexpr (S > 2) step(r1, r2, b + 1);
                if constexpr (S == 3) step(r2, r0, b + 2);
                if constexpr (S > 3) {
                    step(r2, r3, b + 2);
                    step(r3, r0, b + 3);
                }
            }
            if (b < n) {
                step(r0, r1, b);
                if constexpr (S > 2)
                    if (b + 1 < n) {
                        step(r1, r2, b + 1);
                        if constexpr (S > 3)
                            if (b + 2 < n) step(r2, r3, b + 2);
                    }
            }
        }
    } else {
        i4 v[L];
        auto load = [&](int i) {                          // past the end: the last block again
            const int k0 = min(i, n - 1) * kBK;
#pragma unroll
            for (int j = 0; j < L; ++j) v[j] = any16((j < LN ? pw : px) + off[j] + k0);
        };
        auto put = [&](int8_t *buf) {
#pragma unroll
            for (int j = 0; j < L; ++j) *reinterpret_cast<i4 *>(buf + at(j) + lane * 16) = v[j];
        };
        auto step = [&](int8_t *cur, int8_t *nxt, int i) {
            read(cur, 1);
            mul(0);
            __syncthreads();                              // nxt is written, cur is read
            put(cur);                                     // block i + 2
            load(i + 3);
            read(nxt, 0);
            mul(1);
        };
        if (n > 0) {
            load(0);
            put(r0);
            load(1);
            put(r1);
            load(2);
            __syncthreads();
            read(r0, 0);
            for (int b = 0; b < n; b += 2) {
                step(r0, r1, b);
                if (b + 1 < n) step(r1, r0, b + 1);
            }
        }
    }
    // the last fetches have landed, and every wave is done with the ring
    wait_mem<0, true>();
    __syncthreads();
    if (kVec && n * kBK < a.K) {                          // the block past the whole ones
        const int slot = n % S, left = a.K - n * kBK - 16 * g;
        const int8_t *buf = slot == 0 ? r0 : slot == 1 ? r1 : slot == 2 ? r2 : r3;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            read(buf, half);
#pragma unroll
            for (int i = 0; i < TN; ++i)                  // weights past the last k are zero
                wf[half][i] = 64 * half < left ? wf[half][i] : i4{0, 0, 0, 0};
            mul(half);
        }
        __syncthreads();
    }
    if (!kVec && n * kBK < a.K) {                         // the bytes past the last whole block
#pragma unroll 1
        for (int j = wave; j < (BN + BM) / 8; j += NW) {
            const int row = j * 8 + (lane >> 3), in = row < BN ? row : row - BN;
            const int8_t *p = row < BN ? a.w + static_cast<int64_t>(min(c0 + in, a.N - 1)) * a.K
                                       : a.a + static_cast<int64_t>(min(m0 + in, a.M - 1)) * a.K;
            const int8_t *end = row < BN ? a.w + static_cast<int64_t>(a.N) * a.K : a.a + static_cast<int64_t>(a.M) * a.K;
            *reinterpret_cast<i4 *>(r0 + j * 1024 + lane * 16) =
                load16(p, n * kBK + 16 * ((lane & 7) ^ swz(in)), a.K, end);
        }
        __syncthreads();
        read(r0, 0);
        read(r0, 1);
        mul(0);
        mul(1);
        __syncthreads();
    }
    write_tile<OT, TN, TM>(a, c0 + wn * TN * 16, m0 + wm * TM * 16, lane, r0 + wave * kStageBytes, acc);
}

// -------------------------------------------------------------- large product
// Persistent workgroups over tiles of 256 channels x 256 tokens, 8 waves of 64 x
// 128 each: 128 accumulators a lane, two waves a SIMD, all of LDS (two buffers
// of one block, and the waves' pieces for the stores).  The fetches run two
// blocks ahead of the multiplication and over tile borders, so the next tile is
// on its way while this one is written.  Matrix instructions alone reach 3.5
// POP/s here on random operands (the clock drops under them); per block of k
// this loop runs at 2.5, at 8192 x 8192 x 8192 the whole product at 2.3 and at
// 32768 x 12352 x 2048 into bf16 at 1.9, where the results' bytes weigh more.
// 32 x 32 x 32 instructions measured 25 % slower, blocks of 64 k in four
// buffers 10 %.
// k is a multiple of 256 here: masks for a ragged k did not fit beside operands
// held ahead, and one half at a time was 15-75 % slower than rounds of 256 x 128
// tiles (124 us against 89 at 4096 x 8192 x 2176 into f32).
template <typename OT>
__global__ __launch_bounds__(512) void k_linear_tile(LinearArgs a, int tiles_n, int tiles_m) {
    constexpr int BN = 256, BM = 256, WN = 4, NW = 8;
    constexpr int TN = BN / WN / 16, TM = BM / (NW / WN) / 16;
    constexpr int F = BN / 8 / NW;                        // fetches of an operand's block a wave makes
    __shared__ alignas(1024) int8_t b0[(BN + BM) * kBK], b1[(BN + BM) * kBK];
    __shared__ alignas(16) int8_t stage[NW * kStageBytes];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;
    const int blocks = a.K / kBK;                         // of a tile, in pairs
    const int tiles = tiles_n * tiles_m;

    // each XCD (ids modulo 8) takes a run of consecutive tiles
    const int per_xcd = (tiles + 7) / 8, step = gridDim.x / 8;
    const int first = (blockIdx.x & 7) * per_xcd, end = min(tiles, first + per_xcd);
    int tile = first + (blockIdx.x >> 3);
    if (tile >= end) return;

    int off[F];
#pragma unroll
    for (int j = 0; j < F; ++j) {
        const int row = (j * NW + wave) * 8 + (lane >> 3);
        off[j] = row * a.K + 16 * ((lane & 7) ^ swz(row));
    }
    const int rd[2] = {r * kBK + 16 * (g ^ swz(r)), r * kBK + 16 * ((4 + g) ^ swz(r))};

    // The fetch stream: block fb of tile ft, and the tile after it (past the
    // last tile, that one again).
    Tile t = tile_at(tile, tiles_n, tiles_m);
    int fb = 0, ft = tile, ftn = tile;
    const int8_t *pw = a.w + static_cast<int64_t>(t.n) * BN * a.K, *pwn = pw;
    const int8_t *px = a.a + static_cast<int64_t>(t.m) * BM * a.K, *pxn = px;
    uint32_t nw = span(a.N - t.n * BN, a.K), nwn = nw, nx = span(a.M - t.m * BM, a.K), nxn = nx;
    auto aim = [&]() {
        ftn = ft + step < end ? ft + step : ft;
        const Tile f = tile_at(ftn, tiles_n, tiles_m);
        pwn = a.w + static_cast<int64_t>(f.n) * BN * a.K;
        pxn = a.a + static_cast<int64_t>(f.m) * BM * a.K;
        nwn = span(a.N - f.n * BN, a.K);
        nxn = span(a.M - f.m * BM, a.K);
    };
    auto fetch = [&](int8_t *buf) {
        const int k0 = fb * kBK;
#pragma unroll
        for (int j = 0; j < F; ++j) fetch16(buf + (j * NW + wave) * 1024, pw, nw, off[j], k0);
#pragma unroll
        for (int j = 0; j < F; ++j) fetch16(buf + BN * kBK + (j * NW + wave) * 1024, px, nx, off[j], k0);
        const bool wrap = ++fb == blocks;                  // at most once a tile
        fb = wrap ? 0 : fb;
        ft = wrap ? ftn : ft;
        pw = wrap ? pwn : pw;
        px = wrap ? pxn : px;
        nw = wrap ? nwn : nw;
        nx = wrap ? nxn : nx;
    };
    i4 acc[TN][TM];
    i4 wf[2][TN], xf[2][TM];
    auto read = [&](const int8_t *buf, int half) {
#pragma unroll
        for (int j = 0; j < TM; ++j)
            xf[half][j] = *reinterpret_cast<const i4 *>(buf + (BN + (wm * TM + j) * 16) * kBK + rd[half]);
#pragma unroll
        for (int i = 0; i < TN; ++i)
            wf[half][i] = *reinterpret_cast<const i4 *>(buf + (wn * TN + i) * 16 * kBK + rd[half]);
    };
    auto mul = [&](int half) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[half][i], xf[half][j], acc[i][j], 0, 0, 0);
    };
    // a block is in cur, its first half in registers, the next block on its way to nxt
    auto block = [&](int8_t *cur, int8_t *nxt) {
        read(cur, 1);
        mul(0);
        wait_mem<0, true>();
        barrier();                                        // nxt has landed, cur is read
        fetch(cur);
        read(nxt, 0);
        mul(1);
    };
    aim();
    fetch(b0);
    fetch(b1);
    wait_mem<0, true>();
    barrier();
    read(b0, 0);
    for (;;) {
        aim();
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = i4{0, 0, 0, 0};
        for (int b = 0; b < blocks; b += 2) {
            block(b0, b1);
            block(b1, b0);
        }
        write_tile<OT, TN, TM>(a, t.n * BN + wn * TN * 16, t.m * BM + wm * TM * 16, lane,
                               stage + wave * kStageBytes, acc);
        tile += step;
        if (tile >= end) break;
        t = tile_at(tile, tiles_n, tiles_m);
    }
    wait_mem<0, true>();                                  // nothing lands in LDS after the end
}

// ------------------------------------------------------------------- dispatch
template <int TN, int TM, int WK, int S>
hipError_t launch_ring(const LinearArgs &a, hipStream_t s) {
    const int tn = static_cast<int>(tiles(a.N, 16 * TN)), tm = static_cast<int>(tiles(a.M, 16 * TM));
    if (a.K % 16 == 0)
        k_linear_ring<TN, TM, WK, S, true><<<tile_grid(tn, tm), dim3(64 * WK), 0, s>>>(a, tn, tm);
    else
        k_linear_ring<TN, TM, WK, S, false><<<tile_grid(tn, tm), dim3(64 * WK), 0, s>>>(a, tn, tm);
    return hipGetLastError();
}

template <typename OT, int BN, int BM, int WN, int WM, int S, bool kAligned = false>
hipError_t launch_block(const LinearArgs &a, hipStream_t s) {
    const int tn = static_cast<int>(tiles(a.N, BN)), tm = static_cast<int>(tiles(a.M, BM));
    const dim3 block(64 * WN * WM);
    if constexpr (kAligned)                               // called for rows of whole chunks only
        k_linear_block<OT, BN, BM, WN, WM, S, true><<<tile_grid(tn, tm), block, 0, s>>>(a, tn, tm);
    else if (a.K % 16 == 0)
        k_linear_block<OT, BN, BM, WN, WM, S, true><<<tile_grid(tn, tm), block, 0, s>>>(a, tn, tm);
    else
        k_linear_block<OT, BN, BM, WN, WM, 2, false><<<tile_grid(tn, tm), block, 0, s>>>(a, tn, tm);
    return hipGetLastError();
}

template <typename OT>
hipError_t launch_tile(const LinearArgs &a, int cus, hipStream_t s) {
    const int tn = static_cast<int>(tiles(a.N, 256)), tm = static_cast<int>(tiles(a.M, 256));
    const int64_t all = static_cast<int64_t>(tn) * tm, most = cus >= 8 ? cus / 8 * 8 : 8;
    const dim3 grid(static_cast<unsigned>(all < most ? (all + 7) / 8 * 8 : most));
    k_linear_tile<OT><<<grid, dim3(512), 0, s>>>(a, tn, tm);
    return hipGetLastError();
}

template <typename OT>
hipError_t launch(const LinearArgs &a, hipStream_t s) {
    // The largest tile that still gives more than half of the compute units a
    // workgroup, and is no wider than the operands rounded up (64 channels, 16
    // tokens at least): a unit holds one workgroup of most kernels here, so the next
    // smaller tile would take two rounds.  Measured over 1..2048 tokens x (2048 channels,
    // k = 4096 | 12352, k = 2048), f32 out: the tile this picks was the fastest or
    // within 5 %, but 13 % slower than a 64 x 128 tile at 64 x 12352; one size
    // larger or smaller cost up to 2x (us, 64 x 64 | 64 x 128 | 128 x 128 tiles:
    // 10.8 | 12.8 | 14.4 at 128 x 2048, 12.5 | 13.3 | 15.8 at 512 x 2048, 55 | 37 |
    // 29 at 512 x 12352), and asking for three of four units up to 2.2x (320 x
    // 2048, k = 4096: 15.2 | 11.3; 5953 x 144, k = 64: 9.7 | 4.4).
    const int cus = device_cus();
    const auto wide = [&](int bn, int bm) { return (bn <= 64 || bn < 2 * a.N) && (bm <= 16 || bm < 2 * a.M); };
    const auto fits = [&](int bn, int bm) {
        return wide(bn, bm) && 2 * tiles(a.N, bn) * tiles(a.M, bm) > static_cast<int64_t>(cus);
    };
    if (fits(128, 128)) {
        // A short k leaves little to hide latency behind but another workgroup, so
        // two buffers and two workgroups a unit (5000 x 5000, k = 64, f32: 21.7 us
        // against 26.3 for what follows; equal at k = 256).
        if (a.K < 256 && a.K % 16 == 0) return launch_block<OT, 128, 128, 2, 4, 2, true>(a, s);
        // Else a unit holds one workgroup, and the tile whose rounds of workgroups end
        // first is taken: ns a round of 4096 k, of no k, measured
        // (us, 128 x 128 | 256 x 128 | 256 x 256 tiles: 29 | 23 | 36 at 512 x 12352,
        // 33 | 24 | 37 at 640, 77 for the last at 2048, k = 2048).  The choice was the
        // fastest or within 10 % from 300 to 32768 tokens.
        const auto ns = [&](int bn, int bm, int k4096, int none) {
            const int64_t rounds = (tiles(a.N, bn) * tiles(a.M, bm) + cus - 1) / cus;
            return wide(bn, bm) ? rounds * (static_cast<int64_t>(a.K) * k4096 / 4096 + none) : INT64_MAX;
        };
        const int64_t small = ns(128, 128, 16800, 6100);
        if (a.K % 16 == 0) {
            const int64_t mid = ns(256, 128, 33600, 6200),
                          large = a.K % 256 == 0 ? ns(256, 256, 54500, 8700) : INT64_MAX;
            if (large <= mid && large <= small) return launch_tile<OT>(a, cus, s);
            if (mid <= small) return launch_block<OT, 256, 128, 4, 2, 3, true>(a, s);
        }
        return launch_block<OT, 128, 128, 2, 4, 4>(a, s);
    }
    if (fits(64, 128)) return launch_block<OT, 64, 128, 2, 2, 4>(a, s);
    if (fits(64, 64)) return launch_ring<4, 4, 4, 2>(a, s);
    if (fits(32, 64)) return launch_ring<2, 4, 4, 3>(a, s);
    if (fits(64, 32)) return launch_ring<4, 2, 4, 3>(a, s);
    if (fits(32, 32)) return launch_ring<2, 2, 4, 4>(a, s);
    if (fits(64, 16)) return launch_ring<4, 1, 4, 3>(a, s);
    return launch_ring<1, 1, 8, 2>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
    switch (a.out_type) {
    case GDN_F32: return launch<F32>(a, s);
    case GDN_BF16: return launch<BF16>(a, s);
    case GDN_F16: return launch<F16>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
