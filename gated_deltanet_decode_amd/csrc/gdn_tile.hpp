// gdn_tile.hpp - what the kernels of the 8-bit products share: 128-byte lines of k
// on their way to LDS, waits, the order of tiles, and the groups of output
// channels.  Included by kernel sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_serve.hpp"

namespace gdn {
namespace {

typedef int32_t i4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void *lds_t;

constexpr int kBK = 128;      // bytes of k in a block: one line of a row

// A block's row is 8 chunks of 16 bytes; chunk c of row r lies at slot
// c ^ swz(r).  The sixteen rows that one instruction reads at a chunk then
// spread over all banks (no conflict counted).
__device__ __forceinline__ int swz(int row) { return row & 7; }

// Sixteen bytes at any address.
__device__ __forceinline__ i4 any16(const int8_t *p) {
    typedef int32_t any __attribute__((ext_vector_type(4), aligned(1)));
    return *reinterpret_cast<const any *>(p);
}

// Sixteen bytes at k of a row of K bytes, zero past its end.  The load may reach
// into the next rows, but not past the end of the matrix.
__device__ __forceinline__ i4 load16(const int8_t *row, int k, int K, const int8_t *end) {
    i4 v = {0, 0, 0, 0};
    if (k >= K) return v;
    if (row + k + 16 <= end) {
        v = any16(row + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = K - k - 4 * i;                  // bytes of this word that are the row's
            v[i] = n >= 4 ? v[i] : n <= 0 ? 0 : v[i] & ((1 << 8 * n) - 1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k + i < K)
                v[i / 4] |= static_cast<int32_t>(static_cast<uint32_t>(static_cast<uint8_t>(row[k + i]))
                                                 << (8 * (i % 4)));
    }
    return v;
}

// 1 KiB straight into LDS from the `bytes` bytes at base: lane l's 16 bytes at
// off + k0 land at lds + 16 l.  Lanes past the end touch no memory.
__device__ __forceinline__ void fetch16(int8_t *lds, const int8_t *base, uint32_t bytes, int off, int k0) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, bytes, 0x00020000), (lds_t)lds, 16,
        off, k0, 0, 0);
}

// Bytes of `rows` rows of K bytes, as a buffer's size.  No offset into a tile's 256
// rows passes 2^31.
static_assert(int64_t{256} * kTileMaxK < INT64_C(0x7fffffff), "offsets into a tile");
__device__ __forceinline__ uint32_t span(int rows, int K) {
    const int64_t b = static_cast<int64_t>(rows) * K;
    return b < 0x7fffffff ? static_cast<uint32_t>(b) : 0x7fffffffu;
}

// At most N of this wave's vector-memory operations are still on their way
// (they complete in order), and none of its LDS operations if kLds.
template <int N, bool kLds>
__device__ __forceinline__ void wait_mem() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kLds ? 0x0070 : 0x0F70) | (N & 15) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The group of channel c: its number and its first channel.
template <typename Args>
__device__ __forceinline__ int group_of(const Args &a, int c, int &first) {
    int s = 0;
    first = 0;
#pragma unroll
    for (int j = 0; j < kLinearMaxOuts - 1; ++j)
        if (c >= a.end[j]) {
            s = j + 1;
            first = a.end[j];
        }
    return s;
}

// The channel and token tile of workgroup id.  Each XCD (ids modulo 8) takes a
// run of consecutive tiles, the token tiles of a channel tile after each other,
// so that its L2 holds their weights; ids past the last tile have tn >= tiles_n.
__device__ __forceinline__ void tile_of(int id, int tiles_n, int tiles_m, int &tn, int &tm) {
    const int t = (id & 7) * static_cast<int>(gridDim.x >> 3) + (id >> 3);
    tn = t / tiles_m;
    tm = t - tn * tiles_m;
}
inline dim3 tile_grid(int64_t tiles_n, int64_t tiles_m) {
    return dim3(static_cast<unsigned>((tiles_n * tiles_m + 7) / 8 * 8));
}

constexpr int64_t tiles(int64_t n, int64_t b) { return (n + b - 1) / b; }

struct Tile {
    int n, m;
};
// Tile i in an order that keeps neighbours close: groups of 8 token tiles by
// all channel tiles.
__device__ __forceinline__ Tile tile_at(int i, int tiles_n, int tiles_m) {
    constexpr int kG = 8;
    const int per = kG * tiles_n;
    const int grp = i / per, in = i - grp * per;
    const int gm = min(kG, tiles_m - grp * kG);
    const int n = in / gm;
    return Tile{__builtin_amdgcn_readfirstlane(n), __builtin_amdgcn_readfirstlane(grp * kG + in - n * gm)};
}

}  // namespace
}  // namespace gdn
