// i4_common.hpp -- what the 4-bit products share: unpacking, group scales, and
// the tiles of routes that are grouped by expert.
#pragma once

#include "ffn_common.hpp"

namespace loom {

typedef int int16v __attribute__((ext_vector_type(16)));

// 16 bytes of packed weights are 32 neighbours of k: byte b holds element b in
// its low half and element 16 + b in its high half.  Each half is moved into the
// high bits of a byte, where it is the int8 16 q: sums carry that factor 16 (so
// they overflow from 2^124 on) and are brought back by a product with 1/16, exact
// for all that f32 holds in full.
constexpr int kI4High = (int)0xF0F0F0F0;
constexpr float kI4Unit = 0.0625f;
__device__ __forceinline__ int4v i4_low(int4v w) { return (w << 4) & kI4High; }
__device__ __forceinline__ int4v i4_high(int4v w) { return w & kI4High; }

// A scale of type ST as f32.
template <int ST>
__device__ __forceinline__ float scale_at(const void *scales, int64_t at) {
    return (float)((const typename ElementOf<ST>::type *)scales)[at];
}

// Sums over the lanes up to and including this one.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1, 2, 4, 8 within 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
    return v;
}

// Tile `index` of the routes grouped by expert, in tiles of up to `size` rows of
// one expert: which expert, its first row and how many.  Every lane takes part
// and returns the same; false past the last tile.  offsets that are out of order
// or out of range make an expert's rows fewer, never others; where ranges overlap there
// may be more tiles than the grid, which counts on each row once, and the last are left out.
__device__ __forceinline__ bool routed_tile(const I4Product &p, int size, int64_t index, int &expert, int64_t &first, int &rows) {
    const int lane = lane_id();
    // more tiles than a grid has, so that sums stay in 32 bits whatever the offsets say
    constexpr int64_t kMost = 1 << 24;
    int64_t before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += kWave) {
        const int e = e0 + lane;
        int begin = 0, end = 0;
        if (e < p.experts) {
            begin = max(p.offsets[e], 0);
            end = min(p.offsets[e + 1], p.tokens);
        }
        const int n = end > begin ? end - begin : 0, tiles = (int)min(((int64_t)n + size - 1) / size, kMost);
        const int scan = wave_scan(tiles);
        const uint64_t past = __ballot(before + scan > index);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int skip = (int)(index - before) - (readlane(scan, at) - readlane(tiles, at));
            expert = e0 + at;
            first = (int64_t)readlane(begin, at) + (int64_t)skip * size;
            rows = min(readlane(n, at) - skip * size, size);
            return true;
        }
        before += readlane(scan, kWave - 1);
    }
    return false;
}

// Row of x for routed row `at`, and whether it is one.
__device__ __forceinline__ bool x_row(const I4Product &p, int64_t at, int64_t &row) {
    row = p.index ? p.index[at] : at;
    const bool there = row >= 0 && row < p.x_rows;
    if (!there) row = 0;
    return there;
}

}  // namespace loom
