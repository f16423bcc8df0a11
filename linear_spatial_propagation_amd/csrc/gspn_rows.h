// gspn_rows.h -- packed rows of many sequences (or requests), cut into tiles
// that never hold rows of two (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gspn {

struct Tile {
    int64_t row;     // first row of the sequence
    int64_t rows;    // rows of the sequence
    int64_t n;       // the sequence (N: the rows behind the last)
    int64_t j;       // which of its tiles; none of its rows are in it if j * TILE >= rows
};

// Packed sequences take the tiles begin / TILE + n and on: that gives each
// at least ceil(rows / TILE) tiles, and one, and needs no table.  find_tile takes
// the largest n of 0 .. N whose first tile is not behind tile w; the lanes of a
// wave compare 64 sequences at a time, so that up to 4096 take two steps.
// Whatever the offsets hold, the rows lie inside the tensors.
//
// What the first step compares does not depend on the tile: first_offsets is to
// be called before the tile is known, so that the loads run beside that wait.
__device__ __forceinline__ int32_t first_offsets(const int32_t* __restrict__ offsets, int64_t N, int lane) {
    const int64_t i = lane * ((N + 64) / 64);
    return offsets && i <= N ? offsets[i] : 0;
}

template <int TILE>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int64_t T, int64_t N, uint32_t tiles,
                                          uint32_t w, int lane, int32_t first) {
    Tile r;
    if (!offsets) {
        r.n = w / tiles;   // tiles: of a sequence
        r.j = w - (uint32_t)r.n * tiles;
        r.rows = T / N;
        r.row = r.n * r.rows;
        return r;
    }
    auto clamped = [&](int32_t o) { return o < 0 ? 0 : o > T ? T : (int64_t)o; };
    int64_t low = 0, count = N + 1, step = (N + 64) / 64;
    int32_t mine = first;   // offsets[low + lane step]
    for (;;) {
        const int64_t i = lane * step;
        const uint64_t which = __ballot(i < count && clamped(mine) / TILE + low + i <= w);
        const int at = which ? 63 - __clzll(which) : 0;
        if (step == 1) {   // the lanes hold the offsets of neighbours
            low += at;
            r.row = clamped(__builtin_amdgcn_readlane(mine, at));
            const int64_t end = low == N ? T
                                         : clamped(at < 63 ? __builtin_amdgcn_readlane(mine, at + 1) : offsets[low + 1]);
            r.rows = end > r.row ? end - r.row : 0;
            break;
        }
        low += at * step;
        count = count - at * step < step ? count - at * step : step;
        step = (count + 63) / 64;
        mine = low + lane * step <= N ? offsets[low + lane * step] : 0;
    }
    r.n = low;
    r.j = (int64_t)w - r.row / TILE - low;
    if (r.j < 0) r.j = r.rows / TILE + 1;
    return r;
}

// Tiles of rows of equal length, of each sequence and of all; of packed rows,
// of all (the last ones for the rows behind the last sequence).
template <int TILE>
inline uint32_t tiles_of_sequence(int64_t T, int64_t N) {
    const int64_t rows = T / N;
    return (uint32_t)(rows > 0 ? (rows + TILE - 1) / TILE : 1);
}
template <int TILE>
inline uint32_t total_tiles(bool packed, int64_t T, int64_t N) {
    return packed ? (uint32_t)(T / TILE + N + 1) : (uint32_t)N * tiles_of_sequence<TILE>(T, N);
}

}  // namespace gspn
