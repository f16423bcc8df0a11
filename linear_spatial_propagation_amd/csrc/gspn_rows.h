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
// at least ceil(rows / TILE) tiles, and one, and needs no table.  Largest
// n of 0 .. N whose first tile is not behind tile w; the lanes of a wave
// compare 64 sequences at a time.  Whatever the offsets hold, the rows lie
// inside the tensors.
template <int TILE>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int64_t T, int64_t N, uint32_t tiles,
                                          uint32_t w, int lane) {
    Tile r;
    if (!offsets) {
        r.n = w / tiles;   // tiles: of a sequence
        r.j = w - (uint32_t)r.n * tiles;
        r.rows = T / N;
        r.row = r.n * r.rows;
        return r;
    }
    auto clamped = [&](int64_t i) {
        const int64_t o = offsets[i];
        return o < 0 ? 0 : o > T ? T : o;
    };
    int64_t low = 0, count = N + 1;
    while (count > 1) {
        const int64_t step = (count + 63) / 64;
        const int64_t i = lane * step;
        const bool in_front = i < count && clamped(low + i) / TILE + low + i <= w;
        const uint64_t which = __ballot(in_front);
        const int64_t skip = (which ? 63 - __clzll(which) : 0) * step;
        low += skip;
        count = count - skip < step ? count - skip : step;
    }
    const int64_t begin = clamped(low), end = low == N ? T : clamped(low + 1);
    r.n = low;
    r.row = begin;
    r.rows = end > begin ? end - begin : 0;
    r.j = (int64_t)w - begin / TILE - low;
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
