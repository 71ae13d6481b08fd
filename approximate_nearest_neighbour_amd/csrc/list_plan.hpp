// Arithmetic of the products per list that the device kernels share with the
// host (the launchers, and a CPU test that walks every tile of a product).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ivfpq {

// Rows sorted by list fall into nlist + 2 parts: the rows before the first list
// (part 0), the lists (part e + 1), the rows past the last one.  Part i begins
// at row part_begin(i); an offset outside [0, rows] counts as the nearer end.
__host__ __device__ inline int64_t part_begin(const int32_t *offsets, int nlist, int64_t rows,
                                              int i)
{
    if (i <= 0)
        return 0;
    if (i >= nlist + 2)
        return rows;
    const int64_t o = offsets[i - 1];
    return o < 0 ? 0 : o > rows ? rows : o;
}

// Where the tiles of a part stand among the tile numbers of a product.  With
// `by_row` a tile number is a row, and a tile stands at its first row's.  Else
// part i begins at number begin(i) / tm + i, which leaves room for the last tile
// of the part before to be a short one.  Either way the numbers follow from the
// offset of the part alone, so a workgroup finds its part by search, without sums
// along the lists; numbers between two parts' tiles are empty.
__host__ __device__ inline int64_t part_slot(int64_t begin, int part, int tm, bool by_row)
{
    return by_row ? begin : begin / tm + part;
}

// Tile numbers of a product: the fewer of both ways.
inline bool slots_by_row(int64_t rows, int nlist, int tm)
{
    return rows <= rows / tm + nlist + 2;
}
inline int64_t tile_slots(int64_t rows, int nlist, int tm)
{
    return slots_by_row(rows, nlist, tm) ? rows : rows / tm + nlist + 2;
}

// First row of tile number `slot` inside the part that begins at `begin`; not
// below the part's end: no tile stands there.
__host__ __device__ inline int64_t slot_row(int64_t slot, int64_t begin, int64_t end, int part,
                                            int tm, bool by_row)
{
    if (by_row)
        return (slot - begin) % tm == 0 ? slot : end;
    const int64_t row = begin + (slot - part_slot(begin, part, tm, false)) * tm;
    return row < end ? row : end;
}

// Part s of the rows [p0, p1) of a list that `splits` workgroups share: whole chunks of
// 64 rows but for the last part, the same number of them for all that have any.
__host__ __device__ inline void split_rows(int64_t &p0, int64_t &p1, int s, int splits)
{
    const int64_t chunks = (p1 - p0 + 63) / 64, per = (chunks + splits - 1) / splits * 64;
    const int64_t end = p1;
    p0 = p0 + s * per < end ? p0 + s * per : end;
    p1 = p0 + per < end ? p0 + per : end;
}

// The gradient's tiles: 256 x 256 results if these are 32 at least, else 128 x 128; and
// the workgroups that share a list's rows where the tiles are few: up to one a CU of the
// larger tiles, two of the others, with at least eight chunks of an even list's rows
// each.
struct GradientShare {
    int size, splits;
};
inline GradientShare gradient_share(int64_t rows, int nlist, int n, int d)
{
    auto tiles = [&](int size) {
        return (int64_t)nlist * ((n + size - 1) / size) * ((d + size - 1) / size);
    };
    GradientShare g{tiles(256) >= 32 ? 256 : 128, 1};
    while (g.splits < 64 && 2 * g.splits * tiles(g.size) <= (g.size == 256 ? 256 : 512) &&
           rows / nlist >= 2 * g.splits * 512)
        g.splits *= 2;
    return g;
}

} // namespace ivfpq
