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
// along the lists; numbers between two parts' tiles are empty.  `part` counts from
// first_part: part 0 mostly has no rows, and an empty number at the front would shift
// all tiles against the groups that share operands (1024 rows of one list, 4096 x 4096,
// 128 x 128 tiles with four chunks under way: 56 us with it, 37 without).
__host__ __device__ inline int first_part(const int32_t *offsets)
{
    return offsets[0] <= 0 ? 1 : 0;
}
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

// Whether position base + lane is before `last`, for positions that fit 32 bits and 64
// lanes: their sum may not fit (base from 2^31 - 63 on), their distance does.
__host__ __device__ inline bool position_before(int base, int lane, int last)
{
    return lane < last - base;
}

// A kind of tile that 16-bit operands are copied for: tm x tn results, `per_cu`
// workgroups a CU; a chunk of 64 takes `alone` us where no CU has more workgroups than it
// holds, those of 256 tiles `full` us where all have many, and matrices come from
// memory at `memory` TB/s.
struct CopyTile {
    int tm, tn, per_cu;
    double alone, full, memory;
};

// Estimate of a product's time: the matrices' bytes and the tiles' chunks, which
// overlap where neither is much the longer.
inline double copy_time(const CopyTile &t, double tiles, int d, double bytes)
{
    const double chunks = (d + 63) / 64;
    const double rounds = (double)(int64_t)((tiles + 256 * t.per_cu - 1) / (256 * t.per_cu));
    const double turn = t.alone * rounds, all = t.full * tiles / 256;
    const double work = chunks * (turn > all ? turn : all), read = bytes / t.memory * 1e-6;
    return __builtin_sqrt(work * work + read * read);
}

// The tiles of the products of rows; the first two and the fourth with four chunks under
// way, the others with two.  Few rows want many small workgroups with much under way,
// many rows large tiles that read less.  Measured (matrices not in the caches), us:
//   one list of 4096 x 4096, 256 rows      26   32   55   40   59   95
//   the same, 1024 rows                    71   55   57   43   60   97
//   64 lists of 2048 x 2048, 16 rows each 109  123  131  133  146  173
//   the same, 1024 rows each             1294 1087  846  813  699  603
// The three numbers are fitted to 198 such sizes (1 to 64 lists of 512^2 to 8192^2, 4 to
// 4096 rows each, and adapters): the least estimate's tile is 1.5 % slower than the
// fastest on average, more than 10 % at 12 of them and 30 % at most.
constexpr CopyTile kCopyTiles[6] = {
    {32, 128, 1, 0.33, 0.20, 5.4},  {64, 128, 1, 0.45, 0.45, 4.6},  {64, 128, 2, 0.64, 0.38, 5.1},
    {128, 128, 1, 0.63, 0.67, 4.9}, {128, 128, 2, 0.98, 0.56, 3.8}, {256, 256, 1, 1.56, 2.08, 4.8},
};

// Which of them.  `lists`: the rows are sorted by list, each with a matrix of its own, and
// half a tile of a list stands empty on average; else all have the same one.
inline int copy_tile(int64_t rows, int nlist, int n, int d, bool lists)
{
    const int64_t used = rows < nlist ? rows : nlist;
    int best = 0;
    double least = 0;
    for (int i = 0; i < 6; ++i) {
        const CopyTile &t = kCopyTiles[i];
        int64_t high = (rows + t.tm - 1) / t.tm + (lists ? used / 2 : 0);
        if (lists && high < used)
            high = used;
        const double time = copy_time(t, (double)(high * ((n + t.tn - 1) / t.tn)), d,
                                      2.0 * n * d * (lists ? used : 1));
        if (i == 0 || time < least) {
            best = i;
            least = time;
        }
    }
    return best;
}

// The gradient's tiles, 128 x 128 or 256 x 256 results, and the workgroups that share a
// list's rows: by an estimate of the time in us.  A tile's chunk of 64 rows takes 1.3
// us (128, two workgroups a CU) or 1.6 to 2.5 (256, one a CU, the more CUs have one), all
// CUs' together at least 0.85 or 2.5 us for 256 of them; shared lists cost a launch
// and the parts' bytes at 8 TB/s (they stay in the caches).  At least eight chunks of
// an even list's rows a workgroup.  65,536 rows of one list, 1024 x 1024: 128 x 128 tiles
// of eight workgroups 194 us, 256 x 256 of 16 152; 8 lists of 1024 rows, 512 x 512: 25
// us without sharing, 26 with two workgroups, 59 with 16; 64 lists of 512 rows, 512 x 512:
// 46 us in 128 x 128 tiles, 33 in 256 x 256.
struct GradientShare {
    int size, splits;
};
inline GradientShare gradient_share(int64_t rows, int nlist, int n, int d)
{
    GradientShare best{128, 1};
    double least = 0;
    for (int size = 128; size <= 256; size *= 2) {
        const double tiles =
            (double)nlist * ((n + size - 1) / size) * ((d + size - 1) / size);
        const int slots = size == 256 ? 256 : 512; // workgroups at once
        for (int splits = 1; splits <= 64; splits *= 2) {
            if (splits > 1 && (splits * tiles > slots || rows / nlist < (int64_t)splits * 512))
                break;
            const double chunks = (double)((rows / nlist / splits + 63) / 64);
            const double busy = tiles * splits < slots ? tiles * splits / slots : 1;
            const double rounds = (double)(int64_t)((tiles * splits + slots - 1) / slots);
            const double alone = chunks * rounds * (size == 256 ? 1.6 + 0.9 * busy : 1.3);
            const double all = chunks * splits * tiles / 256 * (size == 256 ? 2.5 : 0.85);
            const double join =
                splits == 1 ? 0 : 4 + (double)splits * nlist * n * d * (8 / 8e6);
            const double time = (alone > all ? alone : all) + join;
            if (least == 0 || time < least) {
                best = {size, splits};
                least = time;
            }
        }
    }
    return best;
}

} // namespace ivfpq
