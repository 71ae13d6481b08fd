// Arithmetic of the 4-bit products that the device kernels share with the host
// (the launcher, and a CPU test that walks every copy of a product).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ivfpq {

// A row's blocks come eight at a time: chunks of 128 bytes of codes.  The
// groups of waves that share a tile take two chunks in a row each in turn, the
// same number `own` for every group, an even one where there are several: a
// group's last chunks may lie past the row's end.
__host__ __device__ inline int own_chunks(int chunks, int groups)
{
    return groups == 1 ? chunks : (chunks + 2 * groups - 1) / (2 * groups) * 2;
}

// Which chunk of the row chunk c of group `group` is.
__host__ __device__ inline int row_chunk(int c, int group, int groups)
{
    return groups == 1 ? c : (c & ~1) * groups + 2 * group + (c & 1);
}

// Where the copy of that chunk begins, in bytes from the row's start.  Inside
// the row also for a chunk past its end (the last one is copied again, and its
// exponent bytes are zero): the range check of a copy subtracts this offset from
// the bytes that are left, so it may not pass them.
__host__ __device__ inline int chunk_byte(int c, int group, int groups, int chunks)
{
    const int n = row_chunk(c, group, groups);
    return (n < chunks ? n : chunks - 1) * 128;
}

// Whether the pair of chunks that starts at c has its second one, and whether a
// pair or a tile comes after it: nothing is copied that no product takes.
__host__ __device__ inline bool second_chunk(int c, int own) { return c + 1 < own; }
__host__ __device__ inline bool chunk_after(int c, int own, int tile, int run)
{
    return c + 2 < own || tile + 1 < run;
}

// Tiles of `tn` columns in the run of at most `most` that starts at column n0 < n.
// n may be up to 2^31 - 16: no sum of columns passes n.
__host__ __device__ inline int run_tiles(int n, int n0, int tn, int most)
{
    const int left = (n - n0 - 1) / tn + 1;
    return left < most ? left : most;
}

// Most tiles of `tm` rows that m rows sorted by list can make: every list may end
// inside a tile, and so may the rows before the first list and past the last one.
inline int64_t most_list_tiles(int64_t m, int nlist, int64_t tm)
{
    const int64_t parts = (int64_t)nlist + 2;
    return m / tm + (m < parts ? m : parts);
}

// Kernels of a product: the direct one (its waves sharing a row's blocks among
// 1, 4 or 8), and tiles: of single chunks (64 x 128), of chunks shared between
// two groups of waves (64 x 64), small (64 x 128), middle (128 x 128) and large
// (256 x 256).
enum Mx4Kernel {
    kMx4Direct1, kMx4Direct4, kMx4Direct8, kMx4One, kMx4Shared, kMx4Small, kMx4Middle, kMx4Large
};

// Which kernel.  The direct one reads B once for every 16 rows of A, the tiles
// once for 64 to 256, but they take 10 us and more for their chunks one after
// the other (d 4096).  So the direct one where a matrix has few rows to
// multiply, or all is small: 32 rows by 8192, d 4096 (11.5 us, tiles of up to 64
// rows 11.2 us) is about the limit (48 rows: 15.7 us; 32 rows by 4096, d 8192:
// 12.5 us, tiles 15.7 us).  In 64 lists, 2048 x 2048, of 4 rows on average 29 us
// against 28 to 32, of 8 rows 33 to 38 us against 32; in 128 lists, 1024 x 1024,
// of 4 rows 18 us against 15, of 8 rows 21 to 23 us against 15.
inline Mx4Kernel mx4_kernel_of(bool list, int64_t m, int n, int kb, int nlist, int64_t arows,
                               bool order)
{
    const int64_t mt = list ? most_list_tiles(m, nlist, 16) : (m + 15) / 16;
    const int64_t waves = mt * (((int64_t)n + 15) / 16);
    const int64_t brows = (list ? (int64_t)nlist : 1) * n;
    // what the tiles' 32-bit offsets and 16-byte reads of exponent bytes take
    const bool fits = !(list && order && arows * kb * 16 >= (int64_t)1 << 32) &&
                      brows * kb >= 16 && arows * kb >= 16;
    const bool few = list ? m <= 2ll * nlist : m <= 16 || waves * kb <= 1024 * 128;
    if (few || !fits) {
        // blocks of a row are split only as far as it takes to have 16 waves a
        // CU, with 8 KB each under way, or a turn for each
        if (waves >= 4096 || kb <= 16)
            return kMx4Direct1;
        return waves >= 1024 || kb <= 64 ? kMx4Direct4 : kMx4Direct8;
    }
    auto tiles = [&](int64_t high, int64_t wide) {
        const int64_t parts = list ? (m < nlist ? m : nlist) / 2 : 0; // lists end inside
        return ((m + high - 1) / high + parts) * ((n + wide - 1) / wide);
    };
    if (!list && kb <= 8)
        return kMx4One;
    // Few tiles of long rows wait for their chunks one after the other: tiles of
    // 64 x 64, their chunks shared out between two groups of four waves, while
    // all are under way together (two a CU).  128 x 4096 x 8192 24.4 -> 15.8 us,
    // 512 x 4096 x 8192, which is 512 of them, 29.9 -> 24.7, x 4096 16.6 -> 15.0,
    // x 2048 10.5 -> 11.0; 768 x 4096 x 8192 29.1 -> 36.5.  16 lists of 32 rows, 512
    // x 4096: 15.9 -> 13.5 us.
    if (kb > 64 && tiles(64, 64) <= 512)
        return kMx4Shared;
    // Large tiles (256 x 256) take about three times as long as middle ones (128 x
    // 128) a round of 256: 3000 x 4000 x 4096 35.0 us against 41.2 us, 2048 x 4096 x
    // 4096, which is half a round of them, 32.7 us against 26.3 us.
    // Lists have to fill them: 64 lists, 2048 x 2048, of 512 rows on average 135 us
    // against 147 us, of 256 87 us against 86 us, of 128 71 us against 61 us.
    // Small ones (64 x 128) where few tiles wait for their chunks more than for
    // the matrix cores: 1024 x 2048 x 2048 9.4 us against 9.9 us, 2048 x 2048 x
    // 4096, which is 512 of them, 29.3 us against 18.4 us.  And where lists would
    // leave middle ones empty: 32 rows on average 40 us against 42 us, 64 rows 51
    // us against 52 us (64 rows each 46 us against 38 us).
    const bool large = (!list || m > 256ll * nlist) &&
                       3 * ((tiles(256, 256) + 255) / 256) <= (tiles(128, 128) + 255) / 256;
    const bool small = tiles(64, 128) <= (kb <= 32 ? 512 : 256) || (list && m <= 32ll * nlist);
    return large ? kMx4Large : small ? kMx4Small : kMx4Middle;
}

} // namespace ivfpq
