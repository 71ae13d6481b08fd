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

} // namespace ivfpq
