// Host driver for the arithmetic of the 4-bit products (csrc/mx4_plan.hpp): the
// functions the device kernels call, run on the CPU.
//
// commands on stdin, one a line, an answer line each:
//   copies n lists kb tn groups most
//       walks every copy of the last matrix's tiles in the kernel's order (runs of
//       `most` tiles of `tn` columns) and of a first operand with one row left:
//       "copies <issued> <begun past the bytes left> <chunks not multiplied once>"
//   run n tn most
//       the runs of tiles that start along n columns:
//       "run <runs> <tiles in all> <tiles of the first run> <of the last run>"
//   tiles m nlist tm
//       "tiles <most tiles of m rows sorted by list>"
//   kernel list m n kb nlist arows order
//       "kernel <number of the kernel that a product takes>"
#include "mx4_plan.hpp"

#include <cstdio>
#include <cstring>
#include <vector>

using namespace ivfpq;

static void copies(long long n, long long lists, int kb, long long tn, int groups, long long most)
{
    const int chunks = (kb + 7) / 8, own = own_chunks(chunks, groups);
    const long long row = 16ll * kb, brows = lists * n, brow0 = brows - n;
    long long issued = 0, past = 0, wrong = 0;
    for (long long n0 = 0; n0 < n; n0 += most * tn) {
        const int run = run_tiles((int)n, (int)n0, (int)tn, (int)most);
        for (int g = 0; g < groups; ++g) {
            // a copy of chunk c of tile t's rows and of a last row of the first operand
            auto copy = [&](int t, int c) {
                const long long at = chunk_byte(c, g, groups, chunks);
                issued += 2;
                past += at >= row;
                const long long left = (brows - (brow0 + n0 + t * tn)) * row;
                past += at >= (left > 0 ? left : 0);
            };
            copy(0, 0);
            for (int t = 0; t < run; ++t)
                for (int c = 0; c < own; c += 2) {
                    if (second_chunk(c, own))
                        copy(t, c + 1);
                    if (second_chunk(c, own) && chunk_after(c, own, t, run))
                        copy(c + 2 < own ? t : t + 1, c + 2 < own ? c + 2 : 0);
                }
        }
    }
    std::vector<int> seen(chunks, 0);
    for (int g = 0; g < groups; ++g)
        for (int c = 0; c < own; ++c)
            if (row_chunk(c, g, groups) < chunks)
                ++seen[row_chunk(c, g, groups)];
    for (int s : seen)
        wrong += s != 1;
    std::printf("copies %lld %lld %lld\n", issued, past, wrong);
}

static void runs(int n, int tn, int most)
{
    long long count = 0, tiles = 0, first = 0, last = 0;
    for (long long n0 = 0; n0 < n; n0 += (long long)most * tn) {
        last = run_tiles(n, (int)n0, tn, most);
        first = count == 0 ? last : first;
        tiles += last;
        ++count;
    }
    std::printf("run %lld %lld %lld %lld\n", count, tiles, first, last);
}

int main()
{
    char what[32];
    while (std::scanf("%31s", what) == 1) {
        long long v[8];
        if (!std::strcmp(what, "copies")) {
            for (int i = 0; i < 6; ++i)
                if (std::scanf("%lld", &v[i]) != 1)
                    return 1;
            copies(v[0], v[1], (int)v[2], v[3], (int)v[4], v[5]);
        } else if (!std::strcmp(what, "run")) {
            for (int i = 0; i < 3; ++i)
                if (std::scanf("%lld", &v[i]) != 1)
                    return 1;
            runs((int)v[0], (int)v[1], (int)v[2]);
        } else if (!std::strcmp(what, "tiles")) {
            for (int i = 0; i < 3; ++i)
                if (std::scanf("%lld", &v[i]) != 1)
                    return 1;
            std::printf("tiles %lld\n", (long long)most_list_tiles(v[0], (int)v[1], v[2]));
        } else if (!std::strcmp(what, "kernel")) {
            for (int i = 0; i < 7; ++i)
                if (std::scanf("%lld", &v[i]) != 1)
                    return 1;
            std::printf("kernel %d\n", (int)mx4_kernel_of(v[0], v[1], (int)v[2], (int)v[3],
                                                          (int)v[4], v[5], v[6]));
        } else {
            return 1;
        }
    }
    return 0;
}
