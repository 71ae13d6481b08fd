// Runs the arithmetic of csrc/list_plan.hpp on the CPU.  A line "split P0 P1 SPLITS"
// prints: parts that do not follow each other, rows not in them, parts but the last
// that are no whole chunks.  "share ROWS NLIST N D" prints the gradient's tile size
// and splits.  "batch BASE LAST" prints how many of 64 lanes have a position from BASE on
// before LAST, and how many of those have none.  A line "walk TM ROWS NLIST
// offsets..." prints: tile numbers, rows covered not exactly once, tiles that do not
// start and end inside one part, and whether the fewer numbers of both ways were taken.
#include "list_plan.hpp"

#include <algorithm>
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

using namespace ivfpq;

int main()
{
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string word;
        int tm, nlist;
        int64_t rows;
        in >> word;
        if (word == "split") {
            int64_t p0, p1;
            int splits;
            in >> p0 >> p1 >> splits;
            int64_t at = p0, apart = 0, uneven = 0;
            for (int s = 0; s < splits; ++s) {
                int64_t a = p0, b = p1;
                split_rows(a, b, s, splits);
                apart += a != at || b < a;
                uneven += b != p1 && (b - a) % 64 != 0;
                at = b;
            }
            std::printf("split %lld %lld %lld\n", (long long)apart, (long long)(p1 - at),
                        (long long)uneven);
            continue;
        }
        if (word == "share") {
            int n, d;
            in >> rows >> nlist >> n >> d;
            const GradientShare g = gradient_share(rows, nlist, n, d);
            std::printf("share %d %d\n", g.size, g.splits);
            continue;
        }
        if (word == "batch") {
            int base, last, count = 0, wrong = 0;
            in >> base >> last;
            for (int lane = 0; lane < 64; ++lane)
                if (position_before(base, lane, last)) {
                    ++count;
                    wrong += (int64_t)base + lane >= last;
                }
            std::printf("batch %d %d\n", count, wrong);
            continue;
        }
        in >> tm >> rows >> nlist;
        std::vector<int32_t> offsets(nlist + 1);
        for (int32_t &o : offsets)
            in >> o;
        const bool by_row = slots_by_row(rows, nlist, tm);
        const int64_t slots = tile_slots(rows, nlist, tm);
        std::vector<int> seen(rows, 0);
        int64_t wrong = 0;
        const int from = first_part(offsets.data());
        for (int64_t s = 0; s < slots; ++s) {
            int part = 0; // the last part that begins at or before the number
            for (int i = 0; i < nlist + 2; ++i)
                if (part_slot(part_begin(offsets.data(), nlist, rows, i), i - from, tm, by_row) <= s)
                    part = i;
            const int64_t begin = part_begin(offsets.data(), nlist, rows, part);
            const int64_t end = part_begin(offsets.data(), nlist, rows, part + 1);
            const int64_t p0 = slot_row(s, begin, end, part - from, tm, by_row);
            const int64_t p1 = std::min(p0 + tm, end);
            if (p0 >= p1)
                continue;
            if (p0 < begin || p1 > end || p0 < 0 || p1 > rows) {
                ++wrong;
                continue;
            }
            for (int64_t p = p0; p < p1; ++p)
                ++seen[p];
        }
        int64_t off = 0;
        for (int c : seen)
            off += c != 1;
        std::printf("%s %lld %lld %lld %d\n", word.c_str(), (long long)slots, (long long)off,
                    (long long)wrong, (int)(slots == std::min(rows, rows / tm + nlist + 2)));
    }
    return 0;
}
