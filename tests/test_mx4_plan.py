"""The arithmetic of the 4-bit products on the CPU: the functions that the
device kernels call (csrc/mx4_plan.hpp), compiled for the host and run by
tests/mx4_driver.cpp."""
import os
import random
import subprocess

import pytest

from test_gpu_mx4_tiles import LIST_PARTS, LIST_PRODUCTS, PRODUCTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "approximate_nearest_neighbour_amd", "csrc")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("mx4") / "mx4_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", CSRC, os.path.join(ROOT, "tests", "mx4_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:2000]

    def ask(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True,
                             check=True).stdout.splitlines()
        assert len(out) == len(lines)
        return [[int(v) for v in line.split()[1:]] for line in out]
    return ask


# columns of a tile, groups of waves that share its chunks, longest run of tiles
TILES = [(64, 2, 1), (128, 1, 1), (128, 1, 2), (128, 1, 8), (256, 1, 1), (256, 1, 4)]


def test_no_copy_begins_past_its_matrix(driver):
    """A copy's chunk offset is subtracted from the bytes that are left of the
    matrix in the hardware's range check: it has to be less than those, also in
    the last tile of the last matrix and for the chunks past a row's end."""
    cases = []
    for tn, groups, most in TILES:
        for kb in list(range(1, 35)) + [63, 64, 65, 66, 72, 73, 80, 81, 96, 97, 255, 256, 257]:
            if most > 1 and (kb + 7) // 8 % 2:
                continue  # runs are of rows with an even number of chunks
            for n in (1, tn - 1, tn, tn + 1, 2 * tn + 1, 5 * tn + 3, 8 * tn, 9 * tn + 1):
                for lists in (1, 3):
                    cases.append(f"copies {n} {lists} {kb} {tn} {groups} {most}")
    for case, (issued, past, wrong) in zip(cases, driver(cases)):
        assert issued > 0 and past == 0 and wrong == 0, case


def test_only_chunks_that_are_multiplied_are_copied(driver):
    # one tile of three chunks: three copies of either operand, and none for a tile after it
    (issued, _, _), = driver(["copies 100 1 24 128 1 1"])
    assert issued == 2 * 3
    # a run of three tiles of two chunks
    (issued, _, _), = driver(["copies 300 1 16 128 1 4"])
    assert issued == 2 * 6


def test_runs_cover_the_columns_of_the_largest_matrices(driver):
    # the last columns of a matrix of nearly 2^31 rows, and small ones
    shapes = [(n, tn, most) for tn, _, _ in TILES for most in (1, 2, 8)
              for n in (1, tn, tn + 1, 7 * tn + 5, 2 ** 31 - 16, 2 ** 31 - 17, 2 ** 31 - 128,
                        2 ** 31 - 300)]
    for (n, tn, most), got in zip(shapes, driver([f"run {n} {tn} {most}" for n, tn, most in
                                                  shapes])):
        tiles = -(-n // tn)
        runs = -(-tiles // most)
        assert got == [runs, tiles, min(most, tiles), tiles - (runs - 1) * most], (n, tn, most)


def test_the_grid_covers_the_tiles_of_any_lists(driver):
    # rows before the first list, of each list and past the last one: a tile for
    # each that begins; the largest number is reached
    rng = random.Random(1)
    cases, want, reached = [], [], 0
    for _ in range(400):
        m, nlist, tm = rng.choice([1, 2, 5, 17, 100, 513]), rng.randint(1, 9), rng.choice([16, 64])
        cuts = sorted(rng.randint(0, m) for _ in range(nlist + 1))
        parts = [b - a for a, b in zip([0] + cuts, cuts + [m])]
        cases.append(f"tiles {m} {nlist} {tm}")
        want.append(sum(-(-p // tm) for p in parts))
    for case, tiles, (most,) in zip(cases, want, driver(cases)):
        assert tiles <= most, case
        reached += tiles == most
    assert reached > 0


KERNELS = ["direct1", "direct4", "direct8", "one", "shared", "small", "middle", "large"]


def kernels(driver, shapes):
    """Of products (m, n, d) and products per list (t, k, nlist, n, d)."""
    lines = []
    for s in shapes:
        if len(s) == 3:
            m, n, d = s
            lines.append(f"kernel 0 {m} {n} {-(-d // 32)} 0 {m} 0")
        else:
            t, k, nlist, n, d = s
            lines.append(f"kernel 1 {t * k} {n} {-(-d // 32)} {nlist} {t} 1")
    return [KERNELS[number] for number, in driver(lines)]


def test_the_gpu_tests_reach_the_kernels_that_they_name(driver):
    for cases in (PRODUCTS, LIST_PRODUCTS):
        named = [c[0] for c in cases]
        assert kernels(driver, [c[1:] for c in cases]) == named
    assert {c[0] for c in PRODUCTS} == set(KERNELS)
    assert {c[0] for c in LIST_PRODUCTS} == set(KERNELS) - {"one"}
    assert [kernels(driver, [(t, 2, e1 - e0, n, d)])[0] for _, t, _, n, d, e0, e1 in LIST_PARTS] \
        == [c[0] for c in LIST_PARTS]
    # what the tests of many lists, of graphs and of rows past 4 GiB name
    assert kernels(driver, [(3000, 2, 1000, 20, 64), (3500, 2, 3000, 20, 64),
                            (3000, 2, 1 << 16, 20, 64), (1650, 2, 3, 4200, 512),
                            (140, 3000, 2592), (1301, 8703, 96)]) == \
        ["small", "small", "direct1", "large", "shared", "one"]
    rows = (1 << 20) + 5
    assert driver([f"kernel 1 600 70 256 2 {rows} 1", "kernel 1 600 70 256 2 600 1"]) == \
        [[KERNELS.index("direct8")], [KERNELS.index("shared")]]
