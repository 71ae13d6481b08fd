"""The tile numbers of products per list on the CPU: the functions that the device
kernels call (csrc/list_plan.hpp), compiled for the host and run by
tests/list_driver.cpp."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "approximate_nearest_neighbour_amd", "csrc")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("lists") / "list_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", CSRC, os.path.join(ROOT, "tests", "list_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:2000]

    def ask(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True,
                             check=True).stdout.splitlines()
        assert len(out) == len(lines)
        return [[int(v) for v in line.split()[1:]] for line in out]
    return ask


def test_every_row_is_in_one_tile(driver):
    """Whatever the ascending offsets (also beyond the rows, as the rows before a
    part's first list and past its last one are passed), every row belongs to exactly
    one tile and every tile to one part."""
    rng = random.Random(5)
    cases = []
    for tm in (16, 32, 64, 128, 256):
        for nlist in (1, 2, 3, 7, 64, 200):
            for rows in (1, 2, tm - 1, tm, tm + 1, 3 * tm, 3 * tm + 5, 1000):
                spread = [
                    [0] * (nlist + 1), [rows] * (nlist + 1), [0] * nlist + [rows],
                    sorted(rng.randint(0, rows) for _ in range(nlist + 1)),
                    [0] + sorted(rng.randint(0, rows) for _ in range(nlist - 1)) + [rows],
                    sorted(rng.randint(-rows - 9, 2 * rows + 9) for _ in range(nlist + 1)),
                    sorted(rng.randint(0, rows) // tm * tm for _ in range(nlist + 1))]
                for offsets in spread:
                    offsets = offsets[:nlist + 1] if nlist > 1 else [offsets[0], offsets[-1]]
                    cases.append(f"walk {tm} {rows} {nlist} " + " ".join(map(str, offsets)))
    for case, (slots, off, wrong, fewer) in zip(cases, driver(cases)):
        assert slots > 0 and off == 0 and wrong == 0 and fewer == 1, case


def test_parts_of_a_list_cover_its_rows(driver):
    cases = []
    for splits in (1, 2, 4, 8, 64):
        for p0 in (0, 5, 1000):
            for n in (0, 1, 63, 64, 65, 128, 500, 4096, 4097, 100001):
                cases.append(f"split {p0} {p0 + n} {splits}")
    for case, (apart, left, uneven) in zip(cases, driver(cases)):
        assert apart == 0 and left == 0 and uneven == 0, case


def test_workgroups_share_a_list_only_where_tiles_are_few(driver):
    cases = [(65536, 1, 2048, 2048), (65536, 8, 256, 256), (32768, 64, 2048, 2048), (2000, 16, 256, 128),
             (100000, 2, 64, 64), (1 << 31, 1, 1, 1), (5000, 1, 1100, 2000)]
    for (rows, nlist, n, d), (size, splits) in zip(
            cases, driver([f"share {r} {l} {n} {d}" for r, l, n, d in cases])):
        tiles = nlist * -(-n // size) * -(-d // size)
        assert size in (128, 256) and 1 <= splits <= 64
        assert splits == 1 or (splits * tiles <= 512 and rows // nlist >= splits * 512)


def test_positions_of_a_batch_end_where_the_lists_do(driver):
    """Also where a position and a lane's number have no sum in 32 bits."""
    top = 2 ** 31 - 1
    cases = [(base, last) for last in (0, 1, 63, 64, 65, 1000, top - 64, top - 1, top)
             for base in (0, last - 65, last - 64, last - 63, last - 1, last, last + 1, top - 1)
             if 0 <= base <= top]
    for (base, last), (count, wrong) in zip(cases, driver([f"batch {b} {e}" for b, e in cases])):
        assert count == min(max(last - base, 0), 64) and wrong == 0, (base, last)
