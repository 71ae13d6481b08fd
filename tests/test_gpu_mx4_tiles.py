"""The tiled kernels of the 4-bit products at their edges, against the 64-bit
definitions of oracle/rows.py.  Tolerances are those of test_gpu_mx4.py: codes
multiply exactly, a float32 sum of K products is within K 2^-23 of the sum of
their magnitudes, and storing rounds once by the unit of the type."""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R
from test_gpu_mx4 import TYPES, check_product, cuda, make_lists, random_mx4

pytestmark = pytest.mark.gpu


def operands(rng, m, n, d, dtype, nlist=None):
    a, b = random_mx4(rng, m, d), random_mx4(rng, (nlist or 1) * n, d)
    if dtype == torch.float16:   # keep sums of up to 8192 products below 65504
        a = (a[0], (a[1] - 8).astype(np.uint8))
    if nlist:
        b = tuple(t.reshape(nlist, n, -1) for t in b)
    return a, b


def check_rows(out, a, b, d, dtype, rows):
    va, vb = R.values(a[0][rows], a[1][rows], d), R.values(*b, d)
    check_product(out[torch.from_numpy(rows).cuda()], va @ vb.T, np.abs(va) @ np.abs(vb).T, d,
                  dtype)


def list_case(rng, t, k, nlist, n, d, dtype, drop=0.05):
    """A product per list and what it has to be: (output, exact, magnitudes)."""
    offsets, order, _ = R.route_sort(make_lists(rng, t, k, nlist, drop), nlist)
    a, b = operands(rng, t, n, d, dtype, nlist)
    exact, mag = R.list_product(R.values(*a, d), R.values(*b, d), offsets, order, k, t * k)
    out = A.ivfpq_mx4_list_product_ex(cuda(a), cuda(b), torch.from_numpy(offsets).cuda(),
                                      order=torch.from_numpy(order).cuda(), k=k, dtype=dtype)
    return out, exact, mag


# the last tile has one row of B left and rows end inside a chunk: one block, two
# and a bit chunks, an even number of chunks; also shared between groups of waves
@pytest.mark.parametrize("t,nlist,n,d", [(33, 2, 129, 32), (40, 3, 129, 544), (70, 2, 257, 272)])
@pytest.mark.parametrize("dtype", TYPES)
def test_last_matrix_with_one_row_in_its_last_tile(t, nlist, n, d, dtype):
    rng = np.random.default_rng(t + n + d)
    out, exact, mag = list_case(rng, t, 2, nlist, n, d, dtype)
    check_product(out, exact, mag, d, dtype)


@pytest.mark.parametrize("m,n,d", [(129, 3009, 2592), (193, 2113, 2209)])
@pytest.mark.parametrize("dtype", TYPES)
def test_shared_chunks_with_one_row_in_the_last_tiles(m, n, d, dtype):
    rng = np.random.default_rng(m + n + d)
    a, b = operands(rng, m, n, d, dtype)
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b), dtype=dtype)
    check_rows(out, a, b, d, dtype, np.arange(m))


# part of the lists, as where lists are split over devices: the rows of the lists
# before and after are zero, whatever the output held; direct kernel, middle, large
# and small tiles, tiles with shared chunks
@pytest.mark.parametrize("t,nlist,n,d,e0,e1", [
    (9, 16, 100, 96, 5, 9), (300, 8, 70, 64, 3, 8), (700, 6, 1300, 544, 2, 5),
    (2600, 5, 1100, 512, 1, 2), (200, 5, 330, 2300, 2, 4), (50, 6, 40, 64, 3, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_before_the_first_list_are_zero(t, nlist, n, d, e0, e1, dtype):
    rng = np.random.default_rng(t + nlist + n + e0)
    offsets, order, _ = R.route_sort(make_lists(rng, t, 2, nlist, 0.05), nlist)
    a, b = operands(rng, t, n, d, dtype, nlist)
    ac, bc, o = cuda(a), cuda(b), torch.from_numpy(order).cuda()
    off = torch.from_numpy(offsets).cuda()
    whole = A.ivfpq_mx4_list_product_ex(ac, bc, off, order=o, k=2, dtype=dtype)
    e1 = max(e1, e0 + 1)
    part = torch.full((2 * t, n), float("nan"), device="cuda", dtype=dtype)
    A.ivfpq_mx4_list_product_ex(ac, tuple(x[e0:e1].contiguous() for x in bc),
                                off[e0:e1 + 1].clone(), order=o, k=2, dtype=dtype, out=part)
    lo, hi = int(offsets[e0]), int(offsets[e1])
    assert 0 < lo < hi < 2 * t
    assert (part[:lo] == 0).all() and (part[hi:] == 0).all()
    # another kernel may take the part, so compare with the definition
    va, vb = R.values(*a, d), R.values(*b, d)
    for e in range(e0, e1):
        rows = np.arange(offsets[e], offsets[e + 1])[::7]
        x = va[order[rows] // 2]
        check_product(part[torch.from_numpy(rows).cuda()], x @ vb[e].T,
                      np.abs(x) @ np.abs(vb[e]).T, d, dtype)
    assert torch.isfinite(whole.float()).all()
