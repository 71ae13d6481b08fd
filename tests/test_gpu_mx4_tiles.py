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
