"""Rows of a table by number and the table's gradient, on the GPU against the 64-bit
definitions of oracle/rows.py.

Tolerances.  A looked-up row is one product in float32, rounded once more to its
type.  A sum of n rows in float32 is within n * 2^-23 of the sum of their
magnitudes, one more rounding for the scale and one of the type; small integers
are exact.
"""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R
from test_gpu_list_product import TYPES, UNIT, integers, np64, reals, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d,n", [(1, 1, 1), (5, 7, 3), (100, 8, 1), (1000, 201, 77),
                                      (3000, 64, 1001), (17, 2048, 5), (9, 1030, 4097), (0, 8, 6)])
@pytest.mark.parametrize("dtype", TYPES)
def test_lookup(rows, d, n, dtype):
    rng = np.random.default_rng(rows + d + n)
    table = reals(rng, rows, d, dtype=dtype)
    ids = rng.integers(-1, rows + 2, n).astype(np.int32)
    ids[rng.random(n) < 0.1] = rng.choice([-2 ** 31, 2 ** 31 - 1])
    idt = torch.from_numpy(ids).cuda()
    assert np.array_equal(np64(A.ivfpq_table_lookup_ex(table, idt)),
                          R.table_lookup(np64(table), ids, 1.0))
    scale = float(np.float32(np.sqrt(d)))
    got = np64(A.ivfpq_table_lookup_ex(table, idt, scale=scale))
    want = R.table_lookup(np64(table), ids, scale)
    assert (np.abs(got - want) <= (UNIT[dtype] + 2.0 ** -23) * np.abs(want) + 2.0 ** -25).all()


def ids_of(rng, nvec, k, rows, hot):
    ids = rng.integers(-1, rows + 1, (nvec, k)).astype(np.int32)
    ids[rng.random((nvec, k)) < hot] = rows // 2
    return ids


# hot: share of the numbers that are the same one, whose list is then long
GRADS = [(1, 1, 1, 1, 0.0), (3, 1, 4, 7, 0.0), (33, 1, 2, 64, 0.9), (500, 1, 5003, 201, 0.05),
         (2000, 1, 40, 130, 0.7), (300, 8, 100, 520, 0.3), (1500, 3, 1, 33, 0.0),
         (5000, 1, 3, 72, 0.98), (4096, 2, 2100, 16, 0.5), (70, 1, 9, 2056, 0.6),
         (64, 1, 100000, 8, 0.5)]


@pytest.mark.parametrize("nvec,k,rows,d,hot", GRADS)
@pytest.mark.parametrize("dtype,out", [(t, o) for t in TYPES for o in {t, torch.float32}])
def test_gradient_is_exact_on_integers(nvec, k, rows, d, hot, dtype, out):
    rng = np.random.default_rng(nvec + rows + d)
    grad = integers(rng, nvec, d, dtype=dtype)
    ids = ids_of(rng, nvec, k, rows, hot)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(ids).cuda(), rows)
    got = A.ivfpq_table_grad_ex(grad, offsets, order, scale=0.5, k=k, dtype=out)
    want, _ = R.table_gradient(np64(grad), ids, rows, 0.5)
    assert got.dtype == out and np.array_equal(np64(got), rounded(want, out))


@pytest.mark.parametrize("nvec,k,rows,d,hot", GRADS[2:9])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_reals(nvec, k, rows, d, hot, dtype):
    rng = np.random.default_rng(nvec * k + d)
    grad = reals(rng, nvec, d, dtype=dtype)
    ids = ids_of(rng, nvec, k, rows, hot)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(ids).cuda(), rows)
    scale = float(np.float32(np.sqrt(d)))
    got = np64(A.ivfpq_table_grad_ex(grad, offsets, order, scale=scale, k=k))
    want, mag = R.table_gradient(np64(grad), ids, rows, scale)
    sums = (nvec * k + 1) * 2.0 ** -23 * mag
    assert (np.abs(got - want) <= sums + UNIT[dtype] * (np.abs(want) + sums) + 2.0 ** -25).all()
