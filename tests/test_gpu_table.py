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


def test_gradient_past_the_caches():
    """A gradient of more than 128 MiB, most rows empty, one list of thousands."""
    rows, d, n = 70000, 1024, 6000
    g = torch.Generator(device="cuda").manual_seed(1)
    grad = torch.randint(-3, 4, (n, d), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    ids[::2] = 12345
    offsets, order, _ = A.ivfpq_route_sort_ex(ids.view(-1, 1), rows)
    got = A.ivfpq_table_grad_ex(grad, offsets, order, dtype=torch.float32)
    want = torch.zeros((rows, d), device="cuda").index_add_(0, ids.long(), grad.float())
    assert torch.equal(got, want)       # integers: any order of the sums is exact


@pytest.mark.parametrize("d", [40, 520])
@pytest.mark.parametrize("dtype", TYPES)
def test_bad_values_stay_where_they_are(d, dtype):
    rng = np.random.default_rng(d)
    grad = integers(rng, 900, d, dtype=dtype)
    ids = rng.integers(-1, 30, 900).astype(np.int32)
    ids[::3] = 17
    ids[[5, 7]] = [-1, 4]
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(ids[:, None]).cuda(), 30)
    clean = A.ivfpq_table_grad_ex(grad, offsets, order)
    grad[5], grad[7, 3] = float("nan"), float("inf")   # a masked row, and one of list 4
    got = A.ivfpq_table_grad_ex(grad, offsets, order)
    assert got[4, 3] == float("inf")
    got[4, 3] = clean[4, 3]
    assert torch.equal(got, clean)
    table = integers(rng, 30, d, dtype=dtype)
    table[0] = float("nan")
    out = A.ivfpq_table_lookup_ex(table, torch.tensor([-1, 30, 0, 29], dtype=torch.int32,
                                                      device="cuda"), scale=0.0)
    assert (out[:2] == 0).all() and out[2].isnan().all() and (out[3] == 0).all()


def test_results_repeat_and_nothing_else_is_written():
    rng = np.random.default_rng(4)
    for dtype in TYPES:
        for n, rows, d in ((5000, 50, 130), (5000, 300, 520)):
            grad = reals(rng, n, d, dtype=dtype)
            ids = ids_of(rng, n, 1, rows, 0.4)
            offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(ids).cuda(), rows)
            need = A.ivfpq_table_grad_bytes(n, d)
            results = []
            for fill in (0x00, 0xFF):
                ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
                guard = torch.full((rows * d + 64,), 3.0, dtype=dtype, device="cuda")
                results.append(A.ivfpq_table_grad_ex(grad, offsets, order, workspace=ws[:need],
                                                     out=guard[32:-32].view(rows, d)).clone())
                assert (guard[:32] == 3).all() and (guard[-32:] == 3).all()
                assert (ws[need:] == fill).all()
            assert torch.equal(*results)


def test_shapes_and_refusals():
    table = torch.arange(12, device="cuda", dtype=torch.float32).view(4, 3)
    ids = torch.tensor([[1, 3], [0, 7]], dtype=torch.int32, device="cuda")
    out = A.ivfpq_table_lookup_ex(table, ids, scale=2.0)
    assert out.shape == (2, 2, 3) and out[0, 1].tolist() == [18, 20, 22]
    assert A.ivfpq_table_lookup_ex(table, ids[:0]).shape == (0, 2, 3)
    assert A.ivfpq_table_lookup_ex(table, ids[0, 0]).tolist() == [3, 4, 5]
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    order = torch.zeros(4, dtype=torch.int32, device="cuda")
    for call in (lambda: A.ivfpq_table_lookup_ex(table.t(), ids),
                 lambda: A.ivfpq_table_lookup_ex(table, ids.long()),
                 lambda: A.ivfpq_table_lookup_ex(table.view(2, 2, 3), ids),
                 lambda: A.ivfpq_table_grad_ex(table, o, order[:3]),
                 lambda: A.ivfpq_table_grad_ex(table, o[:1], order),
                 lambda: A.ivfpq_table_grad_ex(table, o, order, k=0),
                 lambda: A.ivfpq_table_grad_ex(table, o, order, dtype=torch.float64)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(A.IVFPQError):
        A.ivfpq_table_grad_ex(table, o, order, dtype=torch.float16)
    empty = torch.empty((0, 3), device="cuda")
    assert (A.ivfpq_table_grad_ex(empty, o, order[:0]) == 0).all()


def test_sums_of_the_lists_vectors():
    """With vectors in the place of the gradient: the sums that k-means divides."""
    rng = np.random.default_rng(9)
    x = integers(rng, 700, 33, dtype=torch.float32)
    lists = rng.integers(0, 12, (700, 2)).astype(np.int32)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(lists).cuda(), 12)
    got = A.ivfpq_table_grad_ex(x, offsets, order, k=2)
    want, _ = R.table_gradient(np64(x), lists, 12, 1.0)
    assert np.array_equal(np64(got), want)


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -1.0])
@pytest.mark.parametrize("d", [5, 40, 520])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_are_not_there_are_zero_whatever_the_factor(dtype, d, scale):
    table = torch.ones((9, d), dtype=dtype, device="cuda")
    ids = torch.tensor([-1, 9, 3, 2 ** 31 - 1, 0, -7], dtype=torch.int32, device="cuda")
    out = A.ivfpq_table_lookup_ex(table, ids, scale=scale)
    want = torch.zeros((6, d), dtype=dtype)
    want[[2, 4]] = scale
    assert torch.equal(out.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
    # lists 0, 3 and 8 have one row each, 5 a long one, the others none
    ids = torch.full((400,), 5, dtype=torch.int32)
    ids[:4] = torch.tensor([0, 3, 8, -1])
    offsets, order, _ = A.ivfpq_route_sort_ex(ids.view(-1, 1).cuda(), 9)
    got = A.ivfpq_table_grad_ex(torch.ones((400, d), dtype=dtype, device="cuda"), offsets, order,
                                scale=scale)
    want = torch.zeros((9, d), dtype=dtype)
    want[[0, 3, 8]], want[5] = scale, 396 * scale
    assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
