"""Products per list, adapters and table rows whose operands pass 2^31 and 2^32
elements: the far end is read and written where it should be."""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from test_gpu_list_product import integers, np64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def cuda(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_table_rows():
    rows, d = (1 << 21) + 3, 2100                      # 4.4e9 elements
    rng = np.random.default_rng(1)
    table = torch.empty((rows, d), dtype=BF, device="cuda")
    at = [0, 1, 1 << 20, rows - 2, rows - 1]
    values = integers(rng, len(at), d, dtype=BF)
    table[at] = values
    assert torch.equal(A.ivfpq_table_lookup_ex(table, cuda(*at, rows), scale=2.0),
                       torch.cat([values * 2, torch.zeros_like(values[:1])]))
    offsets, order, _ = A.ivfpq_route_sort_ex(cuda(*at, rows).view(-1, 1), rows)
    grad = torch.cat([values, values[:1]])
    table.fill_(7)
    got = A.ivfpq_table_grad_ex(grad, offsets, order, out=table)
    assert torch.equal(got[at], values)
    got[at] = 0
    for part in got.split(1 << 19):
        assert not part.any()


@pytest.mark.parametrize("d", [264, 263])
def test_matrices(d):
    nlist, n = 1 << 16, 258                            # 4.4e9 elements
    rng = np.random.default_rng(d)
    matrices = torch.zeros((nlist, n, d), dtype=BF, device="cuda")
    used = [0, 1, nlist // 2, nlist - 1]
    matrices[used] = integers(rng, 4, n, d, dtype=BF)
    w = np64(matrices[used])
    lists = cuda(0, nlist - 1, 1, nlist - 1, nlist // 2, -1).view(-1, 1)
    offsets, order, pos = A.ivfpq_route_sort_ex(lists, nlist)
    where = [used.index(e) for e in lists.view(-1).tolist()[:5]]
    x = integers(rng, 6, d, dtype=BF)
    y = A.ivfpq_route_combine_ex(A.ivfpq_list_product_ex(x, matrices, offsets, order=order), pos)
    want = np.stack([w[e] @ np64(x)[i] for i, e in enumerate(where)] + [np.zeros(n)])
    assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(BF)))
    g = integers(rng, 6, n, dtype=BF)
    y = A.ivfpq_route_combine_ex(
        A.ivfpq_list_product_ex(g, matrices, offsets, order=order, transposed=True), pos)
    want = np.stack([w[e].T @ np64(g)[i] for i, e in enumerate(where)] + [np.zeros(d)])
    assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(BF)))
    matrices.fill_(7)
    got = A.ivfpq_list_product_grad_ex(A.ivfpq_route_gather_ex(g, order, 1), x, offsets, order=order,
                                       out=matrices)
    for i, e in enumerate(used):
        mine = [r for r in range(5) if where[r] == i]
        assert np.array_equal(np64(got[e]), np64(g)[mine].T @ np64(x)[mine])
        got[e] = 0
    for part in got.split(1 << 13):
        assert not part.any()


@pytest.mark.parametrize("d", [2048, 2047])
def test_rows(d):
    rows, n, r = 1_100_000, 24, 8                      # 2.25e9 elements
    rng = np.random.default_rng(d)
    x = torch.zeros((rows, d), dtype=BF, device="cuda")
    at = [0, rows // 2, rows - 2, rows - 1]
    x[at] = integers(rng, 4, d, dtype=BF)
    w = integers(rng, 1, n, d, dtype=BF)
    want = torch.from_numpy(np64(x[at]) @ np64(w[0]).T).to(BF).cuda()
    one = cuda(0, rows)
    order = torch.arange(rows, dtype=torch.int32, device="cuda")
    for sorting in (None, order):
        y = A.ivfpq_list_product_ex(x, w, one, order=sorting)
        assert torch.equal(y[at], want)
        y[at] = 0
        assert not y.any()
        y[at] = integers(rng, 4, n, dtype=BF)
        grad = A.ivfpq_list_product_grad_ex(y, x, one, order=sorting, dtype=torch.float32)
        assert np.array_equal(np64(grad[0]), np64(y[at]).T @ np64(x[at]))
    down, up = integers(rng, 1, r, d, dtype=BF), integers(rng, 1, n, r, dtype=BF)
    offsets = cuda(rows // 2, rows)                    # the first half of no list
    pos = torch.where(order >= rows // 2, order, -1)
    order = torch.where(order >= rows // 2, order, -1)
    y = A.ivfpq_adapter_product_ex(x, w[0], down, up, offsets, order, pos)
    exact = np64(x[at]) @ np64(w[0]).T
    exact[1:] += np64(x[at[1:]]) @ np64(down[0]).T @ np64(up[0]).T
    # the hidden rows are sums of d products of up to 9, exact in two parts of 8 bits
    assert np.array_equal(np64(y[at]), np64(torch.from_numpy(exact).to(BF)))
    y[at] = 0
    assert not y.any()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("n,d", [(3, 1 << 20), (1 << 20, 3), (8, (1 << 20) - 1)])
def test_the_widest_rows(n, d, dtype):
    rng = np.random.default_rng(n)
    x, w = integers(rng, 5, d, dtype=dtype, top=1), integers(rng, 2, n, d, dtype=dtype, top=1)
    offsets, order = cuda(0, 2, 5), cuda(4, 0, 2, 2, 1)
    y = A.ivfpq_list_product_ex(x, w, offsets, order=order)
    rows = np64(x)[order.tolist()]
    want = np.concatenate([rows[:2] @ np64(w[0]).T, rows[2:] @ np64(w[1]).T])
    assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(dtype)))
    wt = w.transpose(1, 2).contiguous()
    assert torch.equal(A.ivfpq_list_product_ex(x, wt, offsets, order=order, transposed=True), y)
    g = integers(rng, 5, n, dtype=dtype, top=1)
    got = A.ivfpq_list_product_grad_ex(g, x, offsets, order=order, dtype=torch.float32)
    for e, (lo, hi) in enumerate(((0, 2), (2, 5))):
        assert np.array_equal(np64(got[e]), np64(g)[lo:hi].T @ rows[lo:hi])
    offsets, order, pos = A.ivfpq_route_sort_ex(cuda(1, -1, 0, 1, 1).view(-1, 1), 2)
    grad = A.ivfpq_table_grad_ex(x, offsets, order, dtype=torch.float32)
    assert np.array_equal(np64(grad), np.stack([np64(x)[2], np64(x)[[0, 3, 4]].sum(0)]))
    assert torch.equal(A.ivfpq_table_lookup_ex(x, cuda(4, 9)), torch.stack([x[4], x[4] * 0]))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("t", [3, 100, 300])
def test_the_highest_rank(t, dtype):
    n, d, r, nlist = 600, 64, 1 << 12, 3
    rng = np.random.default_rng(t)
    x, w = integers(rng, t, d, dtype=dtype, top=1), integers(rng, n, d, dtype=dtype, top=1)
    down = integers(rng, nlist, r, d, dtype=dtype, top=1)
    up = integers(rng, nlist, n, r, dtype=dtype, top=1)
    lists = rng.integers(-1, nlist, t)
    y = A.ivfpq_adapter_product_ex(x, w, down, up, *A.ivfpq_route_sort_ex(
        torch.from_numpy(lists[:, None].astype(np.int32)).cuda(), nlist))
    want = np64(x) @ np64(w).T
    for e in range(nlist):
        mine = lists == e
        want[mine] += np64(x)[mine] @ np64(down[e]).T @ np64(up[e]).T
    assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(dtype)))


@pytest.mark.parametrize("t,d,r", [(20, 64, 64), (600, 64, 64), (600, 63, 63)])
def test_up_matrices(t, d, r):
    nlist, n = 1 << 16, 600                            # 2.5e9 elements
    rng = np.random.default_rng(r)
    up = torch.zeros((nlist, n, r), dtype=BF, device="cuda")
    down = torch.zeros((nlist, r, d), dtype=BF, device="cuda")
    used = [0, 1, nlist // 2, nlist - 2, nlist - 1]
    up[used], down[used] = (integers(rng, 5, n, r, dtype=BF, top=1),
                            integers(rng, 5, r, d, dtype=BF, top=1))
    x, w = integers(rng, t, d, dtype=BF), integers(rng, n, d, dtype=BF)
    pick = rng.integers(-1, 5, t)
    lists = np.where(pick < 0, -1, np.array(used)[pick]).astype(np.int32)
    y = A.ivfpq_adapter_product_ex(x, w, down, up, *A.ivfpq_route_sort_ex(
        torch.from_numpy(lists[:, None]).cuda(), nlist))
    want = np64(x) @ np64(w).T
    for i, e in enumerate(used):
        mine = pick == i
        want[mine] += np64(x)[mine] @ np64(down[e]).T @ np64(up[e]).T
    assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(BF)))
