"""The tiled kernels of the 4-bit products at their edges, against the 64-bit
definitions of oracle/rows.py.  Tolerances are those of test_gpu_mx4.py: codes
multiply exactly, a float32 sum of K products is within K 2^-23 of the sum of
their magnitudes, and storing rounds once by the unit of the type."""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R
from test_gpu_mx4 import TYPES, cuda, make_lists, random_mx4

pytestmark = pytest.mark.gpu

# A product for each kernel and edge: (kernel, m, n, d).  test_mx4_plan.py checks
# without a GPU that each takes the kernel named here.
PRODUCTS = [
    ("direct1", 130, 131, 500), ("direct4", 33, 4097, 1000), ("direct8", 16, 515, 2100),
    ("one", 1301, 13001, 33), ("one", 1301, 8703, 96), ("one", 515, 8001, 250),
    ("one", 517, 8003, 256),
    ("small", 1025, 3713, 320),        # two chunks, one column in the last tile
    ("small", 705, 2311, 700),         # three, seven columns
    ("small", 321, 2311, 2000),        # eight
    ("shared", 129, 3009, 2592),       # 81 blocks, the last alone in its chunk
    ("shared", 193, 2369, 2209), ("shared", 300, 1025, 8192),
    ("middle", 1301, 4103, 1030), ("middle", 1283, 4103, 1500),
    ("large", 2570, 8203, 544), ("large", 2570, 8203, 1024)]
# and for lists: (kernel, t, k, nlist, n, d)
LIST_PRODUCTS = [
    ("direct1", 60, 2, 70, 65, 96), ("direct1", 5, 1, 1, 40, 32), ("direct4", 40, 2, 50, 300, 700),
    ("direct8", 4, 2, 5, 300, 2400),
    ("small", 300, 2, 3, 257, 256), ("small", 700, 2, 9, 129, 800),
    ("shared", 130, 2, 3, 200, 2300), ("shared", 200, 2, 5, 330, 4096),
    ("middle", 2600, 2, 20, 2049, 544), ("middle", 1500, 2, 9, 2055, 1030),
    ("large", 1650, 2, 3, 4200, 512), ("large", 1700, 2, 3, 4103, 544)]
# parts [e0, e1) of the lists, two a vector: (kernel, t, nlist, n, d, e0, e1)
LIST_PARTS = [
    ("direct1", 9, 16, 100, 96, 5, 15), ("small", 300, 8, 70, 64, 3, 8),
    ("small", 50, 6, 40, 64, 3, 4), ("shared", 200, 5, 330, 2300, 2, 4),
    ("middle", 2600, 5, 1100, 512, 1, 2), ("middle", 1500, 5, 2055, 1030, 1, 4),
    ("large", 2600, 5, 4100, 512, 1, 4)]


def one_of_each(cases):
    """The first case of each kernel."""
    first = {}
    for c in cases:
        first.setdefault(c[0], c)
    return list(first.values())



def operands(rng, m, n, d, dtype, nlist=None, spread=3):
    a, b = random_mx4(rng, m, d, spread), random_mx4(rng, (nlist or 1) * n, d, spread)
    if dtype == torch.float16:   # keep sums of up to 8192 products below 65504
        a = (a[0], (a[1] - 8).astype(np.uint8))
    if nlist:
        b = tuple(t.reshape(nlist, n, -1) for t in b)
    return a, b


def routed(rng, t, k, nlist, drop=0.05):
    offsets, order, _ = R.route_sort(make_lists(rng, t, k, nlist, drop), nlist)
    return offsets, order, k


def product(a, b, dtype, route=None):
    """The library's result of a product, of lists with route = (offsets, order, k)."""
    if route is None:
        return A.ivfpq_mx4_product_ex(cuda(a), cuda(b), dtype=dtype)
    offsets, order, k = route
    return A.ivfpq_mx4_list_product_ex(cuda(a), cuda(b), torch.from_numpy(offsets).cuda(),
                                       order=torch.from_numpy(order).cuda(), k=k, dtype=dtype)


def parts(va, vb, route):
    """(output rows, first operand, second operand) of each matrix."""
    if route is None:
        yield slice(0, len(va)), va, vb
        return
    offsets, order, k = route
    for e in range(len(vb)):
        span = slice(int(offsets[e]), int(offsets[e + 1]))
        if span.start < span.stop:
            yield span, va[order[span] // k], vb[e]


def check(out, a, b, d, dtype, route=None):
    """Every result against its definition (the values of oracle/rows.py, multiplied in 64 bits)."""
    va, vb = R.values(*a, d), R.values(*b, d)
    terms, unit = 32 * (-(-d // 32)), {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8,
                                       torch.float16: 2.0 ** -11}[dtype]
    for rows, x, w in parts(va, vb, route):
        x, w = torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda()
        exact, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
        tol = terms * 2.0 ** -23 * mag * (1 + unit) + unit * exact.abs()
        if dtype == torch.float16:
            tol += 2.0 ** -25
        err = (out[rows].double() - exact).abs()
        assert (err <= tol).all(), (rows, (err - tol).argmax())
    if route is not None:
        assert (out[int(route[0][-1]):] == 0).all()


@pytest.mark.parametrize("kernel,m,n,d", PRODUCTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_product_of_each_kernel(kernel, m, n, d, dtype):
    a, b = operands(np.random.default_rng(m + n + d), m, n, d, dtype)
    check(product(a, b, dtype), a, b, d, dtype)


@pytest.mark.parametrize("kernel,t,k,nlist,n,d", LIST_PRODUCTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_list_product_of_each_kernel(kernel, t, k, nlist, n, d, dtype):
    rng = np.random.default_rng(t + nlist + n + d)
    route = routed(rng, t, k, nlist)
    a, b = operands(rng, t, n, d, dtype, nlist)
    check(product(a, b, dtype, route), a, b, d, dtype, route)


# The same special operands through every kernel, whole and per list.
EACH = [c[1:] for c in one_of_each(PRODUCTS)] + [c[1:] for c in one_of_each(LIST_PRODUCTS)]


def each_case(shape, dtype, spread=3):
    rng = np.random.default_rng(sum(shape))
    if len(shape) == 3:
        m, n, d = shape
        return (rng, d, None, *operands(rng, m, n, d, dtype, spread=spread))
    t, k, nlist, n, d = shape
    return (rng, d, routed(rng, t, k, nlist), *operands(rng, t, n, d, dtype, nlist, spread))


@pytest.mark.parametrize("shape", EACH)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_blocks_land_where_they_belong_in_each_kernel(shape, dtype):
    # a single one in each row of the first operand: results are the second one's
    # values at its place, times a power of two, exactly
    rng, d, route, a, b = each_case(shape, dtype, spread=20)
    kb = a[1].shape[1]
    a[0][:], a[1][:] = 0, 100 + np.arange(kb) % 50
    for i in range(len(a[0])):
        c = (i * 37) % d
        a[0][i, c // 2] = 2 << (4 * (c % 2))
    out = product(a, b, dtype, route)
    va, vb = R.values(*a, d), R.values(*b, d)
    for rows, x, w in parts(va, vb, route):
        c = np.abs(x).argmax(axis=1)
        want = (w[:, c] * x[np.arange(len(x)), c]).T
        assert torch.equal(out[rows], torch.from_numpy(want).to(dtype).cuda())


@pytest.mark.parametrize("shape", EACH)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_nan_blocks_in_each_kernel(shape, dtype):
    # one NaN block in every third row of the first operand and in some of the
    # second, another block each time
    rng, d, route, a, b = each_case(shape, dtype)
    kb = a[1].shape[1]
    bad_a = np.arange(len(a[0])) % 3 == 0
    a[1][bad_a, np.arange(bad_a.sum()) % kb] = 255
    bs = b[1].reshape(-1, kb)
    bad_b = np.arange(len(bs)) % 29 == 28
    bs[bad_b, np.arange(bad_b.sum())[::-1] % kb] = 255
    out = product(a, b, dtype, route)
    bad_b = bad_b.reshape(b[1].shape[:-1])
    for rows, x, w in parts(bad_a, bad_b, route):
        want = torch.from_numpy(x[:, None] | w[None, :]).cuda()
        assert torch.equal(torch.isnan(out[rows]), want)


@pytest.mark.parametrize("shape", EACH)
def test_extreme_scales_in_each_kernel(shape):
    rng, d, route, a, b = each_case(shape, torch.float32)
    a[1][:], b[1][:] = 250, 3
    check(product(a, b, torch.float32, route), a, b, d, torch.float32, route)
    a[1][:], b[1][:] = 3, 250
    check(product(a, b, torch.float32, route), a, b, d, torch.float32, route)


@pytest.mark.parametrize("nlist,t", [(1000, 3000), (3000, 3500), (1 << 16, 3000)])
def test_list_product_of_many_lists(nlist, t):
    rng = np.random.default_rng(nlist)
    lists = rng.integers(0, nlist, size=(t, 2)).astype(np.int32)
    lists[: t // 3] = nlist - 1                    # one long list, the last
    offsets, order, _ = R.route_sort(lists, nlist)
    a, b = operands(rng, t, 20, 64, torch.float32, nlist)
    check(product(a, b, torch.float32, (offsets, order, 2)), a, b, 64, torch.float32,
          (offsets, order, 2))


def test_list_product_of_rows_past_4_gib():
    # more than the tiles' 32-bit offsets: the direct kernel, however many rows
    t, nlist, n, d = (1 << 20) + 5, 2, 70, 8192
    rng = np.random.default_rng(2)
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 256, (t, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((t, d // 32), 121, device="cuda", dtype=torch.uint8)
    order = rng.integers(0, t, size=600).astype(np.int32)
    order[::50] = t - 1 - np.arange(12)
    offsets = np.array([0, 333, 590], np.int32)
    b = operands(rng, 1, n, d, torch.float32, nlist)[1]
    o = torch.from_numpy(order).cuda()
    out = A.ivfpq_mx4_list_product_ex((codes, scales), cuda(b), torch.from_numpy(offsets).cuda(),
                                      order=o)
    picked = tuple(m[o.long()].cpu().numpy() for m in (codes, scales))
    check(out, picked, b, d, torch.float32, (offsets, np.arange(600), 1))


def test_tiles_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(33)
    t, k, nlist, n, d = 1650, 2, 3, 4200, 512          # large tiles
    w = tuple(m.view(nlist, n, -1) for m in cuda(random_mx4(rng, nlist * n, d)))
    long = cuda(random_mx4(rng, 3000, 2592))           # shared chunks
    short = cuda(random_mx4(rng, 8703, 96))            # single chunks
    x = torch.empty((t, d), device="cuda")
    y = torch.empty((140, 2592), device="cuda", dtype=torch.bfloat16)
    z = torch.empty((1301, 96), device="cuda", dtype=torch.float16)
    lists = torch.empty((t, k), device="cuda", dtype=torch.int32)

    def step():
        offsets, order, _ = A.ivfpq_route_sort_ex(lists, nlist)
        return (A.ivfpq_mx4_list_product_ex(A.ivfpq_mx4_quantize_ex(x), w, offsets, order=order,
                                            k=k, dtype=torch.bfloat16),
                A.ivfpq_mx4_product_ex(A.ivfpq_mx4_quantize_ex(y), long, dtype=torch.float16),
                A.ivfpq_mx4_product_ex(A.ivfpq_mx4_quantize_ex(z), short))

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for v in (x, y, z):
            v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
        lists.copy_(torch.randint(-1, nlist, (t, k), generator=g, device="cuda"))

    def same(got, want):
        return all(torch.equal(p, q) for p, q in zip(got, want))

    fill(0)
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(1, 5):
        fill(seed)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, want), seed


# the last tile has one row of B left and rows end inside a chunk: one block, two
# and a bit chunks, an even number of chunks
@pytest.mark.parametrize("t,nlist,n,d", [(33, 2, 129, 32), (40, 3, 129, 544), (70, 2, 257, 272)])
@pytest.mark.parametrize("dtype", TYPES)
def test_last_matrix_with_one_row_in_its_last_tile(t, nlist, n, d, dtype):
    rng = np.random.default_rng(t + n + d)
    route = routed(rng, t, 2, nlist)
    a, b = operands(rng, t, n, d, dtype, nlist)
    check(product(a, b, dtype, route), a, b, d, dtype, route)


# part of the lists, as where lists are split over devices: the rows of the lists
# before and after are zero, whatever the output held
@pytest.mark.parametrize("kernel,t,nlist,n,d,e0,e1", LIST_PARTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_before_the_first_list_are_zero(kernel, t, nlist, n, d, e0, e1, dtype):
    rng = np.random.default_rng(t + nlist + n + e0)
    offsets, order, _ = R.route_sort(make_lists(rng, t, 2, nlist, 0.05), nlist)
    a, b = operands(rng, t, n, d, dtype, nlist)
    ac, bc, o = cuda(a), cuda(b), torch.from_numpy(order).cuda()
    off = torch.from_numpy(offsets).cuda()
    whole = A.ivfpq_mx4_list_product_ex(ac, bc, off, order=o, k=2, dtype=dtype)
    part = torch.full((2 * t, n), float("nan"), device="cuda", dtype=dtype)
    A.ivfpq_mx4_list_product_ex(ac, tuple(x[e0:e1].contiguous() for x in bc),
                                off[e0:e1 + 1].clone(), order=o, k=2, dtype=dtype, out=part)
    lo, hi = int(offsets[e0]), int(offsets[e1])
    assert 0 < lo < hi < 2 * t
    assert (part[:lo] == 0).all() and (part[hi:] == 0).all()
    # another kernel may take the part than the whole: both against the definition
    check(whole, a, b, d, dtype, (offsets, order, 2))
    check(part, a, tuple(m[e0:e1] for m in b), d, dtype, (offsets[e0:e1 + 1], order, 2))
