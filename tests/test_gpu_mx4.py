"""4-bit rows and their products on the GPU against the 64-bit definitions of
oracle/rows.py.

Tolerances.  Codes, scales and the values they stand for are exact.  A product
of two codes is exact in float32 and a row has K = 32 kb of them, so a float32
sum in any order is within K * 2^-23 * sum |a b| of the exact one (2^-23, not
2^-24: the matrix cores may truncate inside a step); storing it rounds once
more by the unit of the type (2^-24, 2^-8, 2^-11 of the result, and half the
smallest step of a binary16).
"""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = list(UNIT)


def np64(t):
    return t.detach().cpu().double().numpy()


def random_rows(rng, n, d):
    x = rng.standard_normal((n, d)) * np.exp(rng.standard_normal((n, 1)))
    x[:, rng.random(d) < 0.05] *= 16.0
    return x.astype(np.float32)


def random_mx4(rng, n, d, spread=3):
    """Any codes, scales around 127 (a padded tail stays zero)."""
    kb = -(-d // 32)
    codes = rng.integers(0, 256, size=(n, 16 * kb)).astype(np.uint8)
    if d % 32:
        codes[:, (d + 1) // 2:] = 0
        if d % 2:
            codes[:, d // 2] &= 15
    scales = rng.integers(127 - spread, 128 + spread, size=(n, kb)).astype(np.uint8)
    return codes, scales


def cuda(pair):
    return tuple(torch.from_numpy(a).cuda() for a in pair)


def check_product(out, exact, mag, d, dtype):
    k = 32 * (-(-d // 32))
    tol = (k * 2.0 ** -23 * mag) * (1 + UNIT[dtype]) + UNIT[dtype] * np.abs(exact)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(np64(out) - exact)
    assert (err <= tol).all(), (float((err - tol).max()), np.unravel_index(
        (err - tol).argmax(), err.shape))


# --- rows to 4 bits ---------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 96), (33, 100), (1, 4099),
                                 (64, 257), (129, 8)])
def test_quantize(dtype, n, d):
    rng = np.random.default_rng(n * 1000 + d)
    x = torch.from_numpy(random_rows(rng, n, d)).to(dtype).cuda()
    codes, scales = A.ivfpq_mx4_quantize_ex(x)
    c, s = R.quantize(np64(x))
    assert np.array_equal(scales.cpu().numpy(), s)
    v = R.values(c, s, d)
    assert np.array_equal(R.values(codes.cpu().numpy(), s, 32 * s.shape[1])[:, :d], v)
    assert (R.values(codes.cpu().numpy(), s, 32 * s.shape[1])[:, d:] == 0).all()
    for out in TYPES:
        back = A.ivfpq_mx4_dequantize_ex(codes, scales, d, dtype=out)
        want = torch.from_numpy(v).to(out)   # float16 rounds, the others are exact
        assert torch.equal(back.cpu() + 0.0, want + 0.0)


def test_quantize_every_boundary_and_halfway():
    # magnitudes 0, 1/16, 2/16 .. 8 around an anchor that fixes the scale
    grid = np.arange(0, 129) / 16.0
    for e in (-100, -3, 0, 5, 90):
        x = np.zeros((2 * len(grid), 32), np.float32)
        x[:, 0] = 4.0 * 2.0 ** e
        x[:len(grid), 7] = grid * 2.0 ** e
        x[len(grid):, 30] = -grid * 2.0 ** e
        t = torch.from_numpy(x).cuda()
        codes, scales = A.ivfpq_mx4_quantize_ex(t)
        c, s = R.quantize(x)
        assert np.array_equal(scales.cpu().numpy(), s)
        assert np.array_equal(A.ivfpq_mx4_dequantize_ex(codes, scales, 32).cpu().numpy(),
                              R.values(c, s, 32).astype(np.float32))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_values(dtype):
    tiny = float(torch.finfo(dtype).tiny)
    big = float(torch.finfo(dtype).max)
    x = torch.zeros((10, 64), dtype=dtype)
    x[0, 5] = float("nan")
    x[1, 6], x[1, 40] = float("inf"), 1.0
    x[2, 63] = -float("inf")
    x[3, 1], x[3, 2] = big, -big / 2
    x[4, 1], x[4, 2] = tiny, -tiny / 2
    x[5, 1] = tiny / 8                       # subnormal alone
    x[6, :32] = -0.0
    x[7] = big
    x[8] = tiny / 2
    codes, scales = A.ivfpq_mx4_quantize_ex(x.cuda())
    c, s = R.quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    back = A.ivfpq_mx4_dequantize_ex(codes, scales, 64).cpu().numpy()
    assert np.array_equal(back, R.values(c, s, 64).astype(np.float32), equal_nan=True)
    assert (codes.cpu().numpy()[0, :16] == 0).all() and scales[0, 0] == 255


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_views(dtype):
    rng = np.random.default_rng(5)
    base = torch.from_numpy(random_rows(rng, 40, 210)).to(dtype).cuda()
    for view in (base[:, 3:150], base[::3], base[1:2], base[:, 7:8], base[5:6].expand(4, 210)):
        codes, scales = A.ivfpq_mx4_quantize_ex(view)
        want = A.ivfpq_mx4_quantize_ex(view.contiguous())
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("d", [32, 96, 128, 160])
def test_dequantize_every_code_and_scale(d):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, d // 2)[:, :d // 2].contiguous()
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, d // 32).contiguous()
    out = A.ivfpq_mx4_dequantize_ex(codes.cuda(), scales.cuda(), d).cpu().numpy()
    with np.errstate(over="ignore"):   # the largest scales pass float32's range
        want = R.values(codes.numpy(), scales.numpy(), d).astype(np.float32)
    assert np.array_equal(out, want, equal_nan=True)


# --- product ----------------------------------------------------------------

@pytest.mark.parametrize("m,n,d", [
    (1, 1, 1), (1, 16, 32), (1, 300, 4096), (3, 31, 33), (16, 64, 128), (17, 65, 129),
    (33, 257, 500), (64, 5, 96), (130, 131, 1000), (255, 300, 2049), (257, 513, 64),
    (300, 520, 544), (512, 512, 1024), (700, 40, 256), (2, 4100, 70), (8, 1024, 8192)])
@pytest.mark.parametrize("dtype", TYPES)
def test_product(m, n, d, dtype):
    rng = np.random.default_rng(m * 7 + n * 3 + d)
    a, b = random_mx4(rng, m, d), random_mx4(rng, n, d)
    if dtype == torch.float16:   # keep sums of up to 8192 products below 65504
        a = (a[0], (a[1] - 8).astype(np.uint8))
    va, vb = R.values(*a, d), R.values(*b, d)
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b), dtype=dtype)
    check_product(out, va @ vb.T, np.abs(va) @ np.abs(vb).T, d, dtype)


@pytest.mark.parametrize("m,n,d", [
    (200, 2500, 2080), (130, 1000, 8192), (65, 1700, 8200), (1000, 1030, 2113), (17, 8200, 4100)])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_of_few_tiles_of_long_rows(m, n, d, dtype):
    test_product(m, n, d, dtype)


# tiles of 128 x 128; of 256 x 256; runs of those along n (an even number of chunks)
@pytest.mark.parametrize("m,n,d", [
    (1300, 4100, 1100), (2600, 4200, 1100), (4200, 8200, 512), (2570, 8203, 1024)])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_of_many_tiles(m, n, d, dtype):
    rng = np.random.default_rng(m + n + d)
    a, b = random_mx4(rng, m, d), random_mx4(rng, n, d)
    if dtype == torch.float16:
        a = (a[0], (a[1] - 8).astype(np.uint8))
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b), dtype=dtype)
    rows = np.unique(np.r_[0:m:41, m - 9:m])
    va, vb = R.values(a[0][rows], a[1][rows], d), R.values(*b, d)
    check_product(out[torch.from_numpy(rows).cuda()], va @ vb.T, np.abs(va) @ np.abs(vb).T, d,
                  dtype)
    # every row: its sum against the product with the columns' sum
    total = R.values(*a, d) @ vb.sum(axis=0)
    mag = np.abs(R.values(*a, d)) @ np.abs(vb).sum(axis=0)
    err = np.abs(np64(out.double().sum(dim=1)) - total)
    assert (err <= mag * (d * 2.0 ** -22 + 2 * UNIT[dtype]) + n * 2.0 ** -25).all()


def test_product_nan_in_each_chunk_of_long_rows():
    rng = np.random.default_rng(16)
    m, n, d = 140, 1500, 2592                    # 81 blocks, the last of them alone in its chunk
    a, b = random_mx4(rng, m, d), random_mx4(rng, n, d)
    for row, block in enumerate(range(0, 81)):
        a[1][row, block] = 255
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b)).cpu().numpy()
    assert np.isnan(out[:81]).all() and np.isfinite(out[81:]).all()


def test_product_blocks_land_where_they_belong():
    # one block of one row at a time set: catches any permutation of rows,
    # blocks, nibbles or scales
    d, m, n = 544, 48, 40
    kb = d // 32
    rng = np.random.default_rng(9)
    b = random_mx4(rng, n, d, spread=20)
    a = (np.zeros((m, 16 * kb), np.uint8), np.full((m, kb), 127, np.uint8))
    for i in range(m):
        k = (i * 37) % d
        a[0][i, k // 2] = 2 << (4 * (k % 2))       # a one
        a[1][i] = 100 + np.arange(kb)
    va, vb = R.values(*a, d), R.values(*b, d)
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b)).cpu().numpy()
    assert np.array_equal(out, (va @ vb.T).astype(np.float32))


@pytest.mark.parametrize("m,n,d", [(2, 20, 64), (40, 600, 320), (300, 300, 512)])
def test_product_nan_and_zero_blocks(m, n, d):
    rng = np.random.default_rng(11)
    a, b = random_mx4(rng, m, d), random_mx4(rng, n, d)
    a[0][m - 1] = 0
    a[1][m - 1] = 0                       # a row of zeros at the smallest scale
    a[1][0, d // 32 - 1] = 255            # a NaN block in the first row
    b[1][n - 2, 0] = 255
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b)).cpu().numpy()
    nan = np.zeros((m, n), bool)
    nan[0], nan[:, n - 2] = True, True
    assert np.isnan(out[nan]).all()
    assert np.isfinite(out[~nan]).all()
    last = np.delete(out[m - 1], n - 2)
    assert (last == 0).all()


def test_product_extreme_scales():
    # 2^(s_a + s_b - 254) far from the middle, results still ordinary floats
    rng = np.random.default_rng(12)
    a, b = random_mx4(rng, 20, 128), random_mx4(rng, 24, 128)
    a, b = (a[0], np.full_like(a[1], 250)), (b[0], np.full_like(b[1], 3))
    va, vb = R.values(*a, 128), R.values(*b, 128)
    out = A.ivfpq_mx4_product_ex(cuda(a), cuda(b))
    check_product(out, va @ vb.T, np.abs(va) @ np.abs(vb).T, 128, torch.float32)


def test_product_empty_and_reused_outputs():
    rng = np.random.default_rng(13)
    a, b = cuda(random_mx4(rng, 5, 64)), cuda(random_mx4(rng, 9, 64))
    empty = (a[0][:0], a[1][:0])
    assert A.ivfpq_mx4_product_ex(empty, b).shape == (0, 9)
    assert A.ivfpq_mx4_product_ex(a, (b[0][:0], b[1][:0])).shape == (5, 0)
    assert A.ivfpq_mx4_quantize_ex(torch.empty((0, 40), device="cuda"))[0].shape == (0, 32)
    out = torch.full((5, 9), 7.0, device="cuda")
    want = A.ivfpq_mx4_product_ex(a, b)
    assert A.ivfpq_mx4_product_ex(a, b, out=out) is out and torch.equal(out, want)


def test_product_past_32_bit_offsets():
    # operands above 4 GiB and an output above 2^31 elements: the last rows
    d, n = 4096, (1 << 21) + 300
    g = torch.Generator(device="cuda").manual_seed(3)
    bc = torch.randint(0, 256, (n, 16 * (d // 32)), generator=g, device="cuda", dtype=torch.uint8)
    bs = torch.full((n, d // 32), 120, device="cuda", dtype=torch.uint8)
    rng = np.random.default_rng(14)
    a = random_mx4(rng, 2, d)
    out = A.ivfpq_mx4_product_ex(cuda(a), (bc, bs))
    tail = slice(n - 50, n)
    va = R.values(*a, d)
    vb = R.values(bc[tail].cpu().numpy(), bs[tail].cpu().numpy(), d)
    check_product(out[:, tail], va @ vb.T, np.abs(va) @ np.abs(vb).T, d, torch.float32)
    wide = A.ivfpq_mx4_product_ex((bc, bs), cuda(a))
    assert torch.equal(wide[tail], out[:, tail].t())
    del out, wide
    # few blocks, many results
    m = 1100
    a = random_mx4(rng, m, 32)
    small = (bc[:, :16].contiguous(), bs[:, :1].contiguous())
    out = A.ivfpq_mx4_product_ex(cuda(a), small, dtype=torch.float16)
    vb = R.values(small[0][tail].cpu().numpy(), small[1][tail].cpu().numpy(), 32)
    va = R.values(*a, 32)
    check_product(out[:, tail][-20:], va[-20:] @ vb.T, np.abs(va[-20:]) @ np.abs(vb).T, 32,
                  torch.float16)


def test_product_past_the_threads_of_one_launch():
    n = (1 << 30) + 300                           # 2^32 threads and some
    bc = torch.full((n, 16), 0x22, device="cuda", dtype=torch.uint8)  # ones
    bs = torch.full((n, 1), 127, device="cuda", dtype=torch.uint8)
    bs[-300:] = 128
    a = random_mx4(np.random.default_rng(15), 1, 32)
    out = A.ivfpq_mx4_product_ex(cuda(a), (bc, bs), dtype=torch.float32)
    want = float(R.values(*a, 32).sum())          # sums of small multiples of a power of two
    assert (out[0, :-300] == want).all() and (out[0, -300:] == 2 * want).all()


# --- product per list -------------------------------------------------------

def make_lists(rng, t, k, nlist, drop, hot=None):
    lists = np.stack([rng.choice(nlist, size=k, replace=False) for _ in range(t)]).astype(np.int32)
    if hot is not None:
        lists[:, 0] = hot
    lists[rng.random((t, k)) < drop] = -1
    return lists


@pytest.mark.parametrize("t,k,nlist,n,d,drop", [
    (1, 1, 1, 16, 32, 0.0), (1, 2, 8, 33, 70, 0.0), (5, 2, 4, 130, 128, 0.2),
    (40, 4, 70, 65, 96, 0.1), (300, 2, 3, 257, 256, 0.0), (600, 1, 2, 512, 544, 0.05),
    (513, 3, 130, 48, 64, 0.3), (20, 2, 8, 40, 1000, 1.0), (130, 2, 3, 200, 2300, 0.1)])
@pytest.mark.parametrize("dtype", TYPES)
def test_list_product(t, k, nlist, n, d, drop, dtype):
    rng = np.random.default_rng(t + 10 * k + 100 * nlist + n)
    lists = make_lists(rng, t, k, nlist, drop)
    offsets, order, _ = R.route_sort(lists, nlist)
    a = random_mx4(rng, t, d)
    bc, bs = random_mx4(rng, nlist * n, d)
    b = (bc.reshape(nlist, n, -1), bs.reshape(nlist, n, -1))
    if dtype == torch.float16:
        a = (a[0], (a[1] - 6).astype(np.uint8))
    va, vb = R.values(*a, d), R.values(*b, d)
    exact, mag = R.list_product(va, vb, offsets, order, k, t * k)
    off, orde = torch.from_numpy(offsets).cuda(), torch.from_numpy(order).cuda()
    out = A.ivfpq_mx4_list_product_ex(cuda(a), cuda(b), off, order=orde, k=k, dtype=dtype)
    check_product(out, exact, mag, d, dtype)
    assert (np64(out)[offsets[nlist]:] == 0).all()
    # rows already in list order: the same results
    src = np.where(order >= 0, order // k, 0)
    sorted_a = (a[0][src], a[1][src])
    again = A.ivfpq_mx4_list_product_ex(cuda(sorted_a), cuda(b), off, dtype=dtype)
    assert torch.equal(again, out)


@pytest.mark.parametrize("t,nlist,n,d", [
    (1650, 3, 4200, 512), (2500, 5, 2100, 544), (1000, 40, 1100, 1030)])
@pytest.mark.parametrize("dtype", TYPES)
def test_list_product_of_many_tiles(t, nlist, n, d, dtype):
    rng = np.random.default_rng(t + nlist + n)
    lists = make_lists(rng, t, 2, nlist, 0.02)
    offsets, order, _ = R.route_sort(lists, nlist)
    a = random_mx4(rng, t, d)
    bc, bs = random_mx4(rng, nlist * n, d)
    b = (bc.reshape(nlist, n, -1), bs.reshape(nlist, n, -1))
    if dtype == torch.float16:
        a = (a[0], (a[1] - 8).astype(np.uint8))
    off, orde = torch.from_numpy(offsets).cuda(), torch.from_numpy(order).cuda()
    out = A.ivfpq_mx4_list_product_ex(cuda(a), cuda(b), off, order=orde, k=2, dtype=dtype)
    va, vb = R.values(*a, d), R.values(*b, d)
    for e in range(nlist):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        rows = np.unique(np.r_[lo:hi:17, max(lo, hi - 5):hi])
        x = va[order[rows] // 2]
        check_product(out[torch.from_numpy(rows).cuda()], x @ vb[e].T, np.abs(x) @ np.abs(vb[e]).T,
                      d, dtype)
    assert (out[offsets[nlist]:] == 0).all()


def test_list_product_one_list_takes_all():
    rng = np.random.default_rng(21)
    t, nlist, n, d = 700, 200, 96, 128
    lists = np.full((t, 1), 199, np.int32)
    lists[::7] = 0
    offsets, order, _ = R.route_sort(lists, nlist)
    a = random_mx4(rng, t, d)
    bc, bs = random_mx4(rng, nlist * n, d)
    b = (bc.reshape(nlist, n, -1), bs.reshape(nlist, n, -1))
    exact, mag = R.list_product(R.values(*a, d), R.values(*b, d), offsets, order, 1, t)
    out = A.ivfpq_mx4_list_product_ex(cuda(a), cuda(b), torch.from_numpy(offsets).cuda(),
                                      order=torch.from_numpy(order).cuda())
    check_product(out, exact, mag, d, torch.float32)


# --- streams and graphs -----------------------------------------------------

def test_other_stream_and_graph_replays():
    rng = np.random.default_rng(31)
    t, k, nlist, n, d = 48, 2, 6, 64, 160
    w = cuda(random_mx4(rng, nlist * n, d))
    w = (w[0].view(nlist, n, -1), w[1].view(nlist, n, -1))
    x = torch.empty((t, d), device="cuda", dtype=torch.bfloat16)
    lists = torch.empty((t, k), device="cuda", dtype=torch.int32)
    gate = torch.empty((t, k), device="cuda")

    def layer():
        offsets, order, pos = A.ivfpq_route_sort_ex(lists, nlist)
        a = A.ivfpq_mx4_quantize_ex(x)
        h = A.ivfpq_mx4_list_product_ex(a, w, offsets, order=order, k=k, dtype=torch.bfloat16)
        return A.ivfpq_route_combine_ex(h, pos, gate)

    def fill(seed):
        r = np.random.default_rng(seed)
        x.copy_(torch.from_numpy(random_rows(r, t, d)))
        lists.copy_(torch.from_numpy(make_lists(r, t, k, nlist, 0.1)))
        gate.copy_(torch.from_numpy(r.random((t, k)).astype(np.float32)))

    fill(0)
    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
        layer()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for seed in range(1, 5):
        fill(seed)
        want = layer()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want), seed
