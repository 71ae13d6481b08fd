"""Products per list and the gradient of their matrices on the GPU against the 64-bit
definitions of oracle/rows.py.

Tolerances.  Small integers: every product and partial sum is an integer below 2^24
(2^11 and 2^8 parts of the inputs too), so results are exact, rounded once.  Real
values: K exact products added one after the other in float32 take K - 1 additions
that round, each by at most 2^-23 of the sum of the magnitudes however it rounds.  A
float32 product is six part products, so there are 6 K - 1 such additions, of terms
whose magnitudes sum to at most (1 + 2^-8 + 2^-16)^2 < 1 + 2^-6 of the products';
the three dropped parts add 2^-23.  Storing rounds by half a step of the type, or
2^-25 near zero for binary16 and 2^-134 for bfloat16.
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


def integers(rng, *shape, dtype, top=3):
    return torch.from_numpy(rng.integers(-top, top + 1, shape).astype(np.float32)).to(dtype).cuda()


def reals(rng, *shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape)).to(dtype).cuda()


def ragged(rng, rows, nlist, lo=0, hi=None):
    """Offsets of nlist lists between rows lo and hi, some of them empty."""
    hi = rows if hi is None else hi
    cuts = np.sort(rng.integers(lo, hi + 1, nlist - 1)) if nlist > 1 else np.empty(0, int)
    return np.concatenate([[lo], cuts, [hi]]).astype(np.int32)


def list_product64(x, matrices, offsets, rows, source, transposed):
    out = np.zeros((rows, matrices.shape[1] if not transposed else matrices.shape[2]))
    mag = np.zeros_like(out)
    for e, w in enumerate(matrices):
        lo, hi = max(offsets[e], 0), min(offsets[e + 1], rows)
        if lo < hi:
            w = w if transposed else w.T
            out[lo:hi] = x[source[lo:hi]] @ w
            mag[lo:hi] = np.abs(x[source[lo:hi]]) @ np.abs(w)
    return out, mag


def sum_error(terms, dtype):
    """Share of the sum of magnitudes that a float32 sum of so many products is off by."""
    if dtype == torch.float32:
        return (6 * terms - 1) * 2.0 ** -23 * (1 + 2.0 ** -6) + 2.0 ** -23
    return (terms - 1) * 2.0 ** -23


def rounded(exact, dtype):
    return np64(torch.from_numpy(exact).to(dtype))


# rows, lists, n, d: one row and one value, tiles' edges, odd sizes, many lists of few
# rows, lists longer than any tile
SHAPES = [(1, 1, 1, 1), (3, 1, 5, 7), (16, 2, 16, 32), (17, 3, 33, 31), (64, 1, 64, 64),
          (65, 4, 129, 65), (127, 2, 128, 100), (128, 1, 256, 128), (200, 7, 72, 96),
          (300, 64, 40, 136), (31, 200, 24, 8), (1000, 3, 136, 72), (777, 16, 301, 200),
          (700, 2, 520, 264), (2500, 5, 96, 40), (40, 1, 1024, 512), (513, 2, 257, 1032),
          (33, 9, 1040, 2050), (1500, 1, 16, 24),
          # enough tiles for the larger ones, in every way that operands are read
          (2048, 1, 4200, 72), (2300, 2, 4224, 71), (3000, 3, 1200, 40), (3001, 3, 1201, 39)]


@pytest.mark.parametrize("rows,nlist,n,d", SHAPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_is_exact_on_integers(rows, nlist, n, d, transposed, dtype):
    rng = np.random.default_rng(rows + nlist + n + d)
    x = integers(rng, rows, d, dtype=dtype)
    w = integers(rng, nlist, *((d, n) if transposed else (n, d)), dtype=dtype)
    offsets = ragged(rng, rows, nlist, rows // 9, rows - rows // 7)
    y = A.ivfpq_list_product_ex(x, w, torch.from_numpy(offsets).cuda(), transposed=transposed)
    want, _ = list_product64(np64(x), np64(w), offsets, rows, np.arange(rows), transposed)
    assert y.dtype == dtype and np.array_equal(np64(y), rounded(want, dtype))


@pytest.mark.parametrize("t,k,nlist,n,d", [(1, 1, 1, 8, 8), (1, 8, 64, 64, 128), (4, 8, 16, 136, 64),
                                           (100, 3, 7, 33, 49), (333, 2, 5, 264, 72),
                                           (600, 4, 3, 48, 200)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_gathers_by_order(t, k, nlist, n, d, transposed, dtype):
    rng = np.random.default_rng(t + n)
    lists = rng.integers(-1, nlist, (t, k)).astype(np.int32)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(lists).cuda(), nlist)
    x = integers(rng, t, d, dtype=dtype)
    w = integers(rng, nlist, *((d, n) if transposed else (n, d)), dtype=dtype)
    y = A.ivfpq_list_product_ex(x, w, offsets, order=order, k=k, transposed=transposed)
    source = np.maximum(order.cpu().numpy(), 0) // k
    want, _ = list_product64(np64(x), np64(w), offsets.tolist(), t * k, source, transposed)
    assert np.array_equal(np64(y), rounded(want, dtype))


@pytest.mark.parametrize("rows,nlist,n,d", [(1, 1, 1, 1), (130, 4, 72, 1), (64, 2, 40, 4),
                                            (150, 3, 130, 200), (90, 5, 65, 777)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_of_reals(rows, nlist, n, d, transposed, dtype):
    rng = np.random.default_rng(rows * d)
    x = reals(rng, rows, d, dtype=dtype)
    w = reals(rng, nlist, *((d, n) if transposed else (n, d)), dtype=dtype)
    offsets = ragged(rng, rows, nlist)
    y = A.ivfpq_list_product_ex(x, w, torch.from_numpy(offsets).cuda(), transposed=transposed)
    want, mag = list_product64(np64(x), np64(w), offsets, rows, np.arange(rows), transposed)
    sums = sum_error(d, dtype) * mag
    assert (np.abs(np64(y) - want) <= sums + UNIT[dtype] * (np.abs(want) + sums) + 2.0 ** -25).all()


@pytest.mark.parametrize("t,k,nlist,n,d", [(1, 1, 1, 1, 1), (5, 1, 3, 8, 16), (40, 2, 4, 33, 31),
                                           (64, 1, 1, 64, 64), (333, 3, 5, 65, 129),
                                           (800, 2, 3, 136, 264), (100, 4, 150, 40, 24),
                                           (3000, 1, 2, 32, 48), (500, 2, 7, 257, 520),
                                           (6000, 1, 1, 24, 40),
                                           # larger tiles, workgroups that share a list, lists by
                                           # length
                                           (300, 1, 1, 1104, 2000), (1500, 3, 2, 1056, 1040),
                                           (4500, 1, 2, 130, 264), (5000, 1, 3, 65, 33),
                                           (2100, 2, 5, 1032, 2056)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype,out", [(t, o) for t in TYPES for o in {t, torch.float32}])
def test_gradient_is_exact_on_integers(t, k, nlist, n, d, gather, dtype, out):
    rng = np.random.default_rng(t + n + d)
    lists = rng.integers(-1, nlist, (t, k)).astype(np.int32)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(lists).cuda(), nlist)
    rows = t * k
    grad = integers(rng, rows, n, dtype=dtype)
    x = integers(rng, t if gather else rows, d, dtype=dtype)
    got = A.ivfpq_list_product_grad_ex(grad, x, offsets, order=order if gather else None, k=k,
                                       dtype=out)
    source = np.maximum(order.cpu().numpy(), 0) // k if gather else np.arange(rows)
    g64, x64, bounds = np64(grad), np64(x), offsets.tolist()
    want = np.stack([g64[lo:hi].T @ x64[source[lo:hi]] for lo, hi in zip(bounds, bounds[1:])])
    assert got.dtype == out and np.array_equal(np64(got), rounded(want, out))


def test_definitions_of_the_oracle():
    """The vectorised forms above against the oracle's loops."""
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((6, 5)), rng.standard_normal((3, 4, 5))
    offsets, order = [0, 2, 2, 7], rng.integers(0, 12, 8)
    want, mag = R.list_product(x, w, offsets, order, 2, 8)
    got, mag2 = list_product64(x, w, offsets, 8, order // 2, False)
    assert np.allclose(got, want) and np.allclose(mag, mag2)
    grad = rng.standard_normal((8, 4))
    want, _ = R.list_gradient(grad, x, offsets, order, 2, 3)
    for e in range(3):
        part = slice(offsets[e], offsets[e + 1])
        assert np.allclose(grad[part].T @ x[order[part] // 2], want[e])


def test_offsets_beyond_the_rows_and_entries_that_are_no_rows():
    rng = np.random.default_rng(3)
    x = integers(rng, 40, 64, dtype=torch.bfloat16)
    w = integers(rng, 3, 72, 64, dtype=torch.bfloat16)
    offsets = np.array([-5, 12, 30, 99], np.int32)
    y = A.ivfpq_list_product_ex(x, w, torch.from_numpy(offsets).cuda())
    want, _ = list_product64(np64(x), np64(w), np.clip(offsets, 0, 40), 40, np.arange(40), False)
    assert np.array_equal(np64(y), rounded(want, torch.bfloat16))
    # entries of order outside the rows stand for rows of zeros
    order = np.arange(40, dtype=np.int32)
    order[[3, 20, 39]] = [-1, 40, 2 ** 31 - 1]
    for dtype in TYPES:
        xt, wt = x.to(dtype), w.to(dtype)
        o = torch.from_numpy(order).cuda()
        f = torch.tensor([0, 12, 30, 40], dtype=torch.int32, device="cuda")
        clean = np64(x).copy()
        clean[[3, 20, 39]] = 0
        got = A.ivfpq_list_product_ex(xt, wt, f, order=o)
        want, _ = list_product64(clean, np64(w), [0, 12, 30, 40], 40, np.arange(40), False)
        assert np.array_equal(np64(got), rounded(want, dtype))
        grad = integers(rng, 40, 72, dtype=dtype)
        got = A.ivfpq_list_product_grad_ex(grad, xt, f, order=o, dtype=torch.float32)
        want = np.stack([np64(grad)[lo:hi].T @ clean[lo:hi] for lo, hi in ((0, 12), (12, 30),
                                                                          (30, 40))])
        assert np.array_equal(np64(got), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,nlist,n,d", [(130, 4, 72, 64), (20, 30, 33, 31), (600, 2, 264, 200)])
def test_bad_values_stay_where_they_are(dtype, rows, nlist, n, d):
    """An infinity or NaN in a row reaches that row's results alone, one in a matrix
    that list's column; rows of no list are zero whatever is there."""
    rng = np.random.default_rng(rows)
    x, w = integers(rng, rows, d, dtype=dtype), integers(rng, nlist, n, d, dtype=dtype)
    offsets = ragged(rng, rows, nlist, rows // 8, rows - rows // 9)
    o = torch.from_numpy(offsets).cuda()
    for transposed in (False, True):
        m = w.transpose(1, 2).contiguous() if transposed else w
        clean = A.ivfpq_list_product_ex(x, m, o, transposed=transposed)
        xb, mb = x.clone(), m.clone()
        row = rows // 2
        e = int(np.searchsorted(offsets, row, side="right")) - 1
        xb[row, d - 1] = float("nan")
        xb[0] = float("inf")                       # before the first list
        xb[rows - 1] = float("nan")                # past the last
        (mb[e, 0, n - 1:] if transposed else mb[e, n - 1, :1]).fill_(float("inf"))
        got = A.ivfpq_list_product_ex(xb, mb, o, transposed=transposed)
        touched = torch.zeros_like(clean, dtype=torch.bool)
        touched[row] = True
        touched[offsets[e]:offsets[e + 1], n - 1] = True
        assert torch.equal(got[~touched], clean[~touched])
        assert got[row].isnan().all()
        assert not got[offsets[e]:offsets[e + 1], n - 1].isfinite().any()


def test_gradient_ignores_rows_of_other_lists():
    rng = np.random.default_rng(8)
    for dtype in TYPES:
        for n, d in ((64, 72), (33, 31)):
            grad, x = integers(rng, 500, n, dtype=dtype), integers(rng, 500, d, dtype=dtype)
            o = torch.tensor([100, 170, 170, 333], dtype=torch.int32, device="cuda")
            want = A.ivfpq_list_product_grad_ex(grad, x, o)
            grad[:100], x[:100], grad[333:], x[333:] = (float("nan"), float("inf"), float("inf"),
                                                        float("nan"))
            assert torch.equal(A.ivfpq_list_product_grad_ex(grad, x, o), want)
            assert (want[1] == 0).all()


def test_results_repeat_and_nothing_else_is_written():
    rng = np.random.default_rng(2)
    for dtype in TYPES:
        for rows, nlist, n, d in ((777, 9, 130, 136), (5000, 1, 65, 33), (2048, 1, 4200, 72)):
            x, w = reals(rng, rows, d, dtype=dtype), reals(rng, nlist, n, d, dtype=dtype)
            grad = reals(rng, rows, n, dtype=dtype)
            o = torch.from_numpy(ragged(rng, rows, nlist)).cuda()
            need = A.ivfpq_list_product_grad_bytes(rows, n, d, nlist)
            y, g = [], []
            for fill in (0.0, float("nan")):
                guard = torch.full((rows * n + 64,), fill, dtype=dtype, device="cuda")
                out = guard[32:-32].view(rows, n)
                ws = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
                y.append(A.ivfpq_list_product_ex(x, w, o, out=out).clone())
                g.append(A.ivfpq_list_product_grad_ex(grad, x, o, workspace=ws[:max(need, 16)]))
                edge = torch.cat([guard[:32], guard[-32:]])
                assert edge.isnan().all() if fill != fill else (edge == 0).all()
                assert (ws[max(need, 16):] == 0x7F).all()
            assert torch.equal(y[0], y[1]) and torch.equal(g[0], g[1])


def test_rows_that_begin_at_any_element():
    rng = np.random.default_rng(6)
    for dtype in TYPES:
        for shift in (1, 2, 3, 8):
            for d in (64, 63):
                base = integers(rng, 4 * 150 * 65 + 64, dtype=dtype)
                x = base[shift:shift + 150 * d].view(150, d)
                w = base[2 * shift + 150 * d:2 * shift + 150 * d + 3 * 40 * d].view(3, 40, d)
                o = torch.tensor([0, 70, 71, 150], dtype=torch.int32, device="cuda")
                want, _ = list_product64(np64(x), np64(w), o.tolist(), 150, np.arange(150), False)
                assert np.array_equal(np64(A.ivfpq_list_product_ex(x, w, o)), rounded(want, dtype))
                g = base[5 * shift:5 * shift + 150 * 40].view(150, 40)
                got = A.ivfpq_list_product_grad_ex(g, x, o, dtype=torch.float32)
                want = np.stack([np64(g)[lo:hi].T @ np64(x)[lo:hi]
                                 for lo, hi in ((0, 70), (70, 71), (71, 150))])
                assert np.array_equal(np64(got), want)


def test_refusals_of_device_tensors():
    x = torch.zeros((8, 16), device="cuda")
    w = torch.zeros((2, 4, 16), device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    order = torch.zeros(8, dtype=torch.int32, device="cuda")
    for call in (lambda: A.ivfpq_list_product_ex(x.t(), w, o),
                 lambda: A.ivfpq_list_product_ex(x, w.transpose(1, 2), o, transposed=True),
                 lambda: A.ivfpq_list_product_ex(x, w.to(torch.bfloat16), o),
                 lambda: A.ivfpq_list_product_ex(x, w, o, transposed=True),
                 lambda: A.ivfpq_list_product_ex(x, w, o[:2]),
                 lambda: A.ivfpq_list_product_ex(x, w, o.long()),
                 lambda: A.ivfpq_list_product_ex(x, w, o, order=order.view(4, 2)),
                 lambda: A.ivfpq_list_product_ex(x, w, o, out=torch.zeros((8, 5), device="cuda")),
                 lambda: A.ivfpq_list_product_grad_ex(x, x[:4], o),
                 lambda: A.ivfpq_list_product_grad_ex(x, x, o, order=order[:7]),
                 lambda: A.ivfpq_list_product_grad_ex(x, x, o[:1]),
                 lambda: A.ivfpq_list_product_grad_ex(x, x, o, dtype=torch.int32)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: A.ivfpq_list_product_ex(x, w, o, order=order, k=0),
                 lambda: A.ivfpq_list_product_grad_ex(x, x, o, dtype=torch.bfloat16)):
        with pytest.raises(A.IVFPQError):
            call()
    assert A.ivfpq_list_product_ex(x[:0], w, o).shape == (0, 4)
    assert (A.ivfpq_list_product_grad_ex(x[:0], x[:0], o) == 0).all()


def three_parts(rng, *shape, kind, terms):
    """float32 values that one bfloat16 does not hold, and of which about 12 in `terms` are not
    zero: "wide" ones have 18 bits (three parts), "narrow" ones 1, "two" 9 bits (two
    parts).  Products of wide and narrow, or two and two, are integers below 2^18, so
    60 of them add to less than 2^24."""
    v = {"wide": rng.integers(1 << 16, 1 << 17, shape) * 2 + 1, "narrow": np.ones(shape, int),
         "two": rng.integers(128, 256, shape) * 2 + 1}[kind]
    v = v * rng.choice([-1, 1], shape)
    if kind != "wide":
        v = v * (rng.random(shape) < min(1.0, 12 / terms))
    return torch.from_numpy(v.astype(np.float32)).cuda()


PAIRS = [("wide", "narrow"), ("narrow", "wide"), ("two", "two")]


@pytest.mark.parametrize("rows,nlist,n,d", [s for s in SHAPES if s[0] > 1])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kinds", PAIRS)
def test_float32_products_use_all_parts(rows, nlist, n, d, transposed, kinds):
    rng = np.random.default_rng(rows + n + d)
    x = three_parts(rng, rows, d, kind=kinds[0], terms=d)
    w = three_parts(rng, nlist, *((d, n) if transposed else (n, d)), kind=kinds[1], terms=d)
    offsets = ragged(rng, rows, nlist, rows // 9, rows - rows // 7)
    y = A.ivfpq_list_product_ex(x, w, torch.from_numpy(offsets).cuda(), transposed=transposed)
    want, mag = list_product64(np64(x), np64(w), offsets, rows, np.arange(rows), transposed)
    assert mag.max() < 2 ** 24 and np.array_equal(np64(y), want)


GRADIENT_TILES = [(333, 3, 5, 65, 129), (800, 2, 3, 136, 264), (300, 1, 1, 1104, 2000),
                  (1500, 3, 2, 1056, 1040), (4500, 1, 2, 130, 264), (5000, 1, 3, 65, 33),
                  (2100, 2, 5, 1032, 2056)]


@pytest.mark.parametrize("t,k,nlist,n,d", GRADIENT_TILES)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kinds", PAIRS)
def test_float32_gradients_use_all_parts(t, k, nlist, n, d, gather, kinds):
    rng = np.random.default_rng(t + n)
    lists = rng.integers(-1, nlist, (t, k)).astype(np.int32)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(lists).cuda(), nlist)
    terms = max(np.diff(offsets.tolist()))
    grad = three_parts(rng, t * k, n, kind=kinds[0], terms=terms)
    x = three_parts(rng, t if gather else t * k, d, kind=kinds[1], terms=terms)
    got = A.ivfpq_list_product_grad_ex(grad, x, offsets, order=order if gather else None, k=k)
    source = np.maximum(order.cpu().numpy(), 0) // k if gather else np.arange(t * k)
    g64, x64, bounds = np64(grad), np64(x), offsets.tolist()
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        assert (np.abs(g64[lo:hi]).T @ np.abs(x64[source[lo:hi]])).max() < 2 ** 24
        assert np.array_equal(np64(got[e]), g64[lo:hi].T @ x64[source[lo:hi]])


# enough tiles for the larger copies and for the larger tiles through registers
@pytest.mark.parametrize("rows,nlist,n,d", [(2048, 1, 4200, 72), (3000, 3, 1200, 264),
                                            (3001, 3, 1201, 39), (700, 2, 520, 264)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_products_of_reals_in_larger_tiles(rows, nlist, n, d, transposed, dtype):
    rng = np.random.default_rng(n + d)
    x = reals(rng, rows, d, dtype=dtype)
    w = reals(rng, nlist, *((d, n) if transposed else (n, d)), dtype=dtype)
    offsets = ragged(rng, rows, nlist)
    y = A.ivfpq_list_product_ex(x, w, torch.from_numpy(offsets).cuda(), transposed=transposed)
    want, mag = list_product64(np64(x), np64(w), offsets, rows, np.arange(rows), transposed)
    sums = sum_error(d, dtype) * mag
    assert (np.abs(np64(y) - want) <= sums + UNIT[dtype] * (np.abs(want) + sums) + 2.0 ** -25).all()


@pytest.mark.parametrize("t,k,nlist,n,d", GRADIENT_TILES)
@pytest.mark.parametrize("dtype,out", [(t, o) for t in TYPES for o in {t, torch.float32}])
def test_gradients_of_reals(t, k, nlist, n, d, dtype, out):
    rng = np.random.default_rng(t + d)
    lists = rng.integers(-1, nlist, (t, k)).astype(np.int32)
    offsets, order, _ = A.ivfpq_route_sort_ex(torch.from_numpy(lists).cuda(), nlist)
    grad, x = reals(rng, t * k, n, dtype=dtype), reals(rng, t, d, dtype=dtype)
    got = A.ivfpq_list_product_grad_ex(grad, x, offsets, order=order, k=k, dtype=out)
    g64, x64, bounds = np64(grad), np64(x)[np.maximum(order.cpu().numpy(), 0) // k], offsets.tolist()
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        want = g64[lo:hi].T @ x64[lo:hi]
        # joining the parts of a list adds at most 64 sums
        sums = sum_error(hi - lo + 64, dtype) * (np.abs(g64[lo:hi]).T @ np.abs(x64[lo:hi]))
        assert (np.abs(np64(got[e]) - want) <=
                sums + UNIT[out] * (np.abs(want) + sums) + 2.0 ** -25).all()


@pytest.mark.parametrize("rows,n,d", [(40, 33, 64), (200, 1030, 64), (2048, 2200, 72)])
@pytest.mark.parametrize("transposed", [False, True])
def test_small_float32_factors(rows, n, d, transposed):
    """Factors from 2^-110 on keep their 24 bits, smaller ones are rounded to multiples of
    2^-133: one factor of a result is such a number, the other 2^100 or 0."""
    rng = np.random.default_rng(d)
    for e in (-133, -140, -149):
        whole = rng.integers(1 << 23, 1 << 24, (rows, d)).astype(np.float64)
        if e < -133:
            whole = np.round(whole / 2 ** 8)      # the least have less than 24 bits
        x = torch.from_numpy(np.ldexp(whole, e)).float().cuda()
        assert np.array_equal(np64(x), np.ldexp(whole, e)) or e == -149
        w = torch.zeros((1, n, d), device="cuda")
        w[0, torch.arange(n), torch.from_numpy(rng.integers(0, d, n))] = 2.0 ** 100
        o = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        want = np64(x) @ np64(w[0]).T
        m = w.transpose(1, 2).contiguous() if transposed else w
        y = A.ivfpq_list_product_ex(x, m, o, transposed=transposed)
        error = 0.0 if e == -133 else 2.0 ** (100 - 134)
        assert (np.abs(np64(y) - want) <= error).all()
        g = torch.zeros((rows, 5), device="cuda")
        g[rows // 2] = 2.0 ** 100
        got = A.ivfpq_list_product_grad_ex(g, x, o)
        assert (np.abs(np64(got[0]) - 2.0 ** 100 * np64(x)[rows // 2]) <= error).all()
