"""Rows through a shared matrix with their adapters beside it, on the GPU against the
64-bit definition of oracle/rows.py.

Tolerances.  Small integers: every sum is an integer below 2^24 and the hidden rows
are below 2^16, which two 16-bit parts hold exactly, so results are exact, rounded
once.  Real values: the d + 2 r products of a result and the d of a hidden value are
added in float32 (test_gpu_list_product.py says by how much they are off; the second
parts of hidden values add at most 2^-8 to the magnitudes, and the scale rounds
once); two parts of a hidden value leave 2^-16 of it in bfloat16 (8 bits each, and
the sign of the second), 2^-22 in binary16, none in float32; storing rounds by half a
step.
"""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R
from test_gpu_list_product import TYPES, UNIT, integers, np64, reals, rounded, sum_error

pytestmark = pytest.mark.gpu

PARTS = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}

# t, n, d, lists, r
SHAPES = [(1, 8, 8, 1, 1), (1, 256, 128, 4, 16), (5, 33, 17, 3, 7), (16, 64, 64, 2, 8),
          (32, 136, 200, 40, 16), (64, 128, 72, 1, 64), (129, 65, 49, 5, 33), (200, 264, 136, 300, 5),
          (300, 130, 96, 3, 24), (700, 72, 64, 9, 40), (513, 257, 520, 2, 130),
          # every kind of tile: few and many of each size
          (200, 1000, 64, 3, 8), (500, 4000, 40, 2, 8), (1000, 4000, 24, 2, 16),
          (1300, 4200, 24, 3, 8), (2048, 4200, 32, 2, 8), (2100, 4201, 23, 2, 5), (4200, 72, 64, 3, 64), (4300, 40, 72, 5, 61)]


def lists_of(rng, t, nlist, kind):
    if kind == "runs":      # requests side by side
        cuts = np.sort(rng.integers(0, t + 1, 4))
        lists = np.searchsorted(cuts, np.arange(t), side="right")
        return rng.integers(-1, nlist, 5)[lists].astype(np.int32)
    if kind == "none":
        return np.full(t, -1, np.int32)
    return rng.integers(-1, nlist + 1, t).astype(np.int32)


def adapter64(x, w, down, up, lists, scales):
    """The definition, a list at a time (the oracle's goes by rows)."""
    out, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    for e in range(len(down)):
        mine = np.flatnonzero(lists == e)
        if len(mine):
            s = 1.0 if scales is None else float(scales[e])
            out[mine] += s * (x[mine] @ down[e].T) @ up[e].T
            mag[mine] += abs(s) * (np.abs(x[mine]) @ np.abs(down[e]).T) @ np.abs(up[e]).T
    return out, mag


def test_definition_against_the_oracle():
    rng = np.random.default_rng(1)
    args = (rng.standard_normal((9, 5)), rng.standard_normal((4, 5)),
            rng.standard_normal((3, 2, 5)), rng.standard_normal((3, 4, 2)),
            np.array([0, 2, -1, 3, 1, 1, 2, 0, 9]), rng.random(3))
    for got, want in zip(adapter64(*args), R.adapter(*args)):
        assert np.allclose(got, want)


def call(x, w, down, up, lists, scales, **kw):
    plan = A.ivfpq_route_sort_ex(torch.from_numpy(lists[:, None]).cuda(), down.shape[0])
    return A.ivfpq_adapter_product_ex(x, w, down, up, *plan, scales=scales, **kw)


@pytest.mark.parametrize("t,n,d,nlist,r", SHAPES)
@pytest.mark.parametrize("kind", ["runs", "mixed", "none"])
@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_are_exact_on_integers(t, n, d, nlist, r, kind, dtype):
    rng = np.random.default_rng(t + n + d + r)
    x, w = integers(rng, t, d, dtype=dtype), integers(rng, n, d, dtype=dtype)
    down = integers(rng, nlist, r, d, dtype=dtype, top=2)
    up = integers(rng, nlist, n, r, dtype=dtype, top=2)
    scales = torch.from_numpy(rng.choice([0.5, 1.0, 2.0, -1.0], nlist).astype(np.float32)).cuda()
    lists = lists_of(rng, t, nlist, kind)
    for s in (scales, None):
        y = call(x, w, down, up, lists, s)
        want, _ = adapter64(np64(x), np64(w), np64(down), np64(up), lists,
                            None if s is None else np64(s))
        assert y.dtype == dtype and np.array_equal(np64(y), rounded(want, dtype))


@pytest.mark.parametrize("t,n,d,nlist,r", [(1, 40, 1, 1, 1), (70, 130, 100, 4, 12), (33, 65, 777, 6, 7),
                                           (150, 64, 64, 3, 64)])
@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_of_reals(t, n, d, nlist, r, dtype):
    rng = np.random.default_rng(t * d)
    x, w = reals(rng, t, d, dtype=dtype), reals(rng, n, d, dtype=dtype)
    down, up = reals(rng, nlist, r, d, dtype=dtype), reals(rng, nlist, n, r, dtype=dtype)
    scales = torch.from_numpy(rng.random(nlist).astype(np.float32) + 0.25).cuda()
    lists = lists_of(rng, t, nlist, "mixed")
    got = np64(call(x, w, down, up, lists, scales))
    want, mag = R.adapter(np64(x), np64(w), np64(down), np64(up), lists, np64(scales))
    error = sum_error(d + 2 * r, dtype) + sum_error(d, dtype) + 2.0 ** -24 + PARTS[dtype]
    sums = error * (1 + 2.0 ** -7) * mag
    assert (np.abs(got - want) <= sums + UNIT[dtype] * (np.abs(want) + sums) + 2.0 ** -24).all()


@pytest.mark.parametrize("t,n,d,nlist,r", [(20, 40, 64, 4, 8), (150, 257, 65, 3, 5), (300, 1000, 64, 3, 8),
                                          (500, 4000, 16, 5, 8), (1000, 4000, 24, 4, 16),
                                          (1300, 4200, 24, 9, 8), (2048, 4200, 32, 6, 8),
                                          (2100, 4201, 23, 5, 5), (4200, 72, 136, 5, 64)])
@pytest.mark.parametrize("dtype", TYPES)
def test_bad_values_stay_where_they_are(t, n, d, nlist, r, dtype):
    """What is wrong in one row, or in the matrices of one list, reaches no other row."""
    rng = np.random.default_rng(t)
    x, w = integers(rng, t, d, dtype=dtype), integers(rng, n, d, dtype=dtype)
    down, up = integers(rng, nlist, r, d, dtype=dtype), integers(rng, nlist, n, r, dtype=dtype)
    lists = rng.integers(-1, nlist, t).astype(np.int32)
    lists[:2] = [0, -1]
    clean = call(x, w, down, up, lists, None)
    x[1], down[0, r - 1, d - 1], up[nlist - 1, 0] = float("inf"), float("nan"), float("nan")
    got = call(x, w, down, up, lists, None)
    hit = np.flatnonzero((lists == 0) | (lists == nlist - 1) | (np.arange(t) == 1))
    rest = np.setdiff1d(np.arange(t), hit)
    assert torch.equal(got[rest], clean[rest])
    assert not got[0].isfinite().any() and not got[1].isfinite().any()


def test_results_repeat_and_nothing_else_is_written():
    rng = np.random.default_rng(4)
    for dtype in TYPES:
        for t, n, d, nlist, r in ((32, 130, 72, 6, 8), (200, 1000, 64, 3, 8), (600, 65, 33, 4, 7)):
            x, w = reals(rng, t, d, dtype=dtype), reals(rng, n, d, dtype=dtype)
            down, up = reals(rng, nlist, r, d, dtype=dtype), reals(rng, nlist, n, r, dtype=dtype)
            lists = rng.integers(-1, nlist, t).astype(np.int32)
            need = A.ivfpq_adapter_product_bytes(t, r)
            results = []
            for fill in (0x00, 0xFF):   # the workspace may hold anything, NaN too
                ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
                guard = torch.full((t * n + 64,), 3.0, dtype=dtype, device="cuda")
                out = guard[32:-32].view(t, n)
                results.append(call(x, w, down, up, lists, None, out=out, workspace=ws[:need]).clone())
                assert (guard[:32] == 3).all() and (guard[-32:] == 3).all()
                assert (ws[need:] == fill).all()
            assert torch.equal(*results)


def test_refusals_of_device_tensors():
    x, w = torch.zeros((8, 16), device="cuda"), torch.zeros((4, 16), device="cuda")
    down, up = torch.zeros((2, 3, 16), device="cuda"), torch.zeros((2, 4, 3), device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    order = torch.zeros(8, dtype=torch.int32, device="cuda")
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")
    for call_ in (lambda: A.ivfpq_adapter_product_ex(x, w.t(), down, up, o, order, order),
                  lambda: A.ivfpq_adapter_product_ex(x, w, down.half(), up, o, order, order),
                  lambda: A.ivfpq_adapter_product_ex(x, w, down, up[:, :3].contiguous(), o, order,
                                                     order),
                  lambda: A.ivfpq_adapter_product_ex(x, w, down, up, o[:2], order, order),
                  lambda: A.ivfpq_adapter_product_ex(x, w, down, up, o, order[:7], order),
                  lambda: A.ivfpq_adapter_product_ex(x, w, down, up, o, order, order[:7]),
                  lambda: A.ivfpq_adapter_product_ex(x, w, down, up, o, order, order,
                                                     scales=torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            call_()
    with pytest.raises(A.IVFPQError):
        A.ivfpq_adapter_product_ex(x, w, down, up, o, order, order, workspace=small)
    assert A.ivfpq_adapter_product_ex(x[:0], w, down, up, o, order[:0], order[:0]).shape == (0, 4)


def test_rows_outside_the_lists_take_the_shared_product_alone():
    """offsets narrower than the sort's: what lies outside belongs to no list, whatever
    the workspace held."""
    rng = np.random.default_rng(7)
    for dtype in TYPES:
        for t, n, d, r in ((40, 48, 64, 4), (300, 260, 72, 8), (33, 1, 3, 1)):
            x, w = integers(rng, t, d, dtype=dtype), integers(rng, n, d, dtype=dtype)
            down, up = integers(rng, 3, r, d, dtype=dtype), integers(rng, 3, n, r, dtype=dtype)
            order = torch.arange(t, dtype=torch.int32, device="cuda")
            ws = torch.zeros(A.ivfpq_adapter_product_bytes(t, r), dtype=torch.uint8, device="cuda")
            offsets = torch.tensor([10, 15, 15, 30], dtype=torch.int32, device="cuda")
            y = A.ivfpq_adapter_product_ex(x, w, down, up, offsets, order, order, workspace=ws)
            lists = np.full(t, -1)
            lists[10:15], lists[15:30] = 0, 2
            want, _ = adapter64(np64(x), np64(w), np64(down), np64(up), lists, None)
            assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(dtype)))


# a shape for every kernel that forms the results: blocks of few rows (16 x 16, 32 x 16,
# 32 x 32), copied tiles of every size, tiles through registers of every size
TILES = [(20, 40, 64, 4, 8), (33, 65, 77, 6, 7), (64, 1500, 64, 3, 16), (129, 1500, 64, 3, 16),
         (150, 257, 65, 3, 5), (300, 4000, 64, 3, 8), (500, 4000, 40, 5, 8), (1000, 4000, 24, 4, 16),
         (1300, 4200, 24, 9, 8), (2048, 4200, 32, 6, 8), (600, 1001, 25, 4, 5),
         (2100, 4201, 23, 5, 5), (4200, 72, 136, 5, 64)]


@pytest.mark.parametrize("t,n,d,nlist,r", TILES)
@pytest.mark.parametrize("dtype", TYPES)
def test_bad_values_change_no_other_rounding(t, n, d, nlist, r, dtype):
    """Real values: what a row or a list's matrices hold leaves every other row's sums as
    they are, to the last bit."""
    rng = np.random.default_rng(t + 1)
    x, w = reals(rng, t, d, dtype=dtype), reals(rng, n, d, dtype=dtype)
    down, up = reals(rng, nlist, r, d, dtype=dtype), reals(rng, nlist, n, r, dtype=dtype)
    lists = rng.integers(-1, nlist, t).astype(np.int32)
    lists[:4] = [0, -1, 1, 1]
    clean = call(x, w, down, up, lists, None)
    x[[1, 3, t - 1]] = torch.tensor([[float("inf")], [float("nan")], [float("-inf")]],
                                    device="cuda").to(dtype)
    up[0, n // 2], down[nlist - 1, 0, 0] = float("inf"), float("nan")
    got = call(x, w, down, up, lists, None)
    hit = (lists == 0) | (lists == nlist - 1)
    hit[[1, 3, t - 1]] = True
    rest = np.flatnonzero(~hit)
    assert len(rest) and torch.equal(got[rest], clean[rest])
    assert not got[0, n // 2].isfinite() and not got[[1, 3, t - 1]].isfinite().any()


# the power of two of the hidden rows; up matrices have the one that makes it 2^-10, or 2^-20
POWERS = {torch.float32: (-90, -24, 0, 14, 90), torch.bfloat16: (-90, -24, 0, 14, 90),
          torch.float16: (-34, -24, 0, 14)}


@pytest.mark.parametrize("t,n,d,nlist,r", TILES)
@pytest.mark.parametrize("dtype,power", [(t, p) for t in TYPES for p in POWERS[t]])
def test_hidden_rows_are_held_to_the_last_bit(t, n, d, nlist, r, dtype, power):
    """Hidden values of 21 bits at any power of two, which the shared product cancels for the
    rows of list 0: columns of x hold the bits, rows of down their signs, a row of up one
    entry.  Every term is a multiple of `unit` and all of a result's are below 2^24 units
    together, so that a float32 sum of them is exact in any order."""
    rng = np.random.default_rng(t + r)
    bits, unit = 22, 2.0 ** (-20 if power == -34 else -10)
    x = torch.zeros((t, d))
    x[:, :bits] = torch.from_numpy(rng.integers(0, 2, (t, bits)) * 2.0 ** (np.arange(bits) % 11))
    x[:, bits:] = torch.from_numpy(rng.integers(-3, 4, (t, d - bits)).astype(np.float32))
    down = torch.zeros((nlist, r, d))
    down[:, :, :bits] = torch.from_numpy(rng.choice([-1.0, 1.0], (nlist, r, bits)) *
                                         2.0 ** (np.arange(bits) // 11 * 10))
    up = torch.zeros((nlist, n, r))
    at = torch.from_numpy(rng.integers(0, r, (nlist, n, 1)))
    up.scatter_(2, at, torch.from_numpy(rng.choice([-1.0, 1.0], (nlist, n, 1))).float())
    w = -unit * (up[0] @ down[0])
    w[:, 0] += unit
    up *= unit * 2.0 ** -power
    scales = torch.full((nlist,), 2.0 ** power, device="cuda")
    lists = rng.integers(-1, nlist, t).astype(np.int32)
    lists[::3] = 0
    args = [a.to(dtype).cuda() for a in (x, w, down, up)]
    for a, b in zip(args, (x, w, down, up)):
        assert torch.equal(a.cpu().float(), b)
    y = call(*args, lists, scales)
    want, mag = adapter64(*(np64(a) for a in args), lists, np64(scales))
    assert mag.max() < 2 ** 24 * unit
    assert np.array_equal(want[::3], unit * np64(x)[::3, :1] * np.ones((1, n)))
    assert np.array_equal(np64(y), rounded(want, dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_are_not_finite_cost_no_second_product(dtype):
    """A NaN in every row of x (a value that overflowed) takes the time of a clean batch;
    where each such tile formed its sums again it took more than ten times that."""
    t, n, d, nlist, r = 4096, 2048, 2048, 8, 16
    rng = np.random.default_rng(5)
    x, w = reals(rng, t, d, dtype=dtype), reals(rng, n, d, dtype=dtype)
    down, up = reals(rng, nlist, r, d, dtype=dtype), reals(rng, nlist, n, r, dtype=dtype)
    lists = torch.from_numpy(rng.integers(-1, nlist, (t, 1)).astype(np.int32)).cuda()
    plan = A.ivfpq_route_sort_ex(lists, nlist)
    bad = x.clone()
    bad[:, 7] = float("nan")
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]

    def least(rows):
        times = []
        for _ in range(6):
            ends[0].record()
            for _ in range(3):
                A.ivfpq_adapter_product_ex(rows, w, down, up, *plan)
            ends[1].record()
            ends[1].synchronize()
            times.append(ends[0].elapsed_time(ends[1]))
        return min(times)

    clean_ms, bad_ms = least(x), least(bad)
    assert bad_ms < 4 * clean_ms


# a size for each copied tile, 32 x 128 to 256 x 256, and for the tiles through registers
BY_TILE = [((500, 521, 24), (24, 72, 136)), ((1700, 520, 24), (24, 72, 136)),
           ((1300, 3001, 24), (24, 72, 136)), ((1800, 1032, 24), (24, 72, 136)),
           ((800, 5000, 24), (24, 72, 136)), ((2700, 3000, 24), (24, 72, 136)),
           ((600, 1001, 25), (3, 33, 70)), ((2100, 2001, 23), (3, 33, 70))]


@pytest.mark.parametrize("t,n,d,r", [(*size, r) for size, ranks in BY_TILE for r in ranks])
@pytest.mark.parametrize("kind", ["runs", "mixed"])
@pytest.mark.parametrize("dtype", TYPES)
def test_ranks_in_every_tile(t, n, d, r, kind, dtype):
    """Ranks that end inside a step, a group of steps, or after several; one list in all
    of a tile's rows, or more than 32 in it."""
    rng = np.random.default_rng(t + r)
    nlist = 3 if kind == "runs" else 40
    x, w = integers(rng, t, d, dtype=dtype), integers(rng, n, d, dtype=dtype)
    down = integers(rng, nlist, r, d, dtype=dtype, top=2)
    up = integers(rng, nlist, n, r, dtype=dtype, top=2)
    lists = lists_of(rng, t, nlist, kind)
    want, mag = adapter64(np64(x), np64(w), np64(down), np64(up), lists, None)
    assert mag.max() < 2 ** 24
    assert np.array_equal(np64(call(x, w, down, up, lists, None)), rounded(want, dtype))
