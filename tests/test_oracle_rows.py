"""The plain definitions of 4-bit rows and routing against hand-worked cases
and identities."""
import numpy as np
import pytest

from oracle import rows as R


def test_quantize_hand_case():
    # largest magnitude 5 = 1.25 * 2^2: exponent byte 127, values are codes
    x = np.zeros((1, 33))
    x[0, :9] = [5.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.5 + 1.0, 0.26]
    x[0, 32] = 24.0                        # alone in the second block: 24 = 6 * 2^2
    codes, scales = R.quantize(x)
    assert scales.tolist() == [[127, 129]]
    v = R.values(codes, scales, 33)
    assert v[0, :9].tolist() == [4.0, -0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -4.0, 0.5]
    assert v[0, 32] == 24.0
    assert codes[0, 0] == 6 | (8 << 4)      # 4.0 low, -0 high
    assert codes.shape == (1, 32)


def test_quantize_error_bound():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 96)).astype(np.float32).astype(np.float64)
    codes, scales = R.quantize(x)
    v = R.values(codes, scales, 96).reshape(20, 3, 32)
    x = x.reshape(20, 3, 32)
    unit = 2.0 ** (scales.astype(float) - 127)[:, :, None]
    y = np.abs(x) / unit
    assert (y < 8).all() and (y.max(axis=2) >= 4).all()
    # half a step, or the saturation from below 8 to 6
    bound = np.where(y < 2, 0.25, np.where(y < 4, 0.5, np.where(y <= 6, 1.0, 2.0)))
    assert (np.abs(v - x) / unit <= bound).all()
    # what is representable comes back as it is
    again, s2 = R.quantize(v.reshape(20, 96))
    assert np.array_equal(R.values(again, s2, 96), v.reshape(20, 96))


def test_quantize_special_blocks():
    x = np.zeros((4, 32))
    x[1, 3], x[2, 5], x[3, 0] = np.nan, -np.inf, 2.0 ** -140
    codes, scales = R.quantize(x)
    assert scales[:, 0].tolist() == [0, 255, 255, 0]
    assert np.isnan(R.values(codes, scales, 32)[1:3]).all()
    assert (R.values(codes, scales, 32)[[0, 3]] == 0).all()


def test_route_sort_is_a_stable_partition():
    rng = np.random.default_rng(1)
    lists = rng.integers(-1, 6, size=(40, 3)).astype(np.int32)
    offsets, order, pos = R.route_sort(lists, 5)   # list 5 is outside
    flat = lists.reshape(-1)
    kept = (flat >= 0) & (flat < 5)
    assert offsets[5] == kept.sum() and (order[offsets[5]:] == -1).all()
    for l in range(5):
        mine = order[offsets[l]:offsets[l + 1]]
        assert np.array_equal(mine, np.flatnonzero(flat == l))
    assert np.array_equal(pos.reshape(-1) >= 0, kept)
    assert all(order[p] == u for u, p in enumerate(pos.reshape(-1)) if p >= 0)


@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_gradient_against_differences(drop):
    # the weighted sum is linear in the rows and in the weights, so a central
    # difference of any step is exact up to rounding
    rng = np.random.default_rng(2)
    lists = rng.integers(0, 4, size=(7, 2)).astype(np.int32)
    lists[rng.random(lists.shape) < drop] = -1
    _, order, pos = R.route_sort(lists, 4)
    rows, w = rng.standard_normal((14, 5)), rng.standard_normal((7, 2))
    g = rng.standard_normal((7, 5))
    f = lambda r, ww: float((R.combine(r, pos, ww)[0] * g).sum())  # noqa: E731
    d_rows, d_w, _ = R.combine_grad(g, rows, pos, w)
    for idx in np.ndindex(rows.shape):
        e = np.zeros_like(rows)
        e[idx] = 0.5
        assert abs(f(rows + e, w) - f(rows - e, w) - d_rows[idx]) < 1e-12
    for idx in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[idx] = 0.5
        assert abs(f(rows, w + e) - f(rows, w - e) - d_w[idx]) < 1e-12
    # and of the gather: its gradient is the sum back
    x = rng.standard_normal((7, 5))
    gr = rng.standard_normal((14, 5))
    back, _ = R.combine(gr, pos)
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = 0.5
        diff = ((R.gather(x + e, order, 2) - R.gather(x - e, order, 2)) * gr).sum()
        assert abs(diff - back[idx]) < 1e-12
