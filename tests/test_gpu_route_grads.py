"""The gradients of a weighted gather on the GPU, as the header says to take them,
against 64-bit sums of the formula and against differences.

Tolerances: a sum of k terms in float32 is within k 2^-23 of the sum of their
magnitudes, a product of d terms within d 2^-23 of theirs; storing rounds by the
unit of the type."""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def problem(rng, t, k, nlist, d, dtype):
    lists = rng.integers(-1, nlist + 1, size=(t, k)).astype(np.int32)  # some outside
    _, order, pos = A.ivfpq_route_sort_ex(torch.from_numpy(lists).cuda(), nlist)
    x = torch.from_numpy(rng.standard_normal((t, d))).to(dtype).cuda()
    g = torch.from_numpy(rng.standard_normal((t * k, d))).to(dtype).cuda()
    w = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).cuda()
    return order, pos, x, g, w


def np64(t):
    return t.cpu().double().numpy()


@pytest.mark.parametrize("t,k,nlist,d", [(1, 1, 1, 1), (40, 3, 5, 33), (130, 2, 9, 1001),
                                         (7, 8, 4, 2048)])
@pytest.mark.parametrize("dtype", list(UNIT))
def test_gradients_of_a_weighted_gather(t, k, nlist, d, dtype):
    order, pos, x, g, w = problem(np.random.default_rng(t + d), t, k, nlist, d, dtype)
    d_x = np64(A.ivfpq_route_combine_ex(g, pos, w))
    _, d_w = A.ivfpq_route_combine_grad_ex(x, g, order, pos, w)
    p, xv, gv, wv = pos.cpu().numpy(), np64(x), np64(g), np64(w)
    e_x, m_x, e_w, m_w = (np.zeros_like(xv), np.zeros_like(xv), np.zeros((t, k)), np.zeros((t, k)))
    for i in range(t):              # rows[p] = w[i, j] x[i] at the slot's position p
        for j in range(k):
            if p[i, j] >= 0:
                e_x[i] += wv[i, j] * gv[p[i, j]]
                m_x[i] += np.abs(wv[i, j] * gv[p[i, j]])
                e_w[i, j] = xv[i] @ gv[p[i, j]]
                m_w[i, j] = np.abs(xv[i]) @ np.abs(gv[p[i, j]])
    tol = k * 2.0 ** -23 * m_x * (1 + UNIT[dtype]) + UNIT[dtype] * np.abs(e_x) + 2.0 ** -25
    assert (np.abs(d_x - e_x) <= tol).all()
    assert (np.abs(np64(d_w) - e_w) <= d * 2.0 ** -23 * m_w).all()


def test_gradients_of_a_weighted_gather_against_differences():
    # <gather(x, w), g> is linear in x and in w: a central difference has no error
    # of its own, only the roundings of the two gathered products
    t, k, d = 5, 2, 6
    order, pos, x, g, w = problem(np.random.default_rng(1), t, k, 4, d, torch.float32)
    d_x = np64(A.ivfpq_route_combine_ex(g, pos, w))
    d_w = np64(A.ivfpq_route_combine_grad_ex(x, g, order, pos, w)[1])
    gv = np64(g)

    def f(xx, ww):
        return float((np64(A.ivfpq_route_gather_ex(xx, order, k, weights=ww)) * gv).sum())

    rows = R.gather(np.abs(np64(x)) + 1, order.cpu().numpy(), k, np.abs(np64(w)) + 1)
    tol = 2.0 ** -22 * float((rows * np.abs(gv)).sum()) * (k + d)
    for v, grad in ((x, d_x), (w, d_w)):
        for i in np.ndindex(*v.shape):
            up, down = v.clone(), v.clone()
            up[i] += 0.5
            down[i] -= 0.5
            step = float(up[i]) - float(down[i])
            change = f(up, w) - f(down, w) if v is x else f(x, up) - f(x, down)
            assert abs(change - step * grad[i]) <= tol
