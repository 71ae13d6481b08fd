"""The routed layer of examples/routed_layer.py: its 4-bit form against the
64-bit definitions, its gradients against torch's, its search's order."""
import os
import sys

import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from oracle import rows as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import routed_layer as E  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 7, 300])
def test_layer_against_definitions(n):
    nlist, d, out, k = 8, 96, 80, 3
    g = torch.Generator(device="cuda").manual_seed(n)
    index = E.make_index(nlist, d)
    x = torch.randn((n, d), generator=g, device="cuda")
    w = torch.randn((nlist, out, d), generator=g, device="cuda")
    y = E.layer_4bit(index, E.pack(w), x, k).double().cpu().numpy()
    lists, weights = (t.cpu().numpy() for t in E.route(index, x, k))
    index.close()
    xv = R.values(*R.quantize(x.cpu().numpy()), d)
    wv = R.values(*R.quantize(w.reshape(-1, d).cpu().numpy()), d).reshape(nlist, out, d)
    offsets, order, pos = R.route_sort(lists, nlist)
    h, mag = R.list_product(xv, wv, offsets, order, k, n * k)
    exact, terms = R.combine(h, pos, weights)
    # products: d 2^-23 of the magnitudes and bfloat16's 2^-8; the sum: k 2^-23; bfloat16 again
    bound, _ = R.combine(d * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(h), pos, np.abs(weights))
    tol = 1.01 * (bound + k * 2.0 ** -23 * terms) + 2.0 ** -8 * np.abs(exact)
    assert (np.abs(y - exact) <= tol).all()


def test_gradients_against_torch():
    nlist, d, out, k, n = 4, 32, 24, 2, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    index = E.make_index(nlist, d)
    x = torch.randn((n, d), generator=g, device="cuda").requires_grad_()
    w = torch.randn((nlist, out, d), generator=g, device="cuda").requires_grad_()
    dy = torch.randn((n, out), generator=g, device="cuda")
    E.layer_train(index, w, x, k).backward(dy)
    lists, weights = E.route(index, x.detach(), k)
    index.close()
    xr = x.detach().double().cpu().requires_grad_()
    wr = w.detach().double().cpu().requires_grad_()
    per = torch.stack([xr @ m.t() for m in wr], dim=1)              # [n, nlist, out]
    picked = torch.stack([per[torch.arange(n), lists[:, j].long().cpu()] for j in range(k)], 1)
    (picked * weights.double().cpu()[:, :, None]).sum(1).backward(dy.double().cpu())
    # float32 sums of up to n k out terms of order one: far below 1e-3
    assert (x.grad.double().cpu() - xr.grad).abs().max() < 1e-3
    assert (w.grad.double().cpu() - wr.grad).abs().max() < 1e-3


def test_search_in_4_bits_orders_by_the_4_bit_scores():
    g = torch.Generator(device="cuda").manual_seed(9)
    rows = torch.randn((3000, 64), generator=g, device="cuda")
    queries = torch.randn((20, 64), generator=g, device="cuda")
    best, ids = E.search_4bit(rows, queries, 10)
    vr = R.values(*R.quantize(rows.cpu().numpy()), 64)
    vq = R.values(*R.quantize(queries.cpu().numpy()), 64)
    scores = vq @ vr.T
    tol = 64 * 2.0 ** -23 * (np.abs(vq) @ np.abs(vr).T).max()
    want = -np.sort(-scores, axis=1)[:, :10]
    assert (np.abs(best.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(np.take_along_axis(scores, ids.long().cpu().numpy(), 1) - want) <= 2 * tol).all()
