"""4-bit rows and list routing together, as a user would run them.

1. A routed layer: an index's coarse step sends each vector to its nearest
   lists, the (vector, list) pairs are sorted by list, every list multiplies its
   vectors with a matrix of its own in 4 bits, and the results come back to
   their vectors, weighted by the lists' distances.  Prompt-sized batches and
   single vectors take the same calls.
2. Its training step: the same route with float32 rows and a matrix per list,
   gradients through the weighted sum and the gather (torch.autograd.Function
   around the library's calls), a few steps of gradient descent.
3. A search over 4-bit rows: scores of all rows from one product, the library's
   k-selection on them, and how much of the exact search it finds.

Run on the GPU:  python examples/routed_layer.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import approximate_nearest_neighbour_amd as A  # noqa: E402
from approximate_nearest_neighbour_amd import datagen as G  # noqa: E402


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order, pos):
        ctx.save_for_backward(pos)
        return A.ivfpq_route_gather_ex(x, order, pos.shape[1])

    @staticmethod
    def backward(ctx, grad):
        pos, = ctx.saved_tensors
        return A.ivfpq_route_combine_ex(grad.contiguous(), pos), None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, order, pos):
        ctx.save_for_backward(rows, weights, order, pos)
        return A.ivfpq_route_combine_ex(rows, pos, weights)

    @staticmethod
    def backward(ctx, grad):
        rows, weights, order, pos = ctx.saved_tensors
        return (*A.ivfpq_route_combine_grad_ex(grad.contiguous(), rows, order, pos, weights),
                None, None)


def route(index, x, k):
    """Lists and weights of vectors x [n, d] float32: the coarse step's k nearest,
    weighted by a softmax of the negated distances."""
    lists, dist = A.ivfpq_coarse_ex(index, x, k)
    return lists, torch.softmax(-dist, dim=1)


def layer_4bit(index, packed, x, k):
    """x [n, d] float32 through the lists' 4-bit matrices: [n, out] bfloat16."""
    lists, weights = route(index, x, k)
    offsets, order, pos = A.ivfpq_route_sort_ex(lists, packed[0].shape[0])
    h = A.ivfpq_mx4_list_product_ex(A.ivfpq_mx4_quantize_ex(x), packed, offsets, order=order, k=k,
                                    dtype=torch.bfloat16)
    return A.ivfpq_route_combine_ex(h, pos, weights)


def layer_train(index, matrices, x, k):
    """The same layer with float32 matrices [nlist, out, d], differentiable."""
    lists, weights = route(index, x.detach(), k)
    offsets, order, pos = A.ivfpq_route_sort_ex(lists, matrices.shape[0])
    rows = Gather.apply(x, order, pos)
    bounds = offsets.tolist()
    h = torch.cat([rows[lo:hi] @ w.t() for w, lo, hi in zip(matrices, bounds, bounds[1:])] +
                  [rows.new_zeros((len(rows) - bounds[-1], matrices.shape[1]))])
    return Combine.apply(h, weights, order, pos)


def pack(matrices):
    nlist, out, d = matrices.shape
    codes, scales = A.ivfpq_mx4_quantize_ex(matrices.reshape(-1, d).contiguous())
    return codes.view(nlist, out, -1), scales.view(nlist, out, -1)


def make_index(nlist, d, seed=0):
    rng = np.random.default_rng(seed)
    return A.ivfpq_load_index_host(G.random_index(rng, nlist, d, 8, [0] * nlist))


def search_4bit(rows, queries, k):
    """k rows of largest inner product, scored in 4 bits: (scores, row numbers)."""
    scores = A.ivfpq_mx4_product_ex(A.ivfpq_mx4_quantize_ex(queries), A.ivfpq_mx4_quantize_ex(rows))
    best, ids = A.ivfpq_select_topk_ex(scores.neg_(), k)
    return best.neg_(), ids


def main():
    nlist, d, out, k = 16, 128, 256, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    index = make_index(nlist, d)
    x = torch.randn((1000, d), generator=g, device="cuda")
    matrices = torch.randn((nlist, out, d), generator=g, device="cuda") / d ** 0.5
    packed = pack(matrices)
    y = layer_4bit(index, packed, x, k).float()
    want = layer_train(index, matrices, x, k)
    error = (y - want).norm() / want.norm()
    print(f"routed layer in 4 bits: relative error {float(error):.3f}")
    one = layer_4bit(index, packed, x[:1], k).float()
    print(f"single vector against the batch: {float((one - y[:1]).abs().max()):.2e}")

    goal = want.detach()
    learned = torch.zeros_like(matrices).requires_grad_()
    for step in range(40):
        loss = (layer_train(index, learned, x, k) - goal).square().mean()
        loss.backward()
        with torch.no_grad():
            learned -= 40.0 * learned.grad
            learned.grad = None
        if step % 13 == 0:
            print(f"step {step}: loss {float(loss.detach()):.4f}")
    index.close()

    rows = torch.nn.functional.normalize(torch.randn((20000, d), generator=g, device="cuda"), dim=1)
    queries = rows[:100] + 0.05 * torch.randn((100, d), generator=g, device="cuda")
    _, found = search_4bit(rows, queries, 10)
    exact = (queries @ rows.t()).topk(10).indices
    hits = (found.long()[:, :, None] == exact[:, None, :]).any(dim=2).float().mean()
    print(f"search in 4 bits: {float(hits):.3f} of the exact 10, nearest row first in "
          f"{float((found[:, 0].long() == exact[:, 0]).float().mean()):.3f}")


if __name__ == "__main__":
    main()
