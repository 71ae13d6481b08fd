"""4-bit rows and list routing together, as a user would run them.

1. A routed layer: an index's coarse step sends each vector to its nearest
   lists, the (vector, list) pairs are sorted by list, every list multiplies its
   vectors with a matrix of its own in 4 bits, and the results come back to
   their vectors, weighted by the lists' distances.  Prompt-sized batches and
   single vectors take the same calls.
2. Its training step: the same route with float32 rows and a matrix per list,
   gradients through the weighted sum, the products and the gather
   (torch.autograd.Function around the library's calls; nothing comes back to the
   host), a few steps of gradient descent.
3. Vectors from a table by their numbers, through one matrix for all and low-rank
   matrices of each vector's own list beside it, with the gradients of the table and
   of the low-rank matrices.
4. A search over 4-bit rows: scores of all rows from one product, the library's
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


class ListProduct(torch.autograd.Function):
    """Sorted rows times their lists' matrices; sorted row p is x[order[p] // k]."""

    @staticmethod
    def forward(ctx, x, matrices, offsets, order, pos):
        ctx.save_for_backward(x, matrices, offsets, order, pos)
        return A.ivfpq_list_product_ex(x, matrices, offsets, order=order, k=pos.shape[1])

    @staticmethod
    def backward(ctx, grad):
        x, matrices, offsets, order, pos = ctx.saved_tensors
        grad = grad.contiguous()
        rows = A.ivfpq_list_product_ex(grad, matrices, offsets, transposed=True)
        return (A.ivfpq_route_combine_ex(rows, pos),
                A.ivfpq_list_product_grad_ex(grad, x, offsets, order=order, k=pos.shape[1]),
                None, None, None)


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


class Lookup(torch.autograd.Function):
    """Rows of a table by number (outside the table: zero), times a factor."""

    @staticmethod
    def forward(ctx, table, ids, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return A.ivfpq_table_lookup_ex(table, ids, scale=scale)

    @staticmethod
    def backward(ctx, grad):
        ids, = ctx.saved_tensors
        offsets, order, _ = A.ivfpq_route_sort_ex(ids.view(-1, 1), ctx.rows)
        return A.ivfpq_table_grad_ex(grad.contiguous(), offsets, order, scale=ctx.scale), None, None


class Adapted(torch.autograd.Function):
    """x [t, d] times w [n, d], and times up[e] down[e] scales[e] for e the row's list;
    w is not trained."""

    @staticmethod
    def forward(ctx, x, w, down, up, scales, offsets, order, pos):
        ctx.save_for_backward(x, w, down, up, scales, offsets, order, pos)
        return A.ivfpq_adapter_product_ex(x, w, down, up, offsets, order, pos, scales=scales)

    @staticmethod
    def backward(ctx, grad):
        x, w, down, up, scales, offsets, order, pos = ctx.saved_tensors
        grad = grad.contiguous()
        nlist = len(scales)
        listed = torch.bucketize(torch.arange(len(x), dtype=torch.int32, device=x.device),
                                 offsets[:-1], right=True) - 1
        factor = scales[listed.clamp(0, nlist - 1)]       # of the sorted rows; others are zero
        # as the rows' weights, so that the product is float32 and rounded once to their type
        weights = factor[pos.clamp(min=0).view(-1).long()]
        rows = A.ivfpq_route_gather_ex(grad, order, 1, weights=weights[:, None])
        hidden = A.ivfpq_list_product_ex(x, down, offsets, order=order)
        grad_hidden = A.ivfpq_list_product_ex(rows, up, offsets, transposed=True)
        grad_rows = A.ivfpq_list_product_ex(grad_hidden, down, offsets, transposed=True)
        one = torch.zeros(2, dtype=torch.int32, device=x.device)
        one[1] = len(x)                                   # all rows are of the one shared matrix
        return (A.ivfpq_list_product_ex(grad, w[None], one, transposed=True) +
                A.ivfpq_route_combine_ex(grad_rows, pos), None,
                A.ivfpq_list_product_grad_ex(grad_hidden, x, offsets, order=order),
                A.ivfpq_list_product_grad_ex(rows, hidden, offsets), None, None, None, None)


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
    h = ListProduct.apply(x, matrices, offsets, order, pos)
    return Combine.apply(h, weights, order, pos)


def layer_adapted(table, ids, w, down, up, scales, lists, scale=1.0):
    """Rows `ids` of a table through w [n, d] and through the low-rank matrices of their
    lists (lists [t]; -1: none): [t, n], differentiable but for w and the scales."""
    offsets, order, pos = A.ivfpq_route_sort_ex(lists.view(-1, 1), down.shape[0])
    x = Lookup.apply(table, ids, scale)
    return Adapted.apply(x, w, down, up, scales, offsets, order, pos)


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

    rank, known = 8, 5000
    table = torch.randn((known, d), generator=g, device="cuda").requires_grad_()
    ids = torch.randint(0, known, (1000,), generator=g, device="cuda", dtype=torch.int32)
    shared = torch.randn((out, d), generator=g, device="cuda") / d ** 0.5
    down = (torch.randn((nlist, rank, d), generator=g, device="cuda") / d ** 0.5).requires_grad_()
    up = torch.zeros((nlist, out, rank), device="cuda").requires_grad_()
    scales = torch.full((nlist,), 0.5, device="cuda")
    lists = torch.randint(-1, nlist, (1000,), generator=g, device="cuda", dtype=torch.int32)
    y = layer_adapted(table, ids, shared, down, up, scales, lists)
    (y - goal).square().mean().backward()
    print(f"adapters: {tuple(y.shape)}, gradients of the table {float(table.grad.norm()):.2e}, "
          f"of the low-rank matrices {float(up.grad.norm()):.2e}")

    rows = torch.nn.functional.normalize(torch.randn((20000, d), generator=g, device="cuda"), dim=1)
    queries = rows[:100] + 0.05 * torch.randn((100, d), generator=g, device="cuda")
    _, found = search_4bit(rows, queries, 10)
    exact = (queries @ rows.t()).topk(10).indices
    hits = (found.long()[:, :, None] == exact[:, None, :]).any(dim=2).float().mean()
    print(f"search in 4 bits: {float(hits):.3f} of the exact 10, nearest row first in "
          f"{float((found[:, 0].long() == exact[:, 0]).float().mean()):.3f}")


if __name__ == "__main__":
    main()
