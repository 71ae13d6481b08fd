"""Calls on a stream of their own while the current one is busy: right results,
and memory that was freed on the current stream with work still to come is left
alone."""
import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from approximate_nearest_neighbour_amd import datagen as G
from test_gpu_mx4 import cuda, make_lists, random_mx4

pytestmark = pytest.mark.gpu


def tensors(result):
    return [result] if isinstance(result, torch.Tensor) else list(result)


def check_beside_busy_stream(call, temporary=()):
    """call(stream): its results beside a busy current stream, against those alone;
    temporary: bytes of the workspaces that the binding allocates."""
    want = [t.clone() for t in tensors(call(None))]
    big = torch.randn((4096, 4096), device="cuda") / 64
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want] + list(temporary)
    torch.cuda.synchronize()
    victims = [torch.full((max(n, 1),), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]
    x = big
    for _ in range(20):           # tens of milliseconds of work
        x = x @ big
    copies = [v.clone() for v in victims]
    victims = None                # freed, and read by what is still to run
    got = tensors(call(side))
    torch.cuda.synchronize()
    for c in copies:
        assert (c == 0x5A).all()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def case(name):
    rng = np.random.default_rng(3)
    t, k, nlist, n, d = 6000, 2, 40, 72, 96
    x = torch.from_numpy(rng.standard_normal((t, d)).astype(np.float32)).cuda()
    rows = torch.from_numpy(rng.standard_normal((t * k, d)).astype(np.float32)).cuda()
    weights = torch.from_numpy(rng.random((t, k)).astype(np.float32)).cuda()
    lists = torch.from_numpy(make_lists(rng, t, k, nlist, 0.1)).cuda()
    offsets, order, pos = A.ivfpq_route_sort_ex(lists, nlist)
    a = cuda(random_mx4(rng, t, d))
    b = cuda(random_mx4(rng, nlist * n, d))
    per = tuple(m.view(nlist, n, -1) for m in b)
    return {
        "quantize": lambda s: A.ivfpq_mx4_quantize_ex(x, stream=s),
        "dequantize": lambda s: A.ivfpq_mx4_dequantize_ex(*a, d, stream=s),
        "product": lambda s: A.ivfpq_mx4_product_ex(a, b, stream=s),
        "list_product": lambda s: A.ivfpq_mx4_list_product_ex(a, per, offsets, order=order, k=k,
                                                              stream=s),
        "sort": lambda s: A.ivfpq_route_sort_ex(lists, nlist, stream=s),
        "gather": lambda s: A.ivfpq_route_gather_ex(x, order, k, weights=weights, stream=s),
        "combine": lambda s: A.ivfpq_route_combine_ex(rows, pos, weights, stream=s),
        "combine_grad": lambda s: A.ivfpq_route_combine_grad_ex(x, rows, order, pos, weights,
                                                                stream=s),
    }[name], [A.ivfpq_route_sort_bytes(t, k, nlist)] if name == "sort" else ()


@pytest.mark.parametrize("name", ["quantize", "dequantize", "product", "list_product", "sort",
                                  "gather", "combine", "combine_grad"])
def test_rows_and_routing_on_another_stream(name):
    check_beside_busy_stream(*case(name))


def test_searches_and_building_on_another_stream():
    rng = np.random.default_rng(5)
    ix = A.ivfpq_load_index_host(G.random_index(rng, 64, 32, 8, rng.integers(10, 200, size=64)))
    q = torch.from_numpy(rng.standard_normal((3000, 32)).astype(np.float32)).cuda()
    probes, _ = A.ivfpq_coarse_ex(ix, q[:40], 4)
    flat = A.ivfpq_flat_load_bf16(G.to_bf16_bits(rng.uniform(-1, 1, (2000, 32)).astype(np.float32)))
    qb = q.to(torch.bfloat16)
    centers = iter([q[:50].clone(), q[:50].clone()])   # updated in place, a copy for each call
    for call in (lambda s: A.ivfpq_search_ex(ix, q, 4, 10, return_probes=True, stream=s),
                 lambda s: A.ivfpq_coarse_ex(ix, q, 4, stream=s),
                 lambda s: A.ivfpq_assign_encode_ex(ix, q, stream=s),
                 lambda s: A.ivfpq_kmeans_ex(q, next(centers), 1, stream=s),
                 lambda s: A.ivfpq_compute_luts_ex(ix, q[:40], probes, stream=s),
                 lambda s: A.ivfpq_select_topk_ex(q, 5, stream=s),
                 lambda s: A.ivfpq_flat_search_bf16_ex(flat, qb, 7, stream=s)):
        check_beside_busy_stream(call)
    ix.close()
    flat.close()


def test_given_stream_while_it_is_captured():
    lists = torch.empty((6000, 2), dtype=torch.int32, device="cuda")
    x = torch.empty((6000, 96), device="cuda")
    side = torch.cuda.Stream()

    def step(stream):
        offsets, order, pos = A.ivfpq_route_sort_ex(lists, 40, stream=stream)
        rows = A.ivfpq_route_gather_ex(x, order, 2, stream=stream)
        return offsets, order, pos, A.ivfpq_route_combine_ex(rows, pos, stream=stream)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        lists.copy_(torch.randint(-1, 40, lists.shape, generator=g, device="cuda"))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))

    fill(0)
    step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step(side)
    for seed in range(1, 5):
        fill(seed)
        want = step(None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(held, want):
            assert torch.equal(got, w), seed
