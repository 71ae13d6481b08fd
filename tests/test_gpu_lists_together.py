"""Products per list, adapters and table rows together, as a user runs them: a table's
rows routed to lists' matrices, summed, and sent through adapters, forward and
backward; on other streams, from threads, and in captured graphs."""
import os
import sys
import threading

import numpy as np
import pytest
import torch

import approximate_nearest_neighbour_amd as A
from test_gpu_list_product import integers, np64, reals
from test_gpu_streams import check_beside_busy_stream

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import routed_layer as E  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


class Model:
    """All entries are small integers and powers of two, so that every sum is exact in
    float32 (below 2^24 in magnitude) and any difference is a fault."""

    def __init__(self, t, rows=50, d=24, n=20, m=31, nlist=5, tenants=6, r=4, k=2, seed=0):
        rng = np.random.default_rng(seed)
        small = lambda *s: torch.from_numpy(rng.integers(-1, 2, s).astype(np.float32)).cuda()  # noqa
        ints = lambda lo, hi, *s: torch.from_numpy(  # noqa: E731
            rng.integers(lo, hi, s).astype(np.int32)).cuda()
        self.table, self.matrices, self.shared = small(rows, d), small(nlist, n, d), small(m, n)
        self.down, self.up = small(tenants, r, n), small(tenants, m, r)
        self.scales = torch.tensor([1, 0.5, 2, -1, 4, 0.25], device="cuda")[:tenants]
        self.weights = torch.from_numpy(2.0 ** rng.integers(-1, 2, (t, k)).astype(np.float32)).cuda()
        self.ids, self.lists = ints(-1, rows, t), ints(-1, nlist, t, k)
        self.tenants = ints(-1, tenants, t)
        self.dy = small(t, m)
        self.k = k

    def parameters(self):
        return [self.table, self.matrices, self.down, self.up, self.weights]

    def forward(self, table, matrices, down, up, weights):
        offsets, order, pos = A.ivfpq_route_sort_ex(self.lists, len(matrices))
        x = E.Lookup.apply(table, self.ids, 2.0)
        h = E.ListProduct.apply(x, matrices, offsets, order, pos)
        z = E.Combine.apply(h, weights, order, pos)
        offsets, order, pos = A.ivfpq_route_sort_ex(self.tenants.view(-1, 1), len(down))
        return E.Adapted.apply(z, self.shared, down, up, self.scales, offsets, order, pos)

    def definition(self, table, matrices, down, up, weights):
        """The same in 64 bits on the CPU, a list at a time."""
        def pick(rows, i):
            return torch.where((i >= 0)[:, None], rows[i.clamp(min=0)], 0.0)

        ids, lists, tenants = (a.long().cpu() for a in (self.ids, self.lists, self.tenants))
        x = 2.0 * pick(table, ids)
        every = torch.stack([x @ w.t() for w in matrices], 1)          # [t, nlist, n]
        z = 0
        for j in range(self.k):
            mine = every[torch.arange(len(x)), lists[:, j].clamp(min=0)]
            z = z + torch.where((lists[:, j] >= 0)[:, None], mine, 0.0) * weights[:, j:j + 1]
        s = self.scales.double().cpu()
        extra = torch.stack([s[e] * (z @ down[e].t()) @ up[e].t() for e in range(len(down))], 1)
        mine = extra[torch.arange(len(x)), tenants.clamp(min=0)]
        return (z @ self.shared.double().cpu().t() +
                torch.where((tenants >= 0)[:, None], mine, 0.0))


@pytest.mark.parametrize("t", [1, 2, 33, 700])
def test_forward_and_gradients_are_exact(t):
    model = Model(t)
    own = [p.clone().requires_grad_() for p in model.parameters()]
    y = model.forward(*own)
    y.backward(model.dy)
    ref = [p.double().cpu().requires_grad_() for p in model.parameters()]
    want = model.definition(*ref)
    want.backward(model.dy.double().cpu())
    assert torch.equal(y.detach().double().cpu(), want.detach())
    for got, w in zip(own, ref):
        assert w.grad.abs().max() < 2 ** 24
        assert torch.equal(got.grad.double().cpu(), w.grad)


@pytest.mark.parametrize("which", range(5))
def test_gradients_against_differences(which):
    """The result is linear in each parameter alone, so its difference along a direction
    is the gradient's product with it, exactly."""
    model = Model(90, seed=which)
    own = [p.clone().requires_grad_() for p in model.parameters()]
    model.forward(*own).backward(model.dy)
    step = torch.zeros_like(own[which])
    rng = np.random.default_rng(which)
    flat = step.view(-1)
    flat[torch.from_numpy(rng.integers(0, flat.numel(), 60)).cuda()] = 1.0
    ends = []
    for sign in (1, -1):
        moved = [p.detach().clone() for p in own]
        moved[which] += sign * step
        ends.append((model.forward(*moved).double() * model.dy.double()).sum())
    assert float(ends[0] - ends[1]) == 2 * float((own[which].grad.double() * step.double()).sum())


def test_example_adapters():
    g = torch.Generator(device="cuda").manual_seed(2)
    make = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t, rows, d, n, nlist, r = 64, 40, 48, 33, 4, 5
    table, down, up = (p.requires_grad_() for p in (make(rows, d), make(nlist, r, d),
                                                    make(nlist, n, r)))
    w, scales, dy = make(n, d), make(nlist), make(t, n)
    ids = torch.randint(-1, rows, (t,), generator=g, device="cuda", dtype=torch.int32)
    lists = torch.randint(-1, nlist, (t,), generator=g, device="cuda", dtype=torch.int32)
    y = E.layer_adapted(table, ids, w, down, up, scales, lists, scale=0.5)
    y.backward(dy)
    ref = [p.detach().double().cpu().requires_grad_() for p in (table, down, up)]
    mags = [p.detach().abs() for p in ref]

    def layer(table, down, up, w, scales):
        i, e = ids.long().cpu(), lists.long().cpu()
        x = torch.where((i >= 0)[:, None], 0.5 * table[i.clamp(min=0)], 0.0)
        per = torch.stack([s * (x @ a.t()) @ b.t() for a, b, s in zip(down, up, scales)], 1)
        return x @ w.t() + torch.where((e >= 0)[:, None], per[torch.arange(t), e.clamp(min=0)], 0.0)

    want = layer(*ref, w.double().cpu(), scales.double().cpu())
    want.backward(dy.double().cpu())
    mags = [p.requires_grad_() for p in mags]
    size = layer(*mags, w.double().cpu().abs(), scales.double().cpu().abs())
    size.backward(dy.double().cpu().abs())
    # A result passes at most three sums, of no more than t, d, n and r terms in turn; a sum of
    # K terms is off by (6 K + 4) 2^-23 of its terms' magnitudes, products and roundings
    # between them included.
    tol = 1.01 * 2.0 ** -23 * (6 * (t + d + n + r) + 16)
    assert ((y.detach().double().cpu() - want.detach()).abs() <= tol * size.detach()).all()
    for got, p, m in zip((table, down, up), ref, mags):
        assert ((got.grad.double().cpu() - p.grad).abs() <= tol * m.grad).all()


def calls(dtype=torch.bfloat16, t=900, d=96, n=72, nlist=12, r=8, rows=300, workspaces=None):
    """Every operator on the same rows: name -> (call(stream), bytes of its workspace)."""
    rng = np.random.default_rng(3)
    x, grad = reals(rng, t, d, dtype=dtype), reals(rng, t, n, dtype=dtype)
    w, shared = reals(rng, nlist, n, d, dtype=dtype), reals(rng, n, d, dtype=dtype)
    down, up = reals(rng, nlist, r, d, dtype=dtype), reals(rng, nlist, n, r, dtype=dtype)
    lists = torch.from_numpy(rng.integers(-1, nlist, (t, 1)).astype(np.int32)).cuda()
    ids = torch.from_numpy(rng.integers(-1, rows, (t, 1)).astype(np.int32)).cuda()
    table = reals(rng, rows, d, dtype=dtype)
    offsets, order, pos = A.ivfpq_route_sort_ex(lists, nlist)
    toffsets, torder, _ = A.ivfpq_route_sort_ex(ids, rows)
    one = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    many = torch.cat([x] * 8)
    many_grad = torch.cat([grad] * 8)
    all_rows = torch.tensor([0, 8 * t], dtype=torch.int32, device="cuda")
    sizes = {"grad": A.ivfpq_list_product_grad_bytes(t, n, d, nlist),
             "grad_shared": A.ivfpq_list_product_grad_bytes(8 * t, n, d, 1),
             "adapter": A.ivfpq_adapter_product_bytes(t, r),
             "table_grad": A.ivfpq_table_grad_bytes(t, d)}
    ws = workspaces if workspaces is not None else {}
    return {
        "product": lambda s: A.ivfpq_list_product_ex(x, w, offsets, order=order, stream=s),
        "product_across": lambda s: A.ivfpq_list_product_ex(grad, w, offsets, transposed=True,
                                                            stream=s),
        "one_list": lambda s: A.ivfpq_list_product_ex(x, shared[None], one, stream=s),
        "grad": lambda s: A.ivfpq_list_product_grad_ex(grad, x, offsets, order=order, stream=s,
                                                       workspace=ws.get("grad")),
        "grad_shared": lambda s: A.ivfpq_list_product_grad_ex(
            many_grad, many, all_rows, stream=s, workspace=ws.get("grad_shared")),
        "adapter": lambda s: A.ivfpq_adapter_product_ex(x, shared, down, up, offsets, order, pos,
                                                        stream=s, workspace=ws.get("adapter")),
        "lookup": lambda s: A.ivfpq_table_lookup_ex(table, ids, stream=s),
        "table_grad": lambda s: A.ivfpq_table_grad_ex(x, toffsets, torder, stream=s,
                                                      workspace=ws.get("table_grad")),
    }, sizes


NAMES = ["product", "product_across", "one_list", "grad", "grad_shared", "adapter", "lookup",
         "table_grad"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name, dtype):
    all_calls, sizes = calls(dtype)
    check_beside_busy_stream(all_calls[name], [sizes[name]] if name in sizes else ())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_together_and_replayed(dtype):
    """All of them in one graph, twice, with workspaces that both graphs share; eager
    calls, and other values in the inputs' place, between the replays."""
    ws = {}
    all_calls, sizes = calls(dtype, workspaces=ws)
    for name, need in sizes.items():
        ws[name] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    want = {name: call(None).clone() for name, call in all_calls.items()}
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results = {name: call(None) for name, call in all_calls.items()}
        graphs.append((graph, results))
    for turn in range(4):
        for graph, results in graphs:
            for out in results.values():
                out.fill_(float("nan"))
            for w in ws.values():
                w.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            for name in all_calls:
                assert torch.equal(results[name], want[name]), (turn, name)
        for name in NAMES[turn::4]:
            assert torch.equal(all_calls[name](None), want[name])


def test_a_graph_follows_its_inputs():
    """A captured sort, product and gradient serve other lists and rows."""
    rng = np.random.default_rng(12)
    t, d, n, nlist = 300, 64, 48, 7
    x, w = integers(rng, t, d, dtype=torch.bfloat16), integers(rng, nlist, n, d, dtype=torch.bfloat16)
    lists = torch.zeros((t, 1), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()

    def run():
        offsets, order, pos = A.ivfpq_route_sort_ex(lists, nlist)
        y = A.ivfpq_list_product_ex(x, w, offsets, order=order)
        return A.ivfpq_route_combine_ex(y, pos), A.ivfpq_list_product_grad_ex(y, x, offsets,
                                                                             order=order)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    with torch.cuda.graph(graph, stream=stream):
        y, g = run()
    for high in (1, nlist, 3, nlist):
        new = rng.integers(-1, high, (t, 1)).astype(np.int32)
        lists.copy_(torch.from_numpy(new))
        x.copy_(integers(rng, t, d, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        assert torch.equal(y, eager[0]) and torch.equal(g, eager[1])
        mine = np64(w)[np.maximum(new[:, 0], 0)] * (new[:, :1, None] >= 0)
        want = np.einsum("tnd,td->tn", mine, np64(x))
        assert np.array_equal(np64(y), np64(torch.from_numpy(want).to(torch.bfloat16)))


def test_threads_with_streams_of_their_own():
    all_calls, _ = calls()
    want = {name: call(None).clone() for name, call in all_calls.items()}
    torch.cuda.synchronize()
    wrong = []

    def work(names):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                for name in names:
                    if not torch.equal(all_calls[name](None), want[name]):
                        wrong.append(name)
    threads = [threading.Thread(target=work, args=(NAMES[i:] + NAMES[:i],)) for i in (0, 2, 4, 6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_adapters_in_every_type(dtype):
    """Small integers and powers of two, sums that 8 bits hold, so that every type's
    gradients are exact, rounded once."""
    rng = np.random.default_rng(21)
    t, n, d, nlist, r = 90, 20, 12, 4, 2
    small = lambda *s: torch.from_numpy(  # noqa: E731
        rng.integers(-1, 2, s).astype(np.float32)).to(dtype).cuda()
    x, down, up = (p.requires_grad_() for p in (small(t, d), small(nlist, r, d), small(nlist, n, r)))
    w, dy = small(n, d), small(t, n)
    scales = torch.tensor([1, 0.5, 2, -1], device="cuda")
    lists = torch.from_numpy(rng.integers(-1, nlist, t).astype(np.int32)).cuda()
    y = E.Adapted.apply(x, w, down, up, scales,
                        *A.ivfpq_route_sort_ex(lists.view(-1, 1), nlist))
    y.backward(dy)
    ref = [p.detach().double().cpu().requires_grad_() for p in (x, down, up)]
    e = lists.long().cpu()
    per = torch.stack([s * (ref[0] @ a.t()) @ b.t()
                       for a, b, s in zip(ref[1], ref[2], scales.double().cpu())], 1)
    want = ref[0] @ w.double().cpu().t() + torch.where(
        (e >= 0)[:, None], per[torch.arange(t), e.clamp(min=0)], 0.0)
    want.backward(dy.double().cpu())
    assert torch.equal(y.detach().cpu(), want.detach().to(dtype))
    for got, p in zip((x, down, up), ref):
        assert got.grad.dtype == dtype and torch.equal(got.grad.cpu(), p.grad.to(dtype))
