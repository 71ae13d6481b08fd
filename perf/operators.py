"""Cases and plain forms of the 4-bit products and the list routing.

Kinds of case, each an operator or the operators that are called together:

* ``quantize``: rows to microscaled 4-bit floats (blocks of 32 values, e2m1
  elements, one power-of-two scale a block) and back to the values they
  stand for;
* ``product``: A B^T of two matrices held in that form;
* ``list_product``: rows sorted by list times their list's own matrix;
* ``route``: (vector, list) pairs sorted by list, the vectors gathered in that
  order, and rows in that order summed back to their vectors with weights;
* ``route_grad``: the gradients of the gather and of the weighted sum.

``own`` false computes the plain forms (elementary torch operations in
float32), ``own`` true calls the library.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the activations of a small decoding batch before a 4-bit product
        dict(name="quantize_step", kind="quantize", rows=16, d=2048, type="bf16"),
        # a database of a million 96-dimensional vectors packed once
        dict(name="quantize_database", kind="quantize", rows=1000000, d=96, type="f32"),
        # one vector through a weight matrix: a single token, bound by latency
        # and by the weights' bytes
        dict(name="product_single", kind="product", m=1, n=8192, d=4096, type="bf16"),
        # a query batch scored against 262,144 centroids of dimension 96: short
        # sums (three blocks), a large float32 result
        dict(name="product_centroids", kind="product", m=1000, n=262144, d=96, type="f32"),
        # a long prompt through a large square matrix: bound by the matrix cores
        dict(name="product_prompt", kind="product", m=8192, n=8192, d=8192, type="bf16"),
        # four tokens with eight lists each: most lists get no row, the rest one
        dict(name="list_step", kind="list_product", t=4, k=8, lists=64, n=2048, d=2048,
             skew=0.5, drop=0.0, type="bf16"),
        # an odd batch, odd sizes, a few masked slots, uneven lists
        dict(name="list_batch", kind="list_product", t=777, k=2, lists=16, n=1501, d=1000,
             skew=1.0, drop=0.05, type="f16"),
        # a prompt's rows over 128 lists of very different sizes
        dict(name="list_prompt", kind="list_product", t=8192, k=8, lists=128, n=2048, d=2048,
             skew=1.0, drop=0.0, type="bf16"),
        # a decoding batch's tokens there and back
        dict(name="route_step", kind="route", t=64, k=8, lists=64, d=2048, skew=0.5, drop=0.0,
             type="bf16"),
        # 10,000 queries of dimension 128 with 32 probes each of 1024 lists
        dict(name="route_queries", kind="route", t=10000, k=32, lists=1024, d=128, skew=1.1,
             drop=0.0, type="f32"),
        # a small training batch of odd width with masked slots
        dict(name="route_grad_small", kind="route_grad", t=500, k=2, lists=8, d=1001, skew=1.0,
             drop=0.1, type="f32"),
        # a training batch of 16,384 tokens with eight lists each
        dict(name="route_grad_batch", kind="route_grad", t=16384, k=8, lists=128, d=2048, skew=1.0,
             drop=0.02, type="bf16"),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3072 else n


def draw(rng):
    kind = rng.choice(["quantize", "product", "product", "list_product", "list_product", "route",
                       "route_grad"])
    kind_type = rng.choice(sorted(TYPES))
    if kind == "quantize":
        d = _log_int(rng, 1, 8192)
        return dict(kind=kind, rows=_log_int(rng, 1, min(1000000, 96000000 // d)), d=d,
                    type=kind_type)
    if kind == "product":
        m = _log_int(rng, 1, 8192)
        d = _log_int(rng, 32, 8192)
        n = _log_int(rng, 16, min(262144, 8192 ** 3 // (m * d), 262144000 // m))
        return dict(kind=kind, m=m, n=n, d=d, type=kind_type)
    t = _log_int(rng, 1, 8192)
    k = rng.choice([1, 2, 4, 6, 8])
    lists = _log_int(rng, 8, 128)
    skew = round(rng.uniform(0.0, 1.2), 2)
    drop = rng.choice([0.0, 0.0, 0.03, 0.2])
    if kind == "list_product":
        return dict(kind=kind, t=t, k=k, lists=lists, n=_log_int(rng, 16, 2048),
                    d=_log_int(rng, 32, 2048), skew=skew, drop=drop, type=kind_type)
    if kind == "route" and rng.random() < 0.5:  # many lists and probes, short rows
        k = rng.choice([1, 8, 16, 32])
        return dict(kind=kind, t=_log_int(rng, 1, 10000), k=k, lists=_log_int(rng, 64, 1024),
                    d=_log_int(rng, 1, 128), skew=skew, drop=drop, type=kind_type)
    return dict(kind=kind, t=t, k=k, lists=lists, d=_log_int(rng, 1, 2048), skew=skew, drop=drop,
                type=kind_type)


def work(case):
    d, kind = case["d"], case["kind"]
    packed = -(-d // BLOCK) * 17  # bytes of one packed row: 16 of codes and 1 of scale a block
    out = SIZE[case["type"]]
    if kind == "quantize":
        rows = case["rows"]
        return {"bytes": rows * (2 * d * out + 2 * packed), "flops": 4 * rows * d}
    if kind == "product":
        m, n = case["m"], case["n"]
        return {"bytes": (m + n) * packed + m * n * out, "flops": 2 * m * n * d}
    t, k, lists = case["t"], case["k"], case["lists"]
    rows = t * k
    if kind == "list_product":
        n = case["n"]
        return {"bytes": t * packed + min(lists, rows) * n * packed + rows * n * out + 8 * rows,
                "flops": 2 * rows * n * d}
    if kind == "route":
        return {"bytes": 2 * (t + rows) * d * out + rows * 16 + 4 * lists,
                "flops": 2 * rows * d}
    return {"bytes": (2 * t + 3 * rows) * d * out + rows * 20, "flops": 4 * rows * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _values(g, *shape):
    """Activations and vectors: normal, each column with a scale of its own
    and one column in 64 much larger, as hidden states have."""
    x = torch.randn(shape, generator=g, device=DEVICE)
    scale = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=DEVICE))
    large = torch.rand(shape[-1], generator=g, device=DEVICE) < 1.0 / 64
    return x.mul_(torch.where(large, 8.0 * scale, scale))


def _pack(x):
    """Rows in the 4-bit form, (codes [..., rows, 16 kb], scales [..., rows, kb])."""
    codes, scales = [], []
    flat = x.reshape(-1, x.shape[-1])
    step = max(1, (1 << 26) // flat.shape[1])
    for part in flat.split(step):
        q, s = _plain_quantize(part)
        codes.append(q)
        scales.append(s)
    lead = x.shape[:-1]
    return torch.cat(codes).reshape(*lead, -1), torch.cat(scales).reshape(*lead, -1)


def _lists(g, case):
    """Lists of each vector, [t, k] int32: k different ones a vector, list l
    chosen with weight (l + 1)^-skew in a shuffled order; masked slots are -1."""
    t, k, lists = case["t"], case["k"], case["lists"]
    weight = -case["skew"] * torch.log(torch.arange(1, lists + 1, device=DEVICE,
                                                    dtype=torch.float32))
    weight = weight[torch.randperm(lists, generator=g, device=DEVICE)]
    u = torch.rand((t, lists), generator=g, device=DEVICE).clamp_(1e-7, 1 - 1e-7)
    ids = (weight - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32)
    if case["drop"]:
        ids = torch.where(torch.rand((t, k), generator=g, device=DEVICE) < case["drop"], -1, ids)
    return ids.to(torch.int32).contiguous()


def _weights(g, case):
    return torch.softmax(torch.randn((case["t"], case["k"]), generator=g, device=DEVICE), dim=1)


def prepare(case, seed):
    g = _generator(seed)
    kind, d = case["kind"], case["d"]
    dtype = TYPES[case["type"]]
    state = dict(case=case, dtype=dtype)
    if kind == "quantize":
        state["x"] = _values(g, case["rows"], d).to(dtype)
    elif kind == "product":
        state["a"] = _pack(_values(g, case["m"], d))
        state["b"] = _pack(torch.randn((case["n"], d), generator=g, device=DEVICE))
    elif kind == "list_product":
        state["a"] = _pack(_values(g, case["t"], d))
        state["b"] = _pack(torch.randn((case["lists"], case["n"], d), generator=g, device=DEVICE))
        state["offsets"], state["order"], _ = _plain_sort(_lists(g, case), case["lists"])
    else:
        t, k = case["t"], case["k"]
        state["ids"] = _lists(g, case)
        state["weights"] = _weights(g, case)
        state["rows"] = _values(g, t * k, d).to(dtype)  # what the lists' products gave
        state["x"] = _values(g, t, d).to(dtype)
        if kind == "route_grad":
            _, state["order"], state["pos"] = _plain_sort(state["ids"], case["lists"])
            state["grad"] = state.pop("x")               # of the weighted sum
            state["grad_rows"] = torch.randn((t * k, d), generator=g,
                                             device=DEVICE).to(dtype)  # of the gathered rows
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_quantize(x):
    x = x.float()
    rows, d = x.shape
    kb = -(-d // BLOCK)
    x = torch.nn.functional.pad(x, (0, kb * BLOCK - d)).view(rows, kb, BLOCK)
    amax = x.abs().amax(dim=2)
    exponent = amax.view(torch.int32) >> 23
    scale = (exponent - 2).clamp(min=0)
    y = x * ((254 - scale) << 23).view(torch.float32).unsqueeze(2)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (y < 0).to(torch.uint8)
    bad = exponent == 255
    code = torch.where(bad.unsqueeze(2), 0, code).to(torch.uint8).view(rows, -1)
    scale = torch.where(bad, 255, scale).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def _plain_dequantize(codes, scales, d):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    low, high = table[(codes & 15).int()], table[(codes >> 4).int()]
    v = torch.stack([low, high], dim=-1).view(*scales.shape, BLOCK)
    s = scales.int()
    # 2^(s - 127) as two factors, so that the smallest scales stay exact
    f = ((s.clamp(min=1)) << 23).view(torch.float32) * torch.where(s == 0, 0.5, 1.0)
    f = torch.where(s == 255, math.nan, f)
    return (v * f.unsqueeze(-1)).view(*scales.shape[:-1], -1)[..., :d]


def _plain_sort(ids, lists):
    t, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < lists), flat, lists)
    key, slot = torch.sort(key, stable=True)
    bounds = torch.arange(lists + 1, device=ids.device)
    offsets = torch.searchsorted(key, bounds).to(torch.int32)
    kept = key < lists
    order = torch.where(kept, slot, -1).to(torch.int32)
    pos = torch.empty_like(slot)
    pos[slot] = torch.where(kept, torch.arange(t * k, device=ids.device), -1)
    return offsets, order, pos.to(torch.int32).view(t, k)


def _plain_gather(x, order, k):
    rows = x[(order.clamp(min=0) // k).long()]
    return torch.where((order >= 0).unsqueeze(1), rows, 0)


def _plain_combine(rows, pos, weights):
    y = torch.zeros((pos.shape[0], rows.shape[1]), device=rows.device)
    for j in range(pos.shape[1]):
        p = pos[:, j]
        r = rows[p.clamp(min=0).long()].float()
        if weights is not None:
            r = r * weights[:, j].unsqueeze(1)
        y = y + torch.where((p >= 0).unsqueeze(1), r, 0.0)
    return y.to(rows.dtype)


def _plain_combine_grad(grad, rows, order, pos, weights):
    k = pos.shape[1]
    slot = order.clamp(min=0).long()
    d_rows = grad[slot // k].float() * weights.reshape(-1)[slot].unsqueeze(1)
    d_rows = torch.where((order >= 0).unsqueeze(1), d_rows, 0.0).to(rows.dtype)
    d_weights = torch.empty(pos.shape, device=rows.device)
    for j in range(k):
        p = pos[:, j]
        dot = (grad.float() * rows[p.clamp(min=0).long()].float()).sum(dim=1)
        d_weights[:, j] = torch.where(p >= 0, dot, 0.0)
    return d_rows, d_weights


def _plain(state):
    case, dtype = state["case"], state["dtype"]
    kind, d = case["kind"], case["d"]
    if kind == "quantize":
        return _plain_dequantize(*_plain_quantize(state["x"]), d).to(dtype)
    if kind == "product":
        a, b = _plain_dequantize(*state["a"], d), _plain_dequantize(*state["b"], d)
        return (a @ b.t()).to(dtype)
    if kind == "list_product":
        order = state["order"]
        a = _plain_gather(_plain_dequantize(*state["a"], d), order, case["k"])
        out = torch.zeros((order.numel(), case["n"]), dtype=dtype, device=DEVICE)
        bounds = state["offsets"].tolist()
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            if lo < hi:
                w = _plain_dequantize(state["b"][0][e], state["b"][1][e], d)
                out[lo:hi] = (a[lo:hi] @ w.t()).to(dtype)
        return out
    if kind == "route":
        offsets, order, pos = _plain_sort(state["ids"], case["lists"])
        return (offsets, order, pos, _plain_gather(state["x"], order, case["k"]),
                _plain_combine(state["rows"], pos, state["weights"]))
    d_rows, d_weights = _plain_combine_grad(state["grad"], state["rows"], state["order"],
                                            state["pos"], state["weights"])
    return d_rows, d_weights, _plain_combine(state["grad_rows"], state["pos"], None)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _library(state):
    import approximate_nearest_neighbour_amd as A

    case, dtype = state["case"], state["dtype"]
    kind = case["kind"]
    if kind == "quantize":
        codes, scales = A.ivfpq_mx4_quantize_ex(state["x"])
        return A.ivfpq_mx4_dequantize_ex(codes, scales, case["d"], dtype=dtype)
    if kind == "product":
        return A.ivfpq_mx4_product_ex(state["a"], state["b"], dtype=dtype)
    if kind == "list_product":
        return A.ivfpq_mx4_list_product_ex(state["a"], state["b"], state["offsets"],
                                           order=state["order"], k=case["k"], dtype=dtype)
    if kind == "route":
        offsets, order, pos = A.ivfpq_route_sort_ex(state["ids"], case["lists"])
        return (offsets, order, pos, A.ivfpq_route_gather_ex(state["x"], order, case["k"]),
                A.ivfpq_route_combine_ex(state["rows"], pos, state["weights"]))
    d_rows, d_weights = A.ivfpq_route_combine_grad_ex(state["grad"], state["rows"],
                                                      state["order"], state["pos"],
                                                      state["weights"])
    return d_rows, d_weights, A.ivfpq_route_combine_ex(state["grad_rows"], state["pos"])


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_values(codes, scales, d):
    """The numbers that 4-bit rows stand for: sign, two exponent bits, one
    mantissa bit, times 2^(scale - 127)."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, m * 0.5, (1.0 + 0.5 * m) * torch.exp2((e - 1).double()))
    v = torch.where(n >= 8, -v, v)
    s = torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=-1)
    return (v * s)[..., :d]


def _exact_quantize(x):
    out = []
    for part in x.split(max(1, (1 << 25) // x.shape[1])):
        v = part.double()
        rows, d = v.shape
        kb = -(-d // BLOCK)
        v = torch.cat([v, v.new_zeros(rows, kb * BLOCK - d)], dim=1).view(rows, kb, BLOCK)
        top = v.abs().amax(dim=2, keepdim=True)
        _, e = torch.frexp(top)                       # top = f 2^e, f in [1/2, 1)
        e = torch.where(top == 0, -127, (e - 1).clamp(min=-125) - 2)
        unit = torch.exp2(e.double())
        y = (v / unit).abs()
        step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
        y = (torch.round(y / step) * step).clamp(max=6.0)  # halves to even
        out.append((torch.sign(v) * y * unit).view(rows, -1)[:, :d].to(torch.float64))
    return torch.cat(out)


def exact(case, seed):
    state = prepare(case, seed)
    kind, d = case["kind"], case["d"]
    if kind == "quantize":
        return _exact_quantize(state["x"])
    if kind == "product":
        return torch.matmul(_exact_values(*state["a"], d), _exact_values(*state["b"], d).t())
    if kind == "list_product":
        order, offsets = state["order"].cpu(), state["offsets"].cpu()
        a = _exact_values(*state["a"], d)
        out = torch.zeros((order.numel(), case["n"]), dtype=torch.float64, device=DEVICE)
        for e in range(case["lists"]):
            span = slice(int(offsets[e]), int(offsets[e + 1]))
            if span.start < span.stop:
                w = _exact_values(state["b"][0][e], state["b"][1][e], d)
                source = torch.div(order[span], case["k"], rounding_mode="floor").long()
                out[span] = torch.matmul(a[source.to(DEVICE)], w.t())
        return out
    t, k, lists = case["t"], case["k"], case["lists"]
    ids = state["ids"].cpu().reshape(-1).tolist()
    weights = state["weights"].double()
    slots = [[] for _ in range(lists)]
    for slot, e in enumerate(ids):
        if 0 <= e < lists:
            slots[e].append(slot)
    sizes = torch.tensor([0] + [len(s) for s in slots], dtype=torch.int64)
    offsets = torch.cumsum(sizes, 0)
    kept = torch.tensor([s for group in slots for s in group], dtype=torch.int64)
    order = torch.full((t * k,), -1, dtype=torch.int64)
    order[:kept.numel()] = kept
    pos = torch.full((t * k,), -1, dtype=torch.int64)
    pos[kept] = torch.arange(kept.numel())
    kept = kept.to(DEVICE)
    token = kept // k

    def back(rows, scale):
        y = torch.zeros((t, d), dtype=torch.float64, device=DEVICE)
        part = rows[:kept.numel()].double()
        if scale is not None:
            part = part * scale.reshape(-1)[kept].unsqueeze(1)
        return y.index_add_(0, token, part)

    if kind == "route":
        rows = torch.zeros((t * k, d), dtype=torch.float64, device=DEVICE)
        rows[:kept.numel()] = state["x"].double()[token]
        return (offsets.to(torch.int32).to(DEVICE), order.to(torch.int32).to(DEVICE),
                pos.to(torch.int32).view(t, k).to(DEVICE), rows, back(state["rows"], weights))
    grad = state["grad"].double()[token]
    d_rows = torch.zeros((t * k, d), dtype=torch.float64, device=DEVICE)
    d_rows[:kept.numel()] = grad * weights.reshape(-1)[kept].unsqueeze(1)
    d_weights = torch.zeros(t * k, dtype=torch.float64, device=DEVICE)
    d_weights[kept] = (grad * state["rows"][:kept.numel()].double()).sum(dim=1)
    return d_rows, d_weights.view(t, k), back(state["grad_rows"], None)
