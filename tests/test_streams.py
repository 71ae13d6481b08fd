"""Where the binding takes memory from when a call is given a stream of its own
(no GPU needed: tensors, streams and the library are stand-ins)."""
import contextlib
import importlib.util
import types

import pytest
import torch

from approximate_nearest_neighbour_amd import binding as B


class OnDevice(torch.Tensor):
    """A host tensor that says it is a device tensor and notes its streams."""
    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


def dev(*shape, dtype=torch.float32):
    return torch.ones(shape, dtype=dtype).as_subclass(OnDevice)


CURRENT, SIDE = types.SimpleNamespace(cuda_stream=1), types.SimpleNamespace(cuda_stream=7)


@pytest.fixture
def world(monkeypatch):
    w = types.SimpleNamespace(active=CURRENT, made=[], called=[])
    empty = torch.empty

    def make(*shape, device=None, **kw):
        t = empty(*shape, **kw).as_subclass(OnDevice)
        w.made.append((t, w.active))
        return t

    @contextlib.contextmanager
    def stream(s):
        before, w.active = w.active, s
        yield
        w.active = before

    class Library:
        def __getattr__(self, name):
            if name == "ivfpq_route_sort_bytes":
                return lambda *a: 64

            def call(*a):
                w.called.append((name, a))
                return 0
            return call

    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.active)
    monkeypatch.setattr(B, "lib", lambda: LIB)
    LIB = Library()
    return w


def u8(*shape):
    return dev(*shape, dtype=torch.uint8)


def i32(*shape):
    return dev(*shape, dtype=torch.int32)


CALLS = {
    "mx4_quantize": (2, lambda s: B.ivfpq_mx4_quantize_ex(dev(4, 64), stream=s)),
    "mx4_dequantize": (1, lambda s: B.ivfpq_mx4_dequantize_ex(u8(4, 32), u8(4, 2), 64, stream=s)),
    "mx4_product": (1, lambda s: B.ivfpq_mx4_product_ex((u8(4, 32), u8(4, 2)),
                                                        (u8(5, 32), u8(5, 2)), stream=s)),
    "mx4_list_product": (1, lambda s: B.ivfpq_mx4_list_product_ex(
        (u8(4, 32), u8(4, 2)), (u8(3, 5, 32), u8(3, 5, 2)), i32(4), order=i32(8), k=2, stream=s)),
    "route_sort": (4, lambda s: B.ivfpq_route_sort_ex(i32(4, 2), 3, stream=s)),
    "route_gather": (1, lambda s: B.ivfpq_route_gather_ex(dev(4, 8), i32(8), 2, stream=s)),
    "route_combine": (1, lambda s: B.ivfpq_route_combine_ex(dev(8, 8), i32(4, 2), stream=s)),
    "route_combine_grad": (2, lambda s: B.ivfpq_route_combine_grad_ex(
        dev(4, 8), dev(8, 8), i32(8), i32(4, 2), dev(4, 2), stream=s)),
}


INDEX = types.SimpleNamespace(handle=1, info={"d": 8, "m": 2})
SEARCH_CALLS = {
    "search": (3, lambda s: B.ivfpq_search_ex(INDEX, dev(4, 8), 2, 3, return_probes=True,
                                              stream=s)),
    "coarse": (2, lambda s: B.ivfpq_coarse_ex(INDEX, dev(4, 8), 2, stream=s)),
    "assign_encode": (2, lambda s: B.ivfpq_assign_encode_ex(INDEX, dev(4, 8), stream=s)),
    "kmeans": (2, lambda s: B.ivfpq_kmeans_ex(dev(9, 8), dev(3, 8), 1, stream=s)),
    "compute_luts": (1, lambda s: B.ivfpq_compute_luts_ex(INDEX, dev(4, 8), i32(4, 2), stream=s)),
    "select_topk": (2, lambda s: B.ivfpq_select_topk_ex(dev(4, 8), 2, stream=s)),
    "flat_search_bf16": (2, lambda s: B.ivfpq_flat_search_bf16_ex(
        INDEX, dev(4, 8, dtype=torch.int16), 2, stream=s)),
}


@pytest.mark.parametrize("name", SEARCH_CALLS)
def test_memory_of_a_search_call_on_another_stream_is_that_streams(world, name):
    count, call = SEARCH_CALLS[name]
    call(SIDE)
    assert [stream for _, stream in world.made] == [SIDE] * count
    assert all(t.__dict__.get("recorded") == [CURRENT] for t, _ in world.made)
    (called, args), = world.called
    assert called == f"ivfpq_{name}_ex" and args[-1].value == SIDE.cuda_stream


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream_is_that_streams(world, name):
    """Memory of the current stream may still be in use there: a kernel on another
    stream may not write it.  And the caller goes on with the results on the current
    stream, so they are not given out again before that stream is past them."""
    count, call = CALLS[name]
    call(SIDE)
    assert len(world.made) == count
    for t, stream in world.made:
        assert stream is SIDE
        assert t.__dict__.get("recorded") == [CURRENT]
    (called, args), = world.called
    assert called == f"ivfpq_{name}_ex" and args[-1] == SIDE.cuda_stream
    assert world.active is CURRENT


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_the_current_stream(world, name, monkeypatch):
    monkeypatch.setattr(B, "_raw_stream", lambda s: CURRENT.cuda_stream if s is None else 0)
    count, call = CALLS[name]
    call(None)
    assert len(world.made) == count
    assert all(stream is CURRENT and "recorded" not in t.__dict__ for t, stream in world.made)
    assert world.called[0][1][-1] == CURRENT.cuda_stream


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_current_stream_without_torchs_private_calls(monkeypatch, missing):
    monkeypatch.delattr(torch._C, missing)
    spec = importlib.util.spec_from_file_location("binding_without_private_calls", B.__file__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    for handle in (5, 0):
        monkeypatch.setattr(torch.cuda, "current_stream",
                            lambda device=None: types.SimpleNamespace(cuda_stream=handle))
        assert other._raw_stream(None) == handle
    assert other._raw_stream(SIDE) == SIDE.cuda_stream
