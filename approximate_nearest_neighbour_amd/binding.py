"""Thin ctypes binding over ``libivfpq.so`` (declared in include/ivfpq.h).

Argument marshalling only: every step of the search runs in the library's
HIP kernels.  PyTorch supplies device memory and the HIP stream; it is
imported before the library is loaded so both share one HIP runtime.  There
is no fallback: if the library is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libivfpq.so")

OK, E_INVALID_ARG, E_IO, E_FORMAT, E_NO_DEVICE, E_OUT_OF_MEMORY, E_DEVICE = range(7)
METRIC_L2, METRIC_IP = 0, 1
LUT_F32, LUT_F16 = 0, 1
MODE_NORMAL, MODE_SCAN_ONLY = 0, 1


class IVFPQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class SearchParams(ctypes.Structure):
    _fields_ = [("nprobe", ctypes.c_int32), ("k", ctypes.c_int32), ("lut", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("chunk_len", ctypes.c_int32),
                ("metric", ctypes.c_int32)]


class Info(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("nlist", ctypes.c_int32), ("m", ctypes.c_int32),
                ("nbits", ctypes.c_int32), ("ntotal", ctypes.c_int64),
                ("max_list", ctypes.c_int64), ("device", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("device_bytes", ctypes.c_int64)]


class HostIndexStruct(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("nlist", ctypes.c_int32), ("m", ctypes.c_int32),
                ("nbits", ctypes.c_int32), ("ntotal", ctypes.c_int64),
                ("centroids", ctypes.c_void_p), ("codebooks", ctypes.c_void_p),
                ("list_sizes", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("ids", ctypes.c_void_p)]


class Timings(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("coarse_ms", ctypes.c_double), ("worklist_ms", ctypes.c_double),
                ("scan_ms", ctypes.c_double), ("merge_ms", ctypes.c_double),
                ("total_ms", ctypes.c_double), ("scanned_entries", ctypes.c_int64),
                ("work_items", ctypes.c_int64)]


class FlatTimings(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("minima_ms", ctypes.c_double), ("kth_ms", ctypes.c_double),
                ("collect_ms", ctypes.c_double), ("select_ms", ctypes.c_double),
                ("fallback_ms", ctypes.c_double), ("total_ms", ctypes.c_double)]


EXPORTS = ("ivfpq_validate_index_file", "ivfpq_validate_host_index", "ivfpq_load_index",
           "ivfpq_load_index_host", "ivfpq_free_index", "ivfpq_index_info", "ivfpq_search",
           "ivfpq_search_ex", "ivfpq_search_noalloc_ex", "ivfpq_coarse_ex", "ivfpq_assign_encode_ex", "ivfpq_kmeans_ex",
           "ivfpq_build_index_ex", "ivfpq_index_export",
           "ivfpq_compute_luts_ex",
           "ivfpq_select_topk_ex",
           "ivfpq_profile_begin",
           "ivfpq_profile_end", "ivfpq_flat_load_bf16", "ivfpq_flat_free",
           "ivfpq_flat_search_bf16_ex", "ivfpq_flat_search_bf16", "ivfpq_flat_profile_begin",
           "ivfpq_flat_profile_end", "ivfpq_mx4_quantize_ex", "ivfpq_mx4_dequantize_ex",
           "ivfpq_mx4_product_ex", "ivfpq_mx4_list_product_ex", "ivfpq_route_sort_bytes",
           "ivfpq_route_sort_ex", "ivfpq_route_gather_ex", "ivfpq_route_combine_ex",
           "ivfpq_route_combine_grad_ex", "ivfpq_stream_read", "ivfpq_last_error",
           "ivfpq_status_string")

_lib = None


def lib():
    """Load libivfpq.so (built in-tree by build_lib.py); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(the IVF-PQ search has no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        st = ctypes.c_int
        sig = {
            "ivfpq_validate_index_file": ([ctypes.c_char_p], st),
            "ivfpq_validate_host_index": ([P], st),
            "ivfpq_load_index": ([ctypes.c_char_p, i32, P], st),
            "ivfpq_load_index_host": ([P, i32, P], st),
            "ivfpq_free_index": ([P], None),
            "ivfpq_index_info": ([P, P], st),
            "ivfpq_search": ([P, P, i64, i32, i32, P, P], st),
            "ivfpq_search_ex": ([P, P, P, i64, P, P, P, P], st),
            "ivfpq_search_noalloc_ex": ([P, P, P, i64, P, P, P, P], st),
            "ivfpq_coarse_ex": ([P, P, i64, i32, P, P, P], st),
            "ivfpq_assign_encode_ex": ([P, P, i64, P, P, P], st),
            "ivfpq_kmeans_ex": ([P, i64, i32, i32, i32, P, P, P, P], st),
            "ivfpq_build_index_ex": ([P, P, i64, i32, i32, i32, P, P, i32, P], st),
            "ivfpq_index_export": ([P, P, P, P, P, P], st),
            "ivfpq_compute_luts_ex": ([P, P, i64, P, i32, i32, P, P], st),
            "ivfpq_select_topk_ex": ([P, i64, i64, i32, P, P, P], st),
            "ivfpq_profile_begin": ([P, i32], st),
            "ivfpq_profile_end": ([P, P], st),
            "ivfpq_flat_load_bf16": ([P, i64, i32, i32, P], st),
            "ivfpq_flat_free": ([P], None),
            "ivfpq_flat_search_bf16_ex": ([P, P, i64, i32, P, P, P], st),
            "ivfpq_flat_search_bf16": ([P, P, i64, i32, P, P], st),
            "ivfpq_flat_profile_begin": ([P, i32], st),
            "ivfpq_flat_profile_end": ([P, P], st),
            "ivfpq_mx4_quantize_ex": ([P, i32, i64, i32, i64, P, P, P], st),
            "ivfpq_mx4_dequantize_ex": ([P, P, i64, i32, i32, P, P], st),
            "ivfpq_mx4_product_ex": ([P, P, i64, P, P, i64, i32, i32, P, P], st),
            "ivfpq_mx4_list_product_ex": ([P, P, i64, P, P, i32, i64, i32, P, P, i32, i64, i32, P,
                                           P], st),
            "ivfpq_route_sort_bytes": ([i64, i32, i32], ctypes.c_size_t),
            "ivfpq_route_sort_ex": ([P, i64, i32, i32, P, ctypes.c_size_t, P, P, P, P], st),
            "ivfpq_route_gather_ex": ([P, i32, i64, i32, P, P, i32, P, P], st),
            "ivfpq_route_combine_ex": ([P, i32, i64, i32, P, P, i32, P, P], st),
            "ivfpq_route_combine_grad_ex": ([P, P, i32, i64, i32, P, P, P, i32, P, P, P], st),
            "ivfpq_stream_read": ([P, ctypes.c_size_t, P, i32, P], st),
            "ivfpq_last_error": ([], ctypes.c_char_p),
            "ivfpq_status_string": ([i32], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != OK:
        raise IVFPQError(status, lib().ivfpq_last_error().decode())


def ivfpq_last_error() -> str:
    return lib().ivfpq_last_error().decode()


def ivfpq_status_string(status: int) -> str:
    return lib().ivfpq_status_string(status).decode()


def ivfpq_validate_index_file(path: str) -> int:
    """Host-only validation; returns the status code (0 = valid)."""
    return lib().ivfpq_validate_index_file(os.fsencode(path))


def _np_ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def _host_struct(index, keep: list) -> HostIndexStruct:
    get = (lambda n: index[n]) if isinstance(index, dict) else (lambda n: getattr(index, n))
    cent = np.ascontiguousarray(get("centroids"), dtype=np.float32)
    books = np.ascontiguousarray(get("codebooks"), dtype=np.float32)
    sizes = np.ascontiguousarray(get("list_sizes"), dtype=np.int64)
    codes = np.ascontiguousarray(get("codes"), dtype=np.uint8)
    ids = np.ascontiguousarray(get("ids"), dtype=np.int64)
    keep.extend([cent, books, sizes, codes, ids])
    s = HostIndexStruct()
    s.d, s.nlist = cent.shape[1], cent.shape[0]
    s.m = books.shape[0]
    s.nbits = 8
    s.ntotal = codes.shape[0]
    s.centroids, s.codebooks, s.list_sizes = _np_ptr(cent), _np_ptr(books), _np_ptr(sizes)
    s.codes, s.ids = _np_ptr(codes), _np_ptr(ids)
    return s


def ivfpq_validate_host_index(index) -> int:
    keep: list = []
    s = _host_struct(index, keep)
    return lib().ivfpq_validate_host_index(ctypes.byref(s))


class Index:
    """Owner of a device index handle."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        self.info = ivfpq_index_info(self)

    @property
    def handle(self):
        if not self._h:
            raise ValueError("index is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().ivfpq_free_index(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def search(self, queries, nprobe, k, **kw):
        return ivfpq_search_ex(self, queries, nprobe, k, **kw)


def ivfpq_load_index(path: str, device: int = 0) -> Index:
    h = ctypes.c_void_p()
    _check(lib().ivfpq_load_index(os.fsencode(path), device, ctypes.byref(h)))
    return Index(h)


def ivfpq_load_index_host(index, device: int = 0) -> Index:
    keep: list = []
    s = _host_struct(index, keep)
    h = ctypes.c_void_p()
    _check(lib().ivfpq_load_index_host(ctypes.byref(s), device, ctypes.byref(h)))
    return Index(h)


def ivfpq_build_index_ex(vectors: torch.Tensor, centroids: torch.Tensor,
                         codebooks: torch.Tensor, ids: torch.Tensor = None,
                         device: int = 0) -> Index:
    """Build an index on the device from device tensors: vectors [n, d]
    float32, centroids [nlist, d] float32, codebooks [m, 256, d/m] float32,
    ids [n] int64 (None: row numbers)."""
    x = _dev(vectors, torch.float32)
    c = _dev(centroids, torch.float32)
    b = _dev(codebooks, torch.float32)
    if x.dim() != 2 or c.dim() != 2 or b.dim() != 3 or c.shape[1] != x.shape[1] or \
            b.shape[1] != 256 or b.shape[0] * b.shape[2] != x.shape[1]:
        raise ValueError("expected vectors [n, d], centroids [nlist, d], codebooks [m, 256, d/m]")
    idp = 0
    if ids is not None:
        ids = _dev(ids, torch.int64)
        if ids.shape != (x.shape[0],):
            raise ValueError("expected ids [n]")
        idp = ids.data_ptr()
    h = ctypes.c_void_p()
    _check(lib().ivfpq_build_index_ex(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(idp),
                                      x.shape[0], x.shape[1], c.shape[0], b.shape[0],
                                      ctypes.c_void_p(c.data_ptr()), ctypes.c_void_p(b.data_ptr()),
                                      device, ctypes.byref(h)))
    return Index(h)


def ivfpq_index_export(index: Index) -> dict:
    """The index's arrays in host memory: centroids, codebooks, list_sizes,
    codes (list-major) and ids (numpy arrays, the host index layout)."""
    i = index.info
    d, nlist, m, n = i["d"], i["nlist"], i["m"], i["ntotal"]
    out = dict(centroids=np.empty((nlist, d), np.float32),
               codebooks=np.empty((m, 256, d // m), np.float32),
               list_sizes=np.empty(nlist, np.int64), codes=np.empty((n, m), np.uint8),
               ids=np.empty(n, np.int64))
    _check(lib().ivfpq_index_export(index.handle, *(_np_ptr(out[k]) for k in
                                                    ("centroids", "codebooks", "list_sizes",
                                                     "codes", "ids"))))
    return out


def ivfpq_free_index(index: Index) -> None:
    index.close()


def ivfpq_index_info(index: Index) -> dict:
    i = Info()
    _check(lib().ivfpq_index_info(index.handle, ctypes.byref(i)))
    return {f: getattr(i, f) for f, _ in Info._fields_ if f != "reserved"}


def ivfpq_search(index: Index, queries: np.ndarray, nprobe: int, k: int):
    """Blocking search on host arrays; returns (distances float32, ids int64)."""
    q = np.ascontiguousarray(queries, dtype=np.float32)
    nq = q.shape[0]
    d = np.empty((nq, k), dtype=np.float32)
    i = np.empty((nq, k), dtype=np.int64)
    _check(lib().ivfpq_search(index.handle, _np_ptr(q), nq, nprobe, k, _np_ptr(d), _np_ptr(i)))
    return d, i


def _dev(t: torch.Tensor, dtype) -> torch.Tensor:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"expected a contiguous {dtype} device tensor")
    return t


def _stream_ptr(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# The current stream's handle itself, without the Stream object that
# torch.cuda.current_stream makes (2.8 of 10 microseconds of a small call); not
# part of torch's public interface, so done without where it is missing.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _raw_stream(stream) -> int:
    if stream is None and _current_raw_stream and _current_device:
        return _current_raw_stream(_current_device())
    return _stream_ptr(stream).value or 0


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory that a call on `stream` (None: the current one) writes.  For a given
    stream it comes from that stream's pool, as what was freed on the current one
    may still be in use there; and as the caller goes on with the result on the
    current stream, it is not given out again before that stream is past its end."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def ivfpq_search_ex(index: Index, queries: torch.Tensor, nprobe: int, k: int, lut: str = "f32",
                    mode: int = MODE_NORMAL, chunk_len: int = 0, return_probes: bool = False,
                    out=None, stream=None, metric: str = "l2", noalloc: bool = False):
    """Asynchronous device search on the current (or given) torch stream.
    metric "l2" (squared L2, ascending) or "ip" (inner product, descending).
    noalloc: call ivfpq_search_noalloc_ex (workspace in the library's fixed
    device scratch; pass `out` too so that nothing is allocated here either).

    Returns (distances [nq,k] float32, ids [nq,k] int64[, probes [nq,nprobe] int32])."""
    if metric not in ("l2", "ip"):
        raise ValueError("metric must be 'l2' or 'ip'")
    q = _dev(queries, torch.float32)
    nq = q.shape[0]
    if out is None:
        dist = _empty((nq, k), torch.float32, q.device, stream)
        ids = _empty((nq, k), torch.int64, q.device, stream)
        probes = _empty((nq, nprobe), torch.int32, q.device, stream) \
            if return_probes else None
    else:
        dist, ids, probes = out
    p = SearchParams(nprobe, k, LUT_F16 if lut == "f16" else LUT_F32, mode, chunk_len,
                     METRIC_IP if metric == "ip" else METRIC_L2)
    fn = lib().ivfpq_search_noalloc_ex if noalloc else lib().ivfpq_search_ex
    _check(fn(index.handle, ctypes.byref(p), ctypes.c_void_p(q.data_ptr()),
              nq, ctypes.c_void_p(dist.data_ptr()),
              ctypes.c_void_p(ids.data_ptr()),
              ctypes.c_void_p(probes.data_ptr() if probes is not None else 0),
              _stream_ptr(stream)))
    return (dist, ids, probes) if return_probes else (dist, ids)


def ivfpq_coarse_ex(index: Index, queries: torch.Tensor, nprobe: int, stream=None):
    q = _dev(queries, torch.float32)
    nq = q.shape[0]
    probes = _empty((nq, nprobe), torch.int32, q.device, stream)
    dist = _empty((nq, nprobe), torch.float32, q.device, stream)
    _check(lib().ivfpq_coarse_ex(index.handle, ctypes.c_void_p(q.data_ptr()), nq, nprobe,
                                 ctypes.c_void_p(probes.data_ptr()),
                                 ctypes.c_void_p(dist.data_ptr()), _stream_ptr(stream)))
    return probes, dist


def ivfpq_assign_encode_ex(index: Index, vectors: torch.Tensor, stream=None):
    """List assignment and PQ codes of database vectors with the index's
    centroids and codebooks: (lists [n] int32, codes [n, m] uint8)."""
    x = _dev(vectors, torch.float32)
    if x.dim() != 2 or x.shape[1] != index.info["d"]:
        raise ValueError(f"expected vectors of shape [n, {index.info['d']}]")
    n = x.shape[0]
    lists = _empty((n,), torch.int32, x.device, stream)
    codes = _empty((n, index.info["m"]), torch.uint8, x.device, stream)
    _check(lib().ivfpq_assign_encode_ex(index.handle, ctypes.c_void_p(x.data_ptr()), n,
                                        ctypes.c_void_p(lists.data_ptr()),
                                        ctypes.c_void_p(codes.data_ptr()), _stream_ptr(stream)))
    return lists, codes


def ivfpq_kmeans_ex(vectors: torch.Tensor, centers: torch.Tensor, iters: int, stream=None):
    """Lloyd's algorithm on the device: `centers` ([k, d] float32, updated in
    place) from `vectors` ([n, d] float32).  Returns the last round's
    (assignment [n] int32, counts [k] int32)."""
    x = _dev(vectors, torch.float32)
    c = _dev(centers, torch.float32)
    if x.dim() != 2 or c.dim() != 2 or x.shape[1] != c.shape[1]:
        raise ValueError("expected vectors [n, d] and centers [k, d]")
    n, (k, d) = x.shape[0], c.shape
    assign = _empty((n,), torch.int32, x.device, stream)
    counts = _empty((k,), torch.int32, x.device, stream)
    with torch.cuda.stream(stream):  # None: the current one
        assign.fill_(-1)
        counts.zero_()
    _check(lib().ivfpq_kmeans_ex(ctypes.c_void_p(x.data_ptr()), n, d, k, iters,
                                 ctypes.c_void_p(c.data_ptr()), ctypes.c_void_p(assign.data_ptr()),
                                 ctypes.c_void_p(counts.data_ptr()), _stream_ptr(stream)))
    return assign, counts


def ivfpq_compute_luts_ex(index: Index, queries: torch.Tensor, probes: torch.Tensor,
                          lut: str = "f32", stream=None):
    q = _dev(queries, torch.float32)
    pr = _dev(probes, torch.int32)
    nq, nprobe = pr.shape
    m = index.info["m"]
    out = _empty((nq, nprobe, m, 256), torch.float32, q.device, stream)
    _check(lib().ivfpq_compute_luts_ex(index.handle, ctypes.c_void_p(q.data_ptr()), nq,
                                       ctypes.c_void_p(pr.data_ptr()), nprobe,
                                       LUT_F16 if lut == "f16" else LUT_F32,
                                       ctypes.c_void_p(out.data_ptr()), _stream_ptr(stream)))
    return out


def ivfpq_select_topk_ex(keys: torch.Tensor, k: int, stream=None):
    """Row-wise k smallest of a [rows, n] float32 device tensor:
    (values [rows,k] float32, column numbers [rows,k] int32)."""
    x = _dev(keys, torch.float32)
    rows, n = x.shape
    d = _empty((rows, k), torch.float32, x.device, stream)
    p = _empty((rows, k), torch.int32, x.device, stream)
    _check(lib().ivfpq_select_topk_ex(ctypes.c_void_p(x.data_ptr()), rows, n, k,
                                      ctypes.c_void_p(d.data_ptr()), ctypes.c_void_p(p.data_ptr()),
                                      _stream_ptr(stream)))
    return d, p


def ivfpq_stream_read(data: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Enqueue the reference streaming read of a contiguous device tensor
    (measurement support); sink: an int32 device tensor of scratch words."""
    if not data.is_cuda or not data.is_contiguous():
        raise ValueError("expected a contiguous device tensor")
    s = _dev(sink, torch.int32)
    _check(lib().ivfpq_stream_read(ctypes.c_void_p(data.data_ptr()),
                                   data.numel() * data.element_size(),
                                   ctypes.c_void_p(s.data_ptr()), s.numel(), _stream_ptr(stream)))


def ivfpq_profile_begin(index: Index, max_calls: int) -> None:
    _check(lib().ivfpq_profile_begin(index.handle, max_calls))


def ivfpq_profile_end(index: Index) -> dict:
    t = Timings()
    _check(lib().ivfpq_profile_end(index.handle, ctypes.byref(t)))
    return {f: getattr(t, f) for f, _ in Timings._fields_ if f != "reserved"}


# ---------------------------------------------------------------------------
# 4-bit rows, their products, and vectors sorted by list
#
# All run on the current stream or the given one, which the caller orders after
# what writes the inputs; what is allocated here is that stream's.
# ---------------------------------------------------------------------------

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _row_type(dtype) -> int:
    if dtype not in TYPES:
        raise ValueError("expected float32, bfloat16 or float16")
    return TYPES[dtype]


def _rows(t: torch.Tensor):
    """The type code and shape of checked rows [n, d]."""
    kind = TYPES.get(t.dtype)
    if kind is None or not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected contiguous device rows of float32, bfloat16 or float16")
    shape = t.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("expected rows [n, d] with d >= 1")
    return kind, shape


def _ptr(t):
    return None if t is None else t.data_ptr()


def _out(out, shape, dtype, device, stream) -> torch.Tensor:
    if out is None:
        return _empty(shape, dtype, device, stream)
    if out.shape != shape:
        raise ValueError(f"expected an output of shape {shape}")
    return _dev(out, dtype)


def _mx4(pair, dims: int):
    """Checked (codes, scales, shape of scales) of 4-bit rows."""
    codes, scales = pair
    _dev(codes, torch.uint8)
    _dev(scales, torch.uint8)
    c, s = codes.shape, scales.shape
    if len(c) != dims or len(s) != dims or c[0] != s[0] or c[dims - 2] != s[dims - 2] or \
            c[dims - 1] != 16 * s[dims - 1] or s[dims - 1] < 1:
        raise ValueError("expected 4-bit rows: codes [..., n, 16 kb] and scales [..., n, kb]")
    return codes, scales, s


def ivfpq_mx4_quantize_ex(x: torch.Tensor, out=None, stream=None):
    """Rows [n, d] (float32, bfloat16 or float16; a view with contiguous rows
    will do) to microscaled 4-bit rows: (codes [n, 16 kb] uint8, scales [n, kb]
    uint8), kb = ceil(d / 32)."""
    kind = _row_type(x.dtype)
    shape, strides = x.shape, x.stride()
    if not x.is_cuda or len(shape) != 2 or shape[1] < 1 or \
            (shape[1] > 1 and strides[1] != 1) or strides[0] < 0:
        raise ValueError("expected device rows [n, d], d >= 1, each row contiguous")
    n, d = shape
    kb = (d + 31) // 32
    codes, scales = (None, None) if out is None else out
    codes = _out(codes, (n, 16 * kb), torch.uint8, x.device, stream)
    scales = _out(scales, (n, kb), torch.uint8, x.device, stream)
    _check(lib().ivfpq_mx4_quantize_ex(x.data_ptr(), kind, n, d, strides[0], codes.data_ptr(),
                                       scales.data_ptr(), _raw_stream(stream)))
    return codes, scales


def ivfpq_mx4_dequantize_ex(codes: torch.Tensor, scales: torch.Tensor, d: int,
                            dtype=torch.float32, out=None, stream=None) -> torch.Tensor:
    """The values [n, d] that 4-bit rows stand for."""
    kind = _row_type(dtype)
    codes, scales, (n, kb) = _mx4((codes, scales), 2)
    if d < 1 or (d + 31) // 32 != kb:
        raise ValueError("d does not fit the rows' blocks")
    out = _out(out, (n, d), dtype, codes.device, stream)
    _check(lib().ivfpq_mx4_dequantize_ex(codes.data_ptr(), scales.data_ptr(), n, d, kind,
                                         out.data_ptr(), _raw_stream(stream)))
    return out


def ivfpq_mx4_product_ex(a, b, dtype=torch.float32, out=None, stream=None) -> torch.Tensor:
    """A B^T of 4-bit rows a = (codes, scales) of [m, d] and b of [n, d]:
    [m, n] of dtype, summed in float32."""
    kind = _row_type(dtype)
    (ac, as_, (m, kb)), (bc, bs, (n, kb_b)) = _mx4(a, 2), _mx4(b, 2)
    if kb != kb_b:
        raise ValueError("the operands' rows have different lengths")
    out = _out(out, (m, n), dtype, ac.device, stream)
    _check(lib().ivfpq_mx4_product_ex(ac.data_ptr(), as_.data_ptr(), m, bc.data_ptr(),
                                      bs.data_ptr(), n, 32 * kb, kind, out.data_ptr(),
                                      _raw_stream(stream)))
    return out


def ivfpq_mx4_list_product_ex(a, b, offsets: torch.Tensor, order: torch.Tensor = None, k: int = 1,
                              dtype=torch.float32, out=None, stream=None) -> torch.Tensor:
    """Rows sorted by list times their list's matrix: b = (codes [nlist, n,
    16 kb], scales [nlist, n, kb]), offsets [nlist + 1] int32.  With order
    ([rows] int32, of ivfpq_route_sort_ex) output row p takes row order[p] // k
    of a, without it row p.  Returns [rows, n] of dtype, zero before offsets[0]
    and past offsets[nlist]."""
    kind = _row_type(dtype)
    (ac, as_, (arows, kb)), (bc, bs, (nlist, n, kb_b)) = _mx4(a, 2), _mx4(b, 3)
    offsets = _dev(offsets, torch.int32)
    if kb != kb_b:
        raise ValueError("the operands' rows have different lengths")
    if offsets.shape != (nlist + 1,):
        raise ValueError("expected offsets [nlist + 1]")
    rows = arows
    if order is not None:
        shape = _slots(order, "order")
        if len(shape) != 1:
            raise ValueError("expected order [rows]")
        rows = shape[0]
    out = _out(out, (rows, n), dtype, ac.device, stream)
    _check(lib().ivfpq_mx4_list_product_ex(ac.data_ptr(), as_.data_ptr(), arows, bc.data_ptr(),
                                           bs.data_ptr(), nlist, n, 32 * kb, offsets.data_ptr(),
                                           _ptr(order), k, rows, kind, out.data_ptr(),
                                           _raw_stream(stream)))
    return out


def ivfpq_route_sort_bytes(nvec: int, k: int, nlist: int) -> int:
    return lib().ivfpq_route_sort_bytes(nvec, k, nlist)


def ivfpq_route_sort_ex(lists: torch.Tensor, nlist: int, out=None, workspace=None, stream=None):
    """(vector, list) pairs sorted by list, stable: lists [nvec, k] int32 (outside
    [0, nlist): masked) -> (offsets [nlist + 1], order [nvec k], pos [nvec, k]),
    all int32.  workspace: uint8 device tensor of
    ivfpq_route_sort_bytes (None: allocated here where one is needed)."""
    shape = _slots(lists, "lists")
    if len(shape) != 2 or shape[1] < 1 or nlist < 1:
        raise ValueError("expected lists [nvec, k], k >= 1, and nlist >= 1")
    nvec, k = shape
    offsets, order, pos = (None, None, None) if out is None else out
    device = lists.device
    offsets = _out(offsets, (nlist + 1,), torch.int32, device, stream)
    order = _out(order, (nvec * k,), torch.int32, device, stream)
    pos = _out(pos, shape, torch.int32, device, stream)
    need = ivfpq_route_sort_bytes(nvec, k, nlist)
    if workspace is not None:
        _dev(workspace, torch.uint8)
    elif need:
        workspace = _empty((need,), torch.uint8, device, stream)
    _check(lib().ivfpq_route_sort_ex(lists.data_ptr(), nvec, k, nlist, _ptr(workspace),
                                     0 if workspace is None else workspace.numel(),
                                     offsets.data_ptr(), order.data_ptr(), pos.data_ptr(),
                                     _raw_stream(stream)))
    return offsets, order, pos


def _slots(t: torch.Tensor, what: str):
    """Shape of checked slot numbers."""
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"expected {what} as a contiguous int32 device tensor")
    return t.shape


def _slot_weights(weights, nvec: int, k: int):
    """Pointer of checked weights, None without them."""
    if weights is None:
        return None
    if _dev(weights, torch.float32).shape != (nvec, k):
        raise ValueError("expected weights [nvec, k]")
    return weights.data_ptr()


def ivfpq_route_gather_ex(x: torch.Tensor, order: torch.Tensor, k: int,
                          weights: torch.Tensor = None, out=None, stream=None) -> torch.Tensor:
    """Row p = x[order[p] // k] (times weights[order[p]]), zero where order is -1:
    [nvec k, d] from x [nvec, d].  For the rows' gradient g, the gradient of x is
    ivfpq_route_combine_ex(g, pos, weights), that of the weights the second result
    of ivfpq_route_combine_grad_ex(x, g, order, pos, weights)."""
    kind, (nvec, d) = _rows(x)
    if k < 1 or _slots(order, "order") != (nvec * k,):
        raise ValueError("expected order [nvec k], k >= 1")
    w = _slot_weights(weights, nvec, k)
    out = _out(out, (nvec * k, d), x.dtype, x.device, stream)
    _check(lib().ivfpq_route_gather_ex(x.data_ptr(), kind, nvec, d, order.data_ptr(), w, k,
                                       out.data_ptr(), _raw_stream(stream)))
    return out


def _routed(rows: torch.Tensor, pos: torch.Tensor):
    kind, (n, d) = _rows(rows)
    shape = _slots(pos, "pos")
    if len(shape) != 2 or shape[1] < 1 or n != shape[0] * shape[1]:
        raise ValueError("expected rows [nvec k, d] and pos [nvec, k], k >= 1")
    return kind, d, *shape


def ivfpq_route_combine_ex(rows: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor = None,
                           out=None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] rows[pos[t, j]] (weights 1 without them), masked
    slots (pos -1) adding nothing: [nvec, d] from rows [nvec k, d]."""
    kind, d, nvec, k = _routed(rows, pos)
    w = _slot_weights(weights, nvec, k)
    out = _out(out, (nvec, d), rows.dtype, rows.device, stream)
    _check(lib().ivfpq_route_combine_ex(rows.data_ptr(), kind, nvec, d, pos.data_ptr(), w, k,
                                        out.data_ptr(), _raw_stream(stream)))
    return out


def ivfpq_route_combine_grad_ex(grad: torch.Tensor, rows: torch.Tensor, order: torch.Tensor,
                                pos: torch.Tensor, weights: torch.Tensor, out=None, stream=None):
    """Gradients of ivfpq_route_combine_ex(rows, pos, weights) for the output
    gradient grad [nvec, d]: (of rows [nvec k, d], of weights [nvec, k] float32)."""
    kind, d, nvec, k = _routed(rows, pos)
    if _rows(grad) != (kind, (nvec, d)):
        raise ValueError("expected grad [nvec, d] of the rows' type")
    if _slots(order, "order") != (nvec * k,):
        raise ValueError("expected order [nvec k]")
    w = _slot_weights(weights, nvec, k)
    if w is None:
        raise ValueError("expected weights [nvec, k]")
    d_rows, d_weights = (None, None) if out is None else out
    d_rows = _out(d_rows, (nvec * k, d), rows.dtype, rows.device, stream)
    d_weights = _out(d_weights, (nvec, k), torch.float32, rows.device, stream)
    _check(lib().ivfpq_route_combine_grad_ex(grad.data_ptr(), rows.data_ptr(), kind, nvec, d,
                                             order.data_ptr(), pos.data_ptr(), w, k,
                                             d_rows.data_ptr(), d_weights.data_ptr(),
                                             _raw_stream(stream)))
    return d_rows, d_weights


# ---------------------------------------------------------------------------
# exact search over a flat bfloat16 database
# ---------------------------------------------------------------------------

class FlatIndex:
    """Owner of a device flat-database handle."""

    def __init__(self, handle: ctypes.c_void_p, n: int, d: int):
        self._h = handle
        self.n, self.d = n, d

    @property
    def handle(self):
        if not self._h:
            raise ValueError("flat index is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().ivfpq_flat_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ivfpq_flat_load_bf16(vectors: np.ndarray, device: int = 0) -> FlatIndex:
    """Upload [n, d] bfloat16 bit patterns (uint16, host)."""
    v = np.ascontiguousarray(vectors, dtype=np.uint16)
    h = ctypes.c_void_p()
    _check(lib().ivfpq_flat_load_bf16(_np_ptr(v), v.shape[0], v.shape[1], device,
                                      ctypes.byref(h)))
    return FlatIndex(h, v.shape[0], v.shape[1])


def ivfpq_flat_free(flat: FlatIndex) -> None:
    flat.close()


def _bf16_bits(t: torch.Tensor) -> torch.Tensor:
    if t.dtype == torch.bfloat16:
        t = t.view(torch.int16)
    return _dev(t, torch.int16)


def ivfpq_flat_search_bf16_ex(flat: FlatIndex, queries: torch.Tensor, k: int, out=None,
                              stream=None):
    """Asynchronous exact search; queries: [nq, d] device tensor of bfloat16 (or
    its bit patterns as int16).  Returns (distances [nq,k] float32, ids [nq,k]
    int64 row numbers)."""
    q = _bf16_bits(queries)
    nq = q.shape[0]
    if out is None:
        dist = _empty((nq, k), torch.float32, q.device, stream)
        ids = _empty((nq, k), torch.int64, q.device, stream)
    else:
        dist, ids = out
    _check(lib().ivfpq_flat_search_bf16_ex(flat.handle, ctypes.c_void_p(q.data_ptr()), nq, k,
                                           ctypes.c_void_p(dist.data_ptr()),
                                           ctypes.c_void_p(ids.data_ptr()), _stream_ptr(stream)))
    return dist, ids


def ivfpq_flat_search_bf16(flat: FlatIndex, queries: np.ndarray, k: int):
    """Blocking exact search on host bfloat16 bit patterns (uint16 [nq, d])."""
    q = np.ascontiguousarray(queries, dtype=np.uint16)
    nq = q.shape[0]
    d = np.empty((nq, k), dtype=np.float32)
    i = np.empty((nq, k), dtype=np.int64)
    _check(lib().ivfpq_flat_search_bf16(flat.handle, _np_ptr(q), nq, k, _np_ptr(d), _np_ptr(i)))
    return d, i


def ivfpq_flat_profile_begin(flat: FlatIndex, max_calls: int) -> None:
    _check(lib().ivfpq_flat_profile_begin(flat.handle, max_calls))


def ivfpq_flat_profile_end(flat: FlatIndex) -> dict:
    t = FlatTimings()
    _check(lib().ivfpq_flat_profile_end(flat.handle, ctypes.byref(t)))
    return {f: getattr(t, f) for f, _ in FlatTimings._fields_ if f != "reserved"}
