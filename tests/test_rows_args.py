"""Refusals of the 4-bit row and routing calls: checked on the host before any
device work, so they need no GPU."""
import ctypes

import pytest
import torch

import approximate_nearest_neighbour_amd as A
from approximate_nearest_neighbour_amd import binding as B

BUF = (ctypes.c_uint8 * 4096)()
P = (ctypes.addressof(BUF) + 15) // 16 * 16   # never dereferenced: every call is refused


def refused(name, *args):
    L = B.lib()
    assert getattr(L, name)(*args) == B.E_INVALID_ARG, (name, args)
    assert L.ivfpq_last_error() != b""


GOOD = {
    # type codes: 0 float32, 1 bfloat16, 2 binary16
    "ivfpq_mx4_quantize_ex": [P, 0, 4, 64, 64, P, P, None],
    "ivfpq_mx4_dequantize_ex": [P, P, 4, 64, 0, P, None],
    "ivfpq_mx4_product_ex": [P, P, 4, P, P, 4, 64, 0, P, None],
    "ivfpq_mx4_list_product_ex": [P, P, 4, P, P, 2, 4, 64, P, P, 2, 8, 0, P, None],
    "ivfpq_route_sort_ex": [P, 20000, 2, 8, P, 1 << 20, P, P, P, None],
    "ivfpq_route_gather_ex": [P, 0, 4, 8, P, P, 2, P, None],
    "ivfpq_route_combine_ex": [P, 0, 4, 8, P, P, 2, P, None],
    "ivfpq_route_combine_grad_ex": [P, P, 0, 4, 8, P, P, P, 2, P, P, None],
}

BIG = 1 << 31
BAD = [
    ("ivfpq_mx4_quantize_ex", {0: None}), ("ivfpq_mx4_quantize_ex", {5: None}),
    ("ivfpq_mx4_quantize_ex", {6: None}), ("ivfpq_mx4_quantize_ex", {1: 3}),
    ("ivfpq_mx4_quantize_ex", {1: -1}), ("ivfpq_mx4_quantize_ex", {2: -1}),
    ("ivfpq_mx4_quantize_ex", {2: BIG}), ("ivfpq_mx4_quantize_ex", {3: 0}),
    ("ivfpq_mx4_quantize_ex", {3: (1 << 20) + 1}), ("ivfpq_mx4_quantize_ex", {4: -1}),
    ("ivfpq_mx4_quantize_ex", {0: P + 2}), ("ivfpq_mx4_quantize_ex", {0: P + 1, 1: 1}),
    ("ivfpq_mx4_quantize_ex", {5: P + 8}),
    ("ivfpq_mx4_dequantize_ex", {0: None}), ("ivfpq_mx4_dequantize_ex", {1: None}),
    ("ivfpq_mx4_dequantize_ex", {5: None}), ("ivfpq_mx4_dequantize_ex", {4: 9}),
    ("ivfpq_mx4_dequantize_ex", {3: 0}), ("ivfpq_mx4_dequantize_ex", {2: -5}),
    ("ivfpq_mx4_dequantize_ex", {0: P + 4}), ("ivfpq_mx4_dequantize_ex", {5: P + 2}),
    ("ivfpq_mx4_product_ex", {0: None}), ("ivfpq_mx4_product_ex", {1: None}),
    ("ivfpq_mx4_product_ex", {3: None}), ("ivfpq_mx4_product_ex", {4: None}),
    ("ivfpq_mx4_product_ex", {8: None}), ("ivfpq_mx4_product_ex", {2: -1}),
    ("ivfpq_mx4_product_ex", {5: BIG}), ("ivfpq_mx4_product_ex", {6: 0}),
    ("ivfpq_mx4_product_ex", {7: 4}), ("ivfpq_mx4_product_ex", {0: P + 1}),
    ("ivfpq_mx4_product_ex", {3: P + 8}), ("ivfpq_mx4_product_ex", {8: P + 1}),
    ("ivfpq_mx4_product_ex", {2: BIG - 1, 5: BIG - 16}),
    ("ivfpq_mx4_list_product_ex", {8: None}), ("ivfpq_mx4_list_product_ex", {5: 0}),
    ("ivfpq_mx4_list_product_ex", {5: (1 << 16) + 1}), ("ivfpq_mx4_list_product_ex", {10: 0}),
    ("ivfpq_mx4_list_product_ex", {11: -1}), ("ivfpq_mx4_list_product_ex", {2: 0}),
    ("ivfpq_mx4_list_product_ex", {9: None}),  # 8 rows of a first operand of 4
    ("ivfpq_mx4_list_product_ex", {12: 7}), ("ivfpq_mx4_list_product_ex", {13: None}),
    ("ivfpq_mx4_list_product_ex", {3: P + 4}), ("ivfpq_mx4_list_product_ex", {7: -3}),
    ("ivfpq_mx4_list_product_ex", {2: BIG - 1, 6: 1 << 20, 11: 1 << 16}),
    ("ivfpq_route_sort_ex", {0: None}), ("ivfpq_route_sort_ex", {1: -1}),
    ("ivfpq_route_sort_ex", {1: 1 << 30}), ("ivfpq_route_sort_ex", {2: 0}),
    ("ivfpq_route_sort_ex", {3: 0}), ("ivfpq_route_sort_ex", {3: 1 << 22}),
    ("ivfpq_route_sort_ex", {4: None}), ("ivfpq_route_sort_ex", {4: P + 4}),
    ("ivfpq_route_sort_ex", {5: 8}), ("ivfpq_route_sort_ex", {6: None}),
    ("ivfpq_route_sort_ex", {7: None}), ("ivfpq_route_sort_ex", {8: None}),
    ("ivfpq_route_gather_ex", {0: None}), ("ivfpq_route_gather_ex", {4: None}),
    ("ivfpq_route_gather_ex", {7: None}), ("ivfpq_route_gather_ex", {1: 5}),
    ("ivfpq_route_gather_ex", {6: 0}), ("ivfpq_route_gather_ex", {3: 0}),
    ("ivfpq_route_gather_ex", {0: P + 1}), ("ivfpq_route_gather_ex", {2: 1 << 30}),
    ("ivfpq_route_combine_ex", {0: None}), ("ivfpq_route_combine_ex", {4: None}),
    ("ivfpq_route_combine_ex", {7: None}), ("ivfpq_route_combine_ex", {7: P + 2}),
    ("ivfpq_route_combine_ex", {2: -1}), ("ivfpq_route_combine_ex", {3: 1 << 21}),
    ("ivfpq_route_combine_grad_ex", {0: None}), ("ivfpq_route_combine_grad_ex", {1: None}),
    ("ivfpq_route_combine_grad_ex", {5: None}), ("ivfpq_route_combine_grad_ex", {6: None}),
    ("ivfpq_route_combine_grad_ex", {7: None}), ("ivfpq_route_combine_grad_ex", {9: None}),
    ("ivfpq_route_combine_grad_ex", {10: None}), ("ivfpq_route_combine_grad_ex", {2: -2}),
    ("ivfpq_route_combine_grad_ex", {9: P + 1}),
]


@pytest.mark.parametrize("name,change", BAD)
def test_bad_arguments_are_refused(name, change):
    args = list(GOOD[name])
    for i, v in change.items():
        args[i] = v
    refused(name, *args)


@pytest.mark.parametrize("name,zero", [
    ("ivfpq_mx4_quantize_ex", 2), ("ivfpq_mx4_dequantize_ex", 2), ("ivfpq_mx4_product_ex", 2),
    ("ivfpq_mx4_product_ex", 5), ("ivfpq_mx4_list_product_ex", 11),
    ("ivfpq_mx4_list_product_ex", 6), ("ivfpq_route_gather_ex", 2), ("ivfpq_route_combine_ex", 2),
    ("ivfpq_route_combine_grad_ex", 3)])
def test_nothing_to_do_is_ok(name, zero):
    args = list(GOOD[name])
    args[zero] = 0
    assert getattr(B.lib(), name)(*args) == B.OK


def test_sort_workspace_size():
    assert A.ivfpq_route_sort_bytes(20000, 2, 8) > 0
    assert A.ivfpq_route_sort_bytes(100, 4, 64) == 0   # a small sort needs none
    for bad in ((-1, 4, 64), (100, 0, 64), (1 << 30, 4, 64), (100, 4, 0), (100, 4, 1 << 22)):
        assert A.ivfpq_route_sort_bytes(*bad) == 0


def test_host_tensors_are_refused():
    x = torch.zeros((4, 64))
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    flat = ids.reshape(-1)
    for call in (lambda: A.ivfpq_mx4_quantize_ex(x),
                 lambda: A.ivfpq_mx4_quantize_ex(x.double()),
                 lambda: A.ivfpq_mx4_dequantize_ex(codes, scales, 64),
                 lambda: A.ivfpq_mx4_product_ex((codes, scales), (codes, scales)),
                 lambda: A.ivfpq_mx4_product_ex((codes, scales), (codes, scales),
                                                dtype=torch.int8),
                 lambda: A.ivfpq_mx4_list_product_ex((codes, scales), (codes[None], scales[None]),
                                                     flat[:2]),
                 lambda: A.ivfpq_route_sort_ex(ids, 4),
                 lambda: A.ivfpq_route_gather_ex(x, flat, 2),
                 lambda: A.ivfpq_route_combine_ex(x, ids),
                 lambda: A.ivfpq_route_combine_grad_ex(x, x, flat, ids, x)):
        with pytest.raises(ValueError):
            call()
