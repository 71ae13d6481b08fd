"""Refusals of the products per list, the adapters and the table rows: checked on the
host before any device work, so they need no GPU."""
import ctypes

import pytest
import torch

import approximate_nearest_neighbour_amd as A
from approximate_nearest_neighbour_amd import binding as B

BUF = (ctypes.c_uint8 * 4096)()
P = (ctypes.addressof(BUF) + 15) // 16 * 16   # never dereferenced: every call is refused
BIG = 1 << 31
WS = 1 << 40

GOOD = {
    # type codes: 0 float32, 1 bfloat16, 2 binary16
    "ivfpq_list_product_ex": [P, 1, 8, 64, P, 0, 3, 32, P, P, 2, 16, P, None],
    "ivfpq_list_product_grad_ex": [P, P, 1, 8, 64, 3, 32, P, P, 2, 16, 0, P, WS, P, None],
    "ivfpq_adapter_product_ex": [P, 1, 8, 64, P, 32, P, P, 3, 16, P, P, P, P, P, WS, P, None],
    "ivfpq_table_lookup_ex": [P, 1, 100, 64, P, 8, 1.0, P, None],
    "ivfpq_table_grad_ex": [P, 1, 800, 64, P, P, 1, 100, 1.0, 0, P, WS, P, None],
}

BAD = [
    *[("ivfpq_list_product_ex", {i: None}) for i in (0, 4, 8, 12)],
    *[("ivfpq_list_product_ex", {i: P + 1}) for i in (0, 4, 12)],
    *[("ivfpq_list_product_ex", {1: v}) for v in (-1, 3)],
    *[("ivfpq_list_product_ex", {2: v}) for v in (-1, BIG, 0)],
    *[("ivfpq_list_product_ex", {3: v}) for v in (0, -4, (1 << 20) + 1)],
    *[("ivfpq_list_product_ex", {6: v}) for v in (0, -1, (1 << 16) + 1)],
    *[("ivfpq_list_product_ex", {7: v}) for v in (0, (1 << 20) + 1)],
    ("ivfpq_list_product_ex", {9: None}),          # 16 rows of 8
    ("ivfpq_list_product_ex", {10: 0}), ("ivfpq_list_product_ex", {11: -1}),
    ("ivfpq_list_product_ex", {11: BIG}), ("ivfpq_list_product_ex", {1: 0, 0: P + 2}),
    *[("ivfpq_list_product_grad_ex", {i: None}) for i in (0, 1, 7, 14)],
    *[("ivfpq_list_product_grad_ex", {i: P + 1}) for i in (0, 1, 14)],
    ("ivfpq_list_product_grad_ex", {14: P + 2}),   # float32 output
    *[("ivfpq_list_product_grad_ex", {11: v}) for v in (2, 3, -1)],
    ("ivfpq_list_product_grad_ex", {2: 0, 11: 1}), ("ivfpq_list_product_grad_ex", {2: 7}),
    *[("ivfpq_list_product_grad_ex", {3: v}) for v in (-1, 0, BIG)],
    ("ivfpq_list_product_grad_ex", {4: 0}), ("ivfpq_list_product_grad_ex", {5: 0}),
    ("ivfpq_list_product_grad_ex", {5: 1 << 17}), ("ivfpq_list_product_grad_ex", {6: 1 << 21}),
    ("ivfpq_list_product_grad_ex", {8: None}), ("ivfpq_list_product_grad_ex", {9: 0}),
    ("ivfpq_list_product_grad_ex", {10: BIG}), ("ivfpq_list_product_grad_ex", {12: P + 8}),
    *[("ivfpq_adapter_product_ex", {i: None}) for i in (0, 4, 6, 7, 11, 12, 13, 14, 16)],
    *[("ivfpq_adapter_product_ex", {i: P + 1}) for i in (0, 4, 6, 7, 16)],
    ("ivfpq_adapter_product_ex", {14: P + 4}), ("ivfpq_adapter_product_ex", {15: 8}),
    ("ivfpq_adapter_product_ex", {1: 9}), ("ivfpq_adapter_product_ex", {2: -1}),
    ("ivfpq_adapter_product_ex", {2: BIG}), ("ivfpq_adapter_product_ex", {3: 0}),
    ("ivfpq_adapter_product_ex", {5: 0}), ("ivfpq_adapter_product_ex", {8: 0}),
    ("ivfpq_adapter_product_ex", {9: 0}), ("ivfpq_adapter_product_ex", {9: (1 << 12) + 1}),
    *[("ivfpq_table_lookup_ex", {i: None}) for i in (0, 4, 7)],
    *[("ivfpq_table_lookup_ex", {i: P + 1}) for i in (0, 7)],
    ("ivfpq_table_lookup_ex", {1: 4}), ("ivfpq_table_lookup_ex", {2: -1}),
    ("ivfpq_table_lookup_ex", {2: BIG}), ("ivfpq_table_lookup_ex", {3: 0}),
    ("ivfpq_table_lookup_ex", {3: 1 << 21}), ("ivfpq_table_lookup_ex", {5: BIG}),
    *[("ivfpq_table_grad_ex", {i: None}) for i in (0, 4, 5, 10, 12)],
    *[("ivfpq_table_grad_ex", {i: P + 1}) for i in (0, 12)],
    ("ivfpq_table_grad_ex", {10: P + 8}), ("ivfpq_table_grad_ex", {11: 8}),
    ("ivfpq_table_grad_ex", {1: 3}), ("ivfpq_table_grad_ex", {9: 2}),
    ("ivfpq_table_grad_ex", {2: -1}), ("ivfpq_table_grad_ex", {2: 1 << 30, 6: 2}),
    ("ivfpq_table_grad_ex", {3: 0}), ("ivfpq_table_grad_ex", {6: 0}),
    ("ivfpq_table_grad_ex", {7: 0}), ("ivfpq_table_grad_ex", {7: 1 << 22}),
]


@pytest.mark.parametrize("name,change", BAD)
def test_bad_arguments_are_refused(name, change):
    args = list(GOOD[name])
    for i, v in change.items():
        args[i] = v
    L = B.lib()
    assert getattr(L, name)(*args) == B.E_INVALID_ARG, (name, change)
    assert L.ivfpq_last_error() != b""


@pytest.mark.parametrize("name,zero", [
    ("ivfpq_list_product_ex", 11), ("ivfpq_adapter_product_ex", 2), ("ivfpq_table_lookup_ex", 5)])
def test_nothing_to_do_is_ok(name, zero):
    args = list(GOOD[name])
    args[zero] = 0
    assert getattr(B.lib(), name)(*args) == B.OK


def test_workspace_sizes():
    assert A.ivfpq_adapter_product_bytes(8, 16) >= 8 * (16 * 4 + 4)
    for bad in ((-1, 16), (BIG, 16), (8, 0), (8, 1 << 13)):
        assert A.ivfpq_adapter_product_bytes(*bad) == 0
    assert A.ivfpq_table_grad_bytes(100000, 64) > 0
    assert A.ivfpq_table_grad_bytes(32, 64) == 0    # no list is long
    for bad in ((-1, 64, 1), (1 << 30, 64, 2), (100000, 0, 1), (100000, 64, 0)):
        assert A.ivfpq_table_grad_bytes(*bad) == 0
    for bad in ((-1, 8, 8, 1), (8, 0, 8, 1), (8, 8, 0, 1), (8, 8, 8, 0)):
        assert A.ivfpq_list_product_grad_bytes(*bad) == 0


def test_host_tensors_are_refused():
    x, m = torch.zeros((4, 8)), torch.zeros((2, 8, 8))
    offsets = torch.zeros(3, dtype=torch.int32)
    order = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: A.ivfpq_list_product_ex(x, m, offsets),
                 lambda: A.ivfpq_list_product_ex(x.double(), m, offsets),
                 lambda: A.ivfpq_list_product_grad_ex(x, x, offsets),
                 lambda: A.ivfpq_adapter_product_ex(x, x, m, m, offsets, order, order),
                 lambda: A.ivfpq_table_lookup_ex(x, order),
                 lambda: A.ivfpq_table_grad_ex(x, offsets, order)):
        with pytest.raises(ValueError):
            call()
