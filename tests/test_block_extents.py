"""Sizes near 2^31 are refused on the host, where indices of whole tiles would no longer fit 32 bits (the
handle and device addresses given are never dereferenced)."""
import ctypes

import pytest

import test_block_abi as abi
from routed_moe_expert_gb300 import binding as B

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("over", [dict(T=MOST), dict(T=MOST - 254), dict(N=MOST, y_stride=MOST), dict(K=MOST - 7, x_stride=MOST + 1, w_stride=MOST + 1)],
                         ids=["T", "T-254", "N", "K"])
def test_linear(built_lib, over):
    assert abi._linear(**over) == 2


def test_linear_sizes(built_lib):
    n, r = ctypes.c_size_t(), (ctypes.c_int32 * 1)(8)
    assert B.lib().moe_lora_linear_workspace_size(MOST, 1, r, ctypes.byref(n)) == 2
    assert B.lib().moe_lora_linear_workspace_size(MOST - 255, 1, r, ctypes.byref(n)) == 0 and n.value > 2 ** 31 * 64 * 6 - 2 ** 20
    assert B.lib().moe_lora_linear_adapters_size(1, MOST, 8, r, ctypes.byref(n)) == 2
    assert B.lib().moe_lora_linear_adapters_size(1, 8, MOST - 7, r, ctypes.byref(n)) == 2


def test_select(built_lib):
    assert abi._select(T=MOST) == 2


def test_qk_norm_rope(built_lib):
    assert abi._qk(T=MOST) == 2
    assert abi._qk(q_heads=MOST, k_heads=2) == 1
