"""The operators around the layer run on their handle's device: tensors of another are refused on the
host.  The other device is a stand-in handle that says so; nothing of it is used but that number."""
import ctypes

import pytest
import torch

from routed_moe_expert_gb300 import binding as B


class Other:
    """A handle whose device is cuda:1 (the first member of the structure)."""

    def __init__(self):
        self.memory = (ctypes.c_int32 * 4096)(1)
        self.address = ctypes.addressof(self.memory)
        self.device = 1


def test_the_device_of_a_handle(built_lib):
    d = ctypes.c_int(-1)
    assert B.lib().moe_lora_device(Other().address, ctypes.byref(d)) == 0 and d.value == 1
    assert B.lib().moe_lora_device(None, ctypes.byref(d)) == 1 and B.lib().moe_lora_device(Other().address, None) == 1


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused():
    h = Other()
    z = torch.zeros((4, 64), device="cuda:0")
    b = z.bfloat16()
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda:0")
    w = torch.ones(64, device="cuda:0")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    A = torch.zeros((1, 8, 64), dtype=torch.bfloat16, device="cuda:0")
    for bad in (lambda: B.moe_lora_select_experts(h, z, 4), lambda: B.moe_lora_linear(h, b, b),
                lambda: B.moe_lora_qk_norm_rope(h, q, q, w, w, z, pos),
                lambda: B.moe_lora_linear_adapters(h, A, torch.zeros((1, 16, 8), dtype=torch.bfloat16, device="cuda:0"), [8], [1.0])):
        with pytest.raises(ValueError, match="handle is on cuda:1"):
            bad()
    with pytest.raises(B.MoELoRAError):     # a closed handle
        closed = B.Handle(0)
        closed.close()
        B.moe_lora_select_experts(closed, z, 4)


@pytest.mark.gpu
def test_a_top_k_past_the_experts_allocates_nothing():
    h = B.Handle(0)
    z = torch.zeros((1024, 64), device="cuda:0")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for k in (65, 2 ** 20, 2 ** 31 - 1, 0, -3):
        with pytest.raises(B.MoELoRAError) as e:
            B.moe_lora_select_experts(h, z, k, packed=True)
        assert e.value.status == 1
    assert torch.cuda.max_memory_allocated() == before
    h.close()
