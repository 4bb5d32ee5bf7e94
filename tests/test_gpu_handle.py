"""Making a handle of the library beside running work."""
import pytest
import torch

import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu


def test_a_new_handle_does_not_wait_for_the_devices_work():
    pkg.Handle(0).close()                    # the library and the context are up
    stream, done = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(1_500_000_000)     # most of a second
        done.record()
    h = pkg.Handle(0)
    running = not done.query()
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    A, B = torch.ones((1, 8, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((1, 64, 8), dtype=torch.bfloat16, device="cuda")
    ad = pkg.moe_lora_linear_adapters(h, A, B, [8], [1.0])
    y = pkg.moe_lora_linear(h, x, x.new_zeros((64, 64)), ad, torch.zeros(4, dtype=torch.int32, device="cuda"))
    torch.cuda.current_stream().synchronize()
    assert (y == 512.0).all()                # its flags are in order from the first call on
    torch.cuda.synchronize()
    assert running
    h.close()
