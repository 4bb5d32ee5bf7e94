"""Part sums of a sliced shrink (moe_lora_linear) are read only once they are written: the same bits
again and again, whatever the part sums' memory held."""
import math

import numpy as np
import pytest
import torch

import block_reference as ref
import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu


# one slice per pair, slices on every pair besides its product tile, slices dealt out over long batches
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K,ranks", [(777, 1536, 2048, (16, 40)), (2450, 1560, 1640, (64, 48)), (300, 8000, 512, (16, 40)),
                                         (5000, 1792, 7168, (64, 48))])
def test_part_sums_of_another_call_are_never_taken(T, N, K, ranks, f32):
    handle, g = pkg.Handle(0), torch.Generator().manual_seed(T)
    r = lambda shape, std: (torch.randn(shape, generator=g) * std).bfloat16()
    S, R = len(ranks), max(ranks)
    x, w, A, B = r((T, K), 1.0), r((N, K), 1 / math.sqrt(K)), r((S, R, K), 1 / math.sqrt(K)), r((S, N, R), 0.3)
    slots = ((torch.arange(T) // 50) % (S + 1) - 1).to(torch.int32)
    ad = pkg.moe_lora_linear_adapters(handle, A.cuda(), B.cuda(), list(ranks), [2.0, 0.5])
    ws = pkg.alloc_linear_workspace(T, ad)
    d = [t.cuda() for t in (x, w, slots)]
    run = lambda t: pkg.moe_lora_linear(handle, t, d[1], ad, d[2], out_dtype=torch.float32 if f32 else torch.bfloat16,
                                        workspace=ws)
    ws.fill_(255)
    first = run(d[0])
    y, tol = ref.linear(x, w, None, A, B, slots.numpy(), ranks, [2.0, 0.5], f32)
    assert (np.abs(ref.f64(first) - y) <= tol).all()
    other = torch.full_like(d[0], float("nan"))
    for _ in range(30):
        run(other)                      # leaves NaN in every part sum
        assert torch.equal(run(d[0]), first)
    handle.close()
