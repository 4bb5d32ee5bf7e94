"""Float32 results of moe_lora_linear over a long K: no accumulator of the tensor cores, which truncate,
takes more than 1024 of K."""
import numpy as np
import pytest
import torch

import block_reference as ref
import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks", [(), (8,), (16,) * 12], ids=["none", "8", "192"])
@pytest.mark.parametrize("T,N,K", [(1, 2048, 18432), (2, 136, 9224), (20, 300, 40960), (60, 136, 30728), (128, 136, 16384),
                                   (100, 264, 70000), (300, 200, 18432), (3, 384, 7168)])
def test_an_accumulator_takes_1024_of_k(T, N, K, ranks):
    """The first product is 2^24 (ulp 2), all others 2^-4: the 16 that one step of the tensor cores adds
    come to 1, which truncation loses where the 2^24 is.  At most 1024 / 16 of them share its
    accumulator; the sums of the other accumulators are exact, and joining them costs half an ulp (1)
    each, of K / 1024 + 8 at most."""
    x = torch.full((T, K), 0.25, dtype=torch.bfloat16)
    w = torch.full((N, K), 0.25, dtype=torch.bfloat16)
    x[:, 0] = 4096.0
    w[:, 0] = 4096.0
    handle, ad, slots = pkg.Handle(0), None, None
    if ranks:   # adapters that add nothing; the last token has none
        S = len(ranks)
        A = torch.ones((S, max(ranks), K), dtype=torch.bfloat16, device="cuda")
        ad = pkg.moe_lora_linear_adapters(handle, A, torch.zeros((S, N, max(ranks)), dtype=torch.bfloat16, device="cuda"),
                                          list(ranks), [1.0] * S)
        slots = (torch.arange(T) % S).to(torch.int32)
        slots[T - 1] = -1
        slots = slots.cuda()
    got = ref.f64(pkg.moe_lora_linear(handle, x.cuda(), w.cuda(), ad, slots, out_dtype=torch.float32))
    want = 2.0 ** 24 + (K - 1) * 2.0 ** -4
    assert np.abs(got - want).max() <= 1024 / 16 + K / 1024 + 8
    handle.close()
