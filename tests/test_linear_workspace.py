"""One workspace for calls of several sizes: what is enough for a call is enough for every smaller one."""
import ctypes
import random

import pytest
import torch

import routed_moe_expert_gb300 as pkg
from routed_moe_expert_gb300 import binding as B
from test_linear_choice import choice


def _size(T, stack):
    """Bytes for T tokens and `stack` stacked columns, in slots of up to 128 ranks."""
    ranks = [128] * (stack // 128) + ([stack % 128] if stack % 128 else [])
    n = ctypes.c_size_t()
    r = (ctypes.c_int32 * max(len(ranks), 1))(*ranks)
    assert B.lib().moe_lora_linear_workspace_size(T, len(ranks), r, ctypes.byref(n)) == 0
    return n.value


def test_the_size_never_falls(built_lib):
    Ts = [0, 1, 64, 128, 129, 256, 257, 300, 2560, 6656, 8192, 27135, 27136, 27137, 27392, 32768, 100000, 2 ** 20]
    stacks = [0, 64, 128, 192, 256, 512, 4096]
    for T in Ts:
        for a, b in zip(stacks, stacks[1:]):
            assert _size(T, a) <= _size(T, b), (T, a, b)
    for s in stacks:
        for a, b in zip(Ts, Ts[1:]):
            assert _size(a, s) <= _size(b, s), (s, a, b)


def test_the_size_covers_every_choice(built_lib):
    rng = random.Random(3)
    for _ in range(20000):
        T, N = int(2 ** rng.uniform(0, 16)), int(2 ** rng.uniform(0, 14))
        K, Rs = 8 * int(2 ** rng.uniform(0, 10)), rng.choice([64, 128, 192, 1024])
        c = choice(T, N, K, rng.random() < 0.5, Rs)
        parts = 0 if c["slices"] == 1 else (T + 255) // 256 * c["slices"] * Rs * 1024
        assert 256 + T * Rs * 6 + parts <= _size(T, Rs), (T, N, K, Rs, c)


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K,most_T,most_ranks", [(27136, 256, 2048, 32768, (64, 64)), (8192, 1792, 7168, 8192, (64, 64, 64)),
                                                     (300, 8000, 512, 300, (128, 64)), (777, 1536, 2048, 40000, (64, 64))])
def test_a_larger_calls_workspace(T, N, K, most_T, most_ranks):
    handle = pkg.Handle(0)
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.05).bfloat16()
    make = lambda ranks: pkg.moe_lora_linear_adapters(handle, r(len(ranks), max(ranks), K), r(len(ranks), N, max(ranks)),
                                                      list(ranks), [1.0] * len(ranks))
    ad = make((64, 48))
    x, w = r(T, K), r(N, K)
    slots = torch.randint(-1, 2, (T,), generator=g, device="cuda").int()
    ws = pkg.alloc_linear_workspace(most_T, make(most_ranks))
    own = pkg.alloc_linear_workspace(T, ad)
    assert ws.numel() >= own.numel()
    assert torch.equal(pkg.moe_lora_linear(handle, x, w, ad, slots, workspace=ws),
                       pkg.moe_lora_linear(handle, x, w, ad, slots, workspace=own))
    handle.close()
