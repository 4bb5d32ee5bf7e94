"""A decoder block over the paged cache, as the example runs it: prompts in pieces, drafts and single tokens, their
attention held to its definition in 64 bits on all the keys and values that the steps before brought."""
import dataclasses
import importlib.util
import math
import os

import pytest
import torch

import paged_reference as ref
import routed_moe_expert_gb300 as pkg
from routed_moe_expert_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_steps_over_the_cache():
    ex = _example()
    cfg = dataclasses.replace(wl.CONFIGS["tiny"], H=256, E=16)
    h = pkg.Handle(0)
    shape = ex.Shape(cfg, q_heads=8, k_heads=2, head_dim=64, n_group=2, topk_group=1)
    block = ex.DecoderBlock(h, shape)
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = ex.Cache(h, shape, requests=2, pages=16, page_size=16, max_pages=6)
    at, keys, values = [0, 0], [[], []], [[], []]
    for new in ([40, 0], [17, 5], [1, 1], [4, 4], [8, 23]):
        T = sum(new) + 2   # two rows of padding
        rows = torch.randn((T, cfg.H), generator=g, device="cuda").bfloat16()
        pos = cache.step(torch.tensor(new, dtype=torch.int32, device="cuda"), T)
        assert pos.tolist() == [p for a, n in zip(at, new) for p in range(a, a + n)] + [0, 0]
        st = block(rows, pos, torch.zeros(T, dtype=torch.int32, device="cuda"), cache, max(new))[1]
        torch.cuda.synchronize()
        v = st["qkv"][:, -2 * 64:].view(T, 2, 64)
        t = 0
        for b, n in enumerate(new):
            keys[b].append(st["k"][t:t + n].cpu())
            values[b].append(v[t:t + n].cpu())
            at[b] += n
            if n > 0:   # the request by itself, in one page that holds it all
                k1, v1 = (torch.cat(x[b]).transpose(0, 1)[None] for x in (keys, values))
                want, _, tol, _ = ref.attention(st["q"][t:t + n], k1, v1, [[0]], [at[b]], [0, n], 0.125, ref.TILES)
                got = st["attn"][t:t + n].view(n, 8, 64).double().cpu()
                assert ((got - want).abs() <= tol).all()
            t += n
    assert cache.lens.tolist() == at and int(cache.taken) == sum(-(-n // 16) for n in at)
    h.close()


def test_example_runs(capsys):
    _example().main(20)
    said = capsys.readouterr().out
    assert "tokens cached: [21, 5]" in said
    assert math.isfinite(float(said.split("rms ")[1].split(",")[0]))
