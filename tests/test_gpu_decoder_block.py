"""The operators around the layer run together as the example does, each stage checked in 64 bits
from the tensors it was given."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_reference as ref
import gpu_helpers as gh
import routed_moe_expert_gb300 as pkg
from oracle import moe_lora_oracle as orc
from routed_moe_expert_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T", [1, 45])
def test_block_stage_by_stage(T):
    ex = _example()
    handle = pkg.Handle(0)
    cfg = wl.LayerConfig("block", T=T, H=256, I=128, E=16, top_k=4, ranks=(8, 16), scalings=(2.0, 0.5))
    shape = ex.Shape(cfg, q_heads=4, k_heads=2, head_dim=64, n_group=4, topk_group=2, max_positions=100)
    b = ex.DecoderBlock(handle, shape, seed=3)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, 256), generator=g).bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32) + 7
    slots = torch.randint(-1, 2, (T,), generator=g, dtype=torch.int32)
    _, st = b(x, pos.cuda(), slots.cuda())
    torch.cuda.synchronize()

    def near(got, want):
        err = np.abs(ref.f64(got) - want[0])
        assert (err <= want[1]).all(), np.max(err / want[1])
    A, Bm = b.lora[(b.rows, 256)]
    lin = ref.linear(st["h1"], b.w_qkv, None, A, Bm, slots.numpy(), cfg.ranks, cfg.scalings)
    nq, nk = 4 * 64, 2 * 64
    near(st["q_in"].reshape(T, -1), (lin[0][:, :nq], lin[1][:, :nq]))
    near(st["k_in"].reshape(T, -1), (lin[0][:, nq:nq + nk], lin[1][:, nq:nq + nk]))
    near(st["qkv"][:, nq + nk:], (lin[0][:, nq + nk:], lin[1][:, nq + nk:]))     # the values stay as projected
    near(st["q"], ref.norm_rope(st["q_in"], b.norm_q, b.table, pos, 1e-6, False))
    near(st["k"], ref.norm_rope(st["k_in"], b.norm_k, b.table, pos, 1e-6, False))
    A, Bm = b.lora[(256, nq)]
    near(st["out"], ref.linear(st["attn"], b.w_out, None, A, Bm, slots.numpy(), cfg.ranks, cfg.scalings))
    near(st["logits"], ref.linear(st["h2"], b.w_router, f32=True))
    ids, w, keys = ref.select(st["logits"], 4, True, b.balance, 4, 2, True, True, 2.5)
    got = st["route"]["topk_ids"].cpu().numpy()
    for t in range(T):   # the same experts, unless two keys are closer than float32 tells apart
        if (got[t] != ids[t]).any():
            assert np.allclose(np.sort(keys[t][got[t]]), np.sort(keys[t][ids[t]]), rtol=0, atol=1e-6)
        else:
            np.testing.assert_allclose(st["route"]["topk_weights"][t].cpu().numpy(), w[t], rtol=1e-5)
    e = b.experts
    want = orc.moe_lora_forward_routed(
        gh.np_(st["h2"]), st["route"]["packed_topk_ids"].cpu().numpy(), gh.np_(e["w1"]), gh.np_(e["w2"]), 4, 16,
        lora_A_gu=gh.np_(e["lora_A_gu"]), lora_B_gu=gh.np_(e["lora_B_gu"]), lora_A_dn=gh.np_(e["lora_A_dn"]),
        lora_B_dn=gh.np_(e["lora_B_dn"]), slot_idx=slots.numpy(), ranks=e["ranks"], scalings=e["scalings"])
    gh.assert_close(st["moe"].float().cpu().numpy(), want["out"], "experts")
    handle.close()


def test_example_runs():
    _example().main(5)
