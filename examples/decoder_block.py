"""A decoder block of an adapter-served mixture-of-experts model, from the residual stream and back:

  merged q/k/v projection with per-token adapters  (moe_lora_linear)
  norm of q and k heads and position rotation       (moe_lora_qk_norm_rope, in place on the rows)
  attention                                          (the caller's; plain torch here)
  output projection with adapters                    (moe_lora_linear)
  router logits in float32                           (moe_lora_linear)
  choice of experts, packed                          (moe_lora_select_experts)
  the experts with their adapters                    (moe_lora_forward_routed)

    python examples/decoder_block.py [tokens]

Random weights; the sizes are those of the decode configuration's expert layer.  What stands
between (layer norms, residual additions) is the caller's as well.
"""
import dataclasses
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_moe_expert_gb300 as pkg  # noqa: E402
from routed_moe_expert_gb300 import workloads as wl  # noqa: E402


@dataclasses.dataclass
class Shape:
    experts: wl.LayerConfig
    q_heads: int = 32
    k_heads: int = 4
    head_dim: int = 128
    n_group: int = 8
    topk_group: int = 4
    max_positions: int = 4096


def rms(x, eps=1e-6):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + eps)).to(x.dtype)


class DecoderBlock:
    """Weights, stacked adapters and workspaces of one block: what a serving program keeps."""

    def __init__(self, handle, shape: Shape, seed=0, device="cuda"):
        self.handle, self.shape = handle, shape
        cfg = shape.experts
        g = torch.Generator(device=device).manual_seed(seed + 100)
        H, D = cfg.H, shape.head_dim
        self.rows = (shape.q_heads + 2 * shape.k_heads) * D

        def rand(*s, std):
            return (torch.randn(s, generator=g, device=device) * std).bfloat16()

        def adapters(n, k):
            self.lora[(n, k)] = (rand(cfg.S, cfg.R, k, std=1 / math.sqrt(k)), rand(cfg.S, n, cfg.R, std=0.02))
            return pkg.moe_lora_linear_adapters(handle, *self.lora[(n, k)], list(cfg.ranks), list(cfg.scalings))

        self.lora = {}
        self.w_qkv, self.w_out = rand(self.rows, H, std=1 / math.sqrt(H)), rand(H, shape.q_heads * D, std=1 / math.sqrt(H))
        self.w_router = rand(cfg.E, H, std=1 / math.sqrt(H))
        self.a_qkv, self.a_out = adapters(self.rows, H), adapters(H, shape.q_heads * D)
        self.norm_q, self.norm_k = 1 + rand(D, std=0.1), 1 + rand(D, std=0.1)
        self.balance = torch.randn(cfg.E, generator=g, device=device) * 0.05
        freq = 1e6 ** (-torch.arange(0, D, 2, device=device, dtype=torch.float64) / D)
        angle = torch.arange(shape.max_positions, device=device, dtype=torch.float64)[:, None] * freq
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.experts = wl.make_inputs(cfg, seed=seed, device=device, T=1)

    def attention(self, q, k, v):
        """Causal attention over the tokens of this call: the caller's own, here in plain torch."""
        n = self.shape.q_heads // self.shape.k_heads
        k, v = (t.repeat_interleave(n, 1) for t in (k, v))
        s = torch.einsum("thd,uhd->htu", q.float(), k.float()) / math.sqrt(q.shape[2])
        T = q.shape[0]
        s = s.masked_fill(torch.ones((T, T), dtype=torch.bool, device=q.device).triu(1), -math.inf)
        return torch.einsum("htu,uhd->thd", s.softmax(2), v.float()).bfloat16().reshape(T, -1)

    def __call__(self, x, positions, slots):
        """x [T, H] bf16 -> (x after the block, every stage's tensors by name)."""
        s, cfg, h, T = self.shape, self.shape.experts, self.handle, x.shape[0]
        D, nq = s.head_dim, s.q_heads * s.head_dim
        st = {"x": x, "h1": rms(x)}
        qkv = st["qkv"] = pkg.moe_lora_linear(h, st["h1"], self.w_qkv, self.a_qkv, slots)
        q, k, v = (qkv[:, a:b].view(T, -1, D) for a, b in
                   ((0, nq), (nq, nq + s.k_heads * D), (nq + s.k_heads * D, self.rows)))
        st["q_in"], st["k_in"] = q.clone(), k.clone()
        pkg.moe_lora_qk_norm_rope(h, q, k, self.norm_q, self.norm_k, self.table, positions, q_out=q, k_out=k)
        st["q"], st["k"] = q, k
        st["attn"] = self.attention(q, k, v)
        st["out"] = pkg.moe_lora_linear(h, st["attn"], self.w_out, self.a_out, slots)
        x = st["x2"] = x + st["out"]
        st["h2"] = rms(x)
        st["logits"] = pkg.moe_lora_linear(h, st["h2"], self.w_router, out_dtype=torch.float32)
        r = st["route"] = pkg.moe_lora_select_experts(
            h, st["logits"], cfg.top_k, scoring=pkg.SCORE_SIGMOID, bias=self.balance, n_group=s.n_group,
            topk_group=s.topk_group, group_score=pkg.GROUP_TOP2, routed_scaling_factor=2.5, packed=True)
        e = self.experts
        st["moe"] = pkg.moe_lora_forward_routed(
            h, st["h2"], r["packed_topk_ids"], e["w1"], e["w2"], cfg.top_k, cfg.E, lora_A_gu=e["lora_A_gu"],
            lora_B_gu=e["lora_B_gu"], lora_A_dn=e["lora_A_dn"], lora_B_dn=e["lora_B_dn"], slot_idx=slots,
            ranks=e["ranks"], scalings=e["scalings"])
        return x + st["moe"], st


def main(tokens=64):
    cfg = wl.CONFIGS["decode"]
    handle = pkg.Handle(0)
    block = DecoderBlock(handle, Shape(cfg))
    x = torch.randn((tokens, cfg.H), device="cuda").bfloat16()
    positions = torch.arange(tokens, device="cuda", dtype=torch.int32)
    slots = torch.randint(-1, cfg.S, (tokens,), device="cuda", dtype=torch.int32)
    y, st = block(x, positions, slots)
    torch.cuda.synchronize()
    load = torch.bincount(st["route"]["topk_ids"].flatten().long(), minlength=cfg.E)
    print(f"{tokens} tokens: block output rms {y.float().square().mean().sqrt().item():.3f}, "
          f"{int((load > 0).sum())} of {cfg.E} experts used")


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
