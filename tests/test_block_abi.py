"""The operators around the layer without a GPU: host checks of their C entry points (which return
before any device work; the handle and device addresses given here are never dereferenced), sizes
and layouts, what the Python side refuses, and pins of their 64-bit reference."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as ref
from routed_moe_expert_gb300 import binding as B

FAKE = 0x7f0000000000          # 16-byte aligned fake device address
P, I, F, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64


class SelectArgs(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("logits", "bias", "topk_ids", "topk_weights", "packed_topk_ids")] + [("logits_stride", L)] +
                [(n, I) for n in ("T", "E", "top_k", "logits_f32", "scoring", "n_group", "topk_group", "group_score",
                                  "renormalize")] + [("factor", F)])


class LinearArgs(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("x", "w", "bias", "y", "adapters", "slot_idx", "h_ranks", "h_scalings")] +
                [(n, L) for n in ("x_stride", "w_stride", "y_stride")] + [(n, I) for n in ("T", "N", "K", "S", "y_f32")])


class QkArgs(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("q", "k", "q_out", "k_out", "q_weight", "k_weight", "cos_sin", "positions")] +
                [(n, L) for n in ("q_t", "q_h", "k_t", "k_h", "qo_t", "qo_h", "ko_t", "ko_h", "cs_stride")] +
                [(n, I) for n in ("T", "q_heads", "k_heads", "head_dim", "rotary_dim", "num_positions", "weight_f32",
                                  "positions_i64", "interleaved")] + [("eps", F)])


def _fill(s, vals, over):
    for k, v in {**vals, **over}.items():
        setattr(s, k, ctypes.cast(v, P) if isinstance(v, ctypes.Array) else v)
    return s


def _select(h=FAKE, **over):
    a = _fill(SelectArgs(), dict(logits=FAKE, topk_ids=FAKE, topk_weights=FAKE, logits_stride=64, T=4, E=64, top_k=8,
                                 n_group=1, topk_group=1, factor=1.0), over)
    return B.lib().moe_lora_select_experts(P(h), ctypes.byref(a), None)


@pytest.mark.parametrize("over,code", [
    (dict(h=0), 1), (dict(T=-1), 1), (dict(E=0), 1), (dict(E=1025), 1), (dict(top_k=0), 1), (dict(top_k=33), 1),
    (dict(scoring=2), 1), (dict(group_score=2), 1), (dict(n_group=0), 1), (dict(n_group=5, topk_group=2), 1),
    (dict(n_group=8, topk_group=0), 1), (dict(n_group=8, topk_group=9), 1), (dict(n_group=16, topk_group=1), 1),
    (dict(n_group=64, topk_group=8), 2), (dict(n_group=32, topk_group=8, E=32, group_score=1), 1),
    (dict(factor=float("nan")), 1), (dict(logits_stride=63), 1), (dict(logits=None), 1), (dict(topk_ids=None), 1),
    (dict(topk_weights=None), 1), (dict(logits=FAKE + 1), 1), (dict(logits=FAKE + 2, logits_f32=1), 1),
    (dict(bias=FAKE + 2), 1), (dict(packed_topk_ids=FAKE + 1), 1), (dict(T=0, logits=None), 0)])
def test_select_host_checks(built_lib, over, code):
    assert _select(**over) == code


RANKS, SCAL = (ctypes.c_int32 * 2)(8, 16), (ctypes.c_float * 2)(1.0, 2.0)


def _linear(h=FAKE, ws=FAKE, nbytes=1 << 30, **over):
    a = _fill(LinearArgs(), dict(x=FAKE, w=FAKE, y=FAKE, adapters=FAKE, slot_idx=FAKE, h_ranks=RANKS, h_scalings=SCAL,
                                 x_stride=64, w_stride=64, y_stride=32, T=4, N=32, K=64, S=2), over)
    return B.lib().moe_lora_linear(P(h), ctypes.byref(a), P(ws), ctypes.c_size_t(nbytes), None)


@pytest.mark.parametrize("over,code", [
    (dict(h=0), 1), (dict(T=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=60), 1), (dict(S=65), 1), (dict(S=-1), 1),
    (dict(h_ranks=None), 1), (dict(h_scalings=None), 1), (dict(h_ranks=(ctypes.c_int32 * 2)(8, 129)), 1),
    (dict(h_ranks=(ctypes.c_int32 * 2)(-1, 8)), 1), (dict(h_scalings=(ctypes.c_float * 2)(1.0, float("nan"))), 1),
    (dict(x_stride=63), 1), (dict(x_stride=68), 1), (dict(w_stride=56), 1), (dict(y_stride=31), 1), (dict(x=None), 1),
    (dict(w=None), 1), (dict(y=None), 1), (dict(ws=0), 1), (dict(x=FAKE + 8), 1), (dict(w=FAKE + 2), 1),
    (dict(y=FAKE + 1), 1), (dict(y=FAKE + 2, y_f32=1), 1), (dict(bias=FAKE + 2), 1), (dict(ws=FAKE + 8), 1),
    (dict(slot_idx=None), 1), (dict(slot_idx=FAKE + 2), 1), (dict(adapters=None), 1), (dict(adapters=FAKE + 8), 1),
    (dict(nbytes=255), 3), (dict(nbytes=256), 3), (dict(T=0, x=None, y=None), 0),
    (dict(S=64, h_ranks=(ctypes.c_int32 * 64)(*[72] * 64), h_scalings=(ctypes.c_float * 64)(*[1.0] * 64)), 2)])
def test_linear_host_checks(built_lib, over, code):
    assert _linear(**over) == code


def test_linear_adapter_and_workspace_sizes(built_lib):
    L_ = B.lib()
    n = ctypes.c_size_t()
    al = lambda b: (b + 255) // 256 * 256
    # ranks rounded up to 8, the stack to 64 columns: 8 + 16 + 24 = 48 -> 64
    r = (ctypes.c_int32 * 4)(5, 16, 0, 17)
    assert L_.moe_lora_linear_adapters_size(4, 100, 72, r, ctypes.byref(n)) == 0
    assert n.value == al(64 * 72 * 2) + al(64 * 100 * 2)
    assert L_.moe_lora_linear_workspace_size(7, 4, r, ctypes.byref(n)) == 0
    assert n.value == 256 + al(7 * 64 * 3 * 2)
    assert B.moe_lora_linear_workspace_size(9) == 256
    assert L_.moe_lora_linear_adapters_size(2, 8, 8, (ctypes.c_int32 * 2)(0, 0), ctypes.byref(n)) == 0 and n.value == 0
    bad = lambda S, N, K, ranks: L_.moe_lora_linear_adapters_size(S, N, K, (ctypes.c_int32 * max(S, 1))(*ranks), ctypes.byref(n))
    assert bad(0, 8, 8, [0]) == 1 and bad(1, 0, 8, [8]) == 1 and bad(1, 8, 12, [8]) == 1 and bad(1, 8, 8, [129]) == 1
    assert bad(64, 8, 8, [65] * 64) == 2
    pack = lambda **o: L_.moe_lora_linear_pack_adapters(
        P(o.get("h", FAKE)), P(o.get("A", FAKE)), P(o.get("Bm", FAKE)), 1, 8, 8, o.get("R", 8), (ctypes.c_int32 * 1)(8),
        P(o.get("out", FAKE)), None)
    assert pack(h=0) == 1 and pack(A=0) == 1 and pack(A=FAKE + 2) == 1 and pack(Bm=0) == 1 and pack(out=FAKE + 4) == 1
    assert pack(R=4) == 1 and pack(R=129) == 1


def _qk(h=FAKE, ws=None, nbytes=0, **over):
    a = _fill(QkArgs(), dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, q_weight=FAKE, k_weight=FAKE, cos_sin=FAKE,
                             positions=FAKE, q_t=256, q_h=64, k_t=64, k_h=64, qo_t=256, qo_h=64, ko_t=64, ko_h=64,
                             cs_stride=64, T=4, q_heads=4, k_heads=1, head_dim=64, rotary_dim=64, num_positions=100,
                             eps=1e-6), over)
    return B.lib().moe_lora_qk_norm_rope(P(h), ctypes.byref(a), P(ws), ctypes.c_size_t(nbytes), None)


@pytest.mark.parametrize("over,code", [
    (dict(h=0), 1), (dict(T=-1), 1), (dict(q_heads=-1), 1), (dict(q_heads=0, k_heads=0), 1), (dict(head_dim=0), 1),
    (dict(head_dim=513), 2), (dict(rotary_dim=63), 1), (dict(rotary_dim=66), 1), (dict(num_positions=-1), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(q=None), 1), (dict(k_out=None), 1), (dict(q_weight=None), 1),
    (dict(positions=None), 1), (dict(cos_sin=None), 1), (dict(q=FAKE + 1), 1), (dict(cos_sin=FAKE + 2), 1),
    (dict(positions=FAKE + 4, positions_i64=1), 1), (dict(q_weight=FAKE + 2, weight_f32=1), 1), (dict(ws=FAKE, nbytes=3), 3),
    (dict(ws=FAKE + 1, nbytes=256), 1), (dict(T=0, q=None), 0)])
def test_qk_norm_rope_host_checks(built_lib, over, code):
    assert _qk(**over) == code


def test_python_side_refuses_cpu_tensors_and_wrong_types(built_lib):
    class H:
        address = FAKE
    z = torch.zeros(4, 8)
    for bad, what in ((lambda: B.moe_lora_select_experts(H, z, 2), "logits"),
                      (lambda: B.moe_lora_select_experts(H, [1.0], 2), "logits"),
                      (lambda: B.moe_lora_linear(H, z.bfloat16(), z.bfloat16()), "x"),
                      (lambda: B.moe_lora_linear(H, z, z, out_dtype=torch.float16), "out_dtype"),
                      (lambda: B.moe_lora_qk_norm_rope(H, z, z, z, z, z, z), "q"),
                      (lambda: B.moe_lora_linear_adapters(H, z, z, [], []), "A")):
        with pytest.raises(ValueError, match=what):
            bad()


def test_marshal_module_missing_fails_loudly(monkeypatch):
    monkeypatch.setattr(B, "_marshal", None)
    monkeypatch.setattr(B, "PKG", "/nonexistent")
    with pytest.raises(B.MoELoRAError):
        B._native()


# -------------------------------------------------------------------------- pins of the reference
def test_reference_linear_is_the_merged_weight():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g).bfloat16()
    x, w, A, Bm = r(6, 16), r(5, 16), r(2, 4, 16), r(2, 5, 4)
    slots = np.array([0, 1, -1, 0, 1, 1])
    y, tol = ref.linear(x, w, None, A, Bm, slots, [4, 3], [0.5, 2.0])
    for t, s in enumerate(slots):
        m = w.double()
        if s >= 0:
            n = [4, 3][s]
            m = m + [0.5, 2.0][s] * Bm[s, :, :n].double() @ A[s, :n].double()
        np.testing.assert_allclose(y[t], (m @ x[t].double()).numpy(), rtol=1e-12)
    assert (tol > 0).all()


def test_reference_select_agrees_with_sorting_by_hand():
    z = torch.tensor([[0.0, 2.0, 1.0, 2.0], [1.0, float("-inf"), 0.0, 3.0]])
    ids, w, _ = ref.select(z, 2, True)
    assert ids.tolist() == [[1, 3], [3, 0]]
    np.testing.assert_allclose(w[0], [0.5, 0.5])
    ids, w, _ = ref.select(z, 2, False, n_group=2, topk_group=1, top2=True, renormalize=False)
    assert ids.tolist() == [[3, 2], [3, 2]]          # the second group holds the better two
    e = np.exp(z[0].double().numpy())
    np.testing.assert_allclose(w[0], [e[3] / e.sum(), e[2] / e.sum()])
    ids, _, _ = ref.select(z, 1, True, bias=torch.tensor([5.0, 9.0, 0.0, 0.0]))
    assert ids.tolist() == [[1], [0]]                # the bias lifts no ruled-out expert


def test_reference_norm_rope_turns_and_keeps_lengths():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((3, 2, 8), generator=g)
    a = torch.rand((5, 3), generator=g, dtype=torch.float64) * 6.3
    table = torch.cat([a.cos(), a.sin()], 1)
    pos = torch.tensor([0, 4, 7])                    # the last is out of range
    one = torch.ones(8)
    for inter in (False, True):
        y, _ = ref.norm_rope(x, one, table, pos, 0.0, inter)
        np.testing.assert_allclose((y * y).sum(2), 8.0, rtol=1e-12)       # unit mean square, turned
        n = x.double().numpy() / np.sqrt((x.double().numpy() ** 2).mean(2, keepdims=True))
        np.testing.assert_allclose(y[2], n[2])                             # no rotation
        np.testing.assert_allclose(y[:, :, 6:], n[:, :, 6:])               # the values past R
        pair = (0, 1) if inter else (0, 3)
        turned = (n[1, 0, pair[0]] + 1j * n[1, 0, pair[1]]) * np.exp(1j * a[4, 0].item())
        np.testing.assert_allclose(y[1, 0, list(pair)], [turned.real, turned.imag])
