"""The operators over the paged cache without a GPU: host checks of their C entry points (which return before any
device work; the addresses given here are never dereferenced), what the Python side refuses, workspace
sizes, and pins of their 64-bit reference."""
import ctypes
import math

import pytest
import torch

import paged_reference as ref
from routed_moe_expert_gb300 import binding as B

FAKE = 0x7f0000000000          # 16-byte aligned fake device address
P, I, F, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64


class TableArgs(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("block_tables", "cached_lens", "new_lens", "free_pages", "taken", "kv_lens", "query_offsets",
                                  "slot_map", "positions", "taken_out")] + [("stride", L)] +
                [(n, I) for n in ("B", "width", "page", "num_free", "T")])


class WriteArgs(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("k", "v", "k_cache", "v_cache", "slot_map")] +
                [(n, L) for n in ("k_t", "k_h", "v_t", "v_h", "kc_p", "kc_h", "kc_t", "vc_p", "vc_h", "vc_t")] +
                [(n, I) for n in ("T", "heads", "head_dim", "num_pages", "page")])


class AttentionArgs(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("q", "k_cache", "v_cache", "block_tables", "kv_lens", "query_offsets", "out", "lse")] +
                [(n, L) for n in ("q_t", "q_h", "o_t", "o_h", "kc_p", "kc_h", "kc_t", "vc_p", "vc_h", "vc_t", "stride")] +
                [(n, I) for n in ("T", "B", "q_heads", "k_heads", "head_dim", "num_pages", "page", "width", "max_query_len",
                                  "shared_len")] + [("scale", F)])


def _call(fn, args, vals, over, h=FAKE, ws=None, nbytes=0):
    a = args()
    for k, v in {**vals, **over}.items():
        setattr(a, k, v)
    return getattr(B.lib(), fn)(P(h), ctypes.byref(a), P(ws), ctypes.c_size_t(nbytes), None)


TABLE = dict(block_tables=FAKE, cached_lens=FAKE, new_lens=FAKE, free_pages=FAKE, taken=FAKE, kv_lens=FAKE, query_offsets=FAKE,
             slot_map=FAKE, positions=FAKE, taken_out=FAKE, stride=8, B=4, width=8, page=16, num_free=9, T=5)


@pytest.mark.parametrize("over,code", [
    (dict(h=0), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(T=2 ** 31 - 1), 1), (dict(width=-1), 1), (dict(page=0), 1),
    (dict(num_free=-1), 1), (dict(B=2 ** 16, width=2 ** 15, stride=2 ** 15), 1), (dict(stride=7), 1), (dict(taken=None), 1),
    (dict(taken_out=None), 1), (dict(query_offsets=None), 1), (dict(cached_lens=None), 1), (dict(new_lens=None), 1),
    (dict(kv_lens=None), 1), (dict(block_tables=None), 1), (dict(free_pages=None), 1), (dict(slot_map=None), 1),
    (dict(positions=None), 1), (dict(slot_map=FAKE + 2), 1), (dict(taken=FAKE + 1), 1), (dict(ws=FAKE, nbytes=3), 3),
    (dict(ws=FAKE + 2, nbytes=4), 1)])
def test_page_tables_host_checks(built_lib, over, code):
    over = dict(over)
    kw = {k: over.pop(k) for k in ("h", "ws", "nbytes") if k in over}
    assert _call("moe_lora_page_tables", TableArgs, TABLE, over, **kw) == code


WRITE = dict(k=FAKE, v=FAKE, k_cache=FAKE, v_cache=FAKE, slot_map=FAKE, k_t=64, k_h=32, v_t=64, v_h=32, kc_p=1024, kc_h=512,
             kc_t=32, vc_p=1024, vc_h=512, vc_t=32, T=3, heads=2, head_dim=32, num_pages=9, page=16)


@pytest.mark.parametrize("over,code", [
    (dict(h=0), 1), (dict(T=-1), 1), (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=513), 2), (dict(T=2 ** 31 - 1), 2),
    (dict(num_pages=-1), 1), (dict(page=0), 1), (dict(num_pages=2 ** 20, page=2 ** 11), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(slot_map=None), 1), (dict(k=FAKE + 1), 1), (dict(v_cache=FAKE + 1), 1),
    (dict(slot_map=FAKE + 2), 1), (dict(ws=FAKE, nbytes=3), 3), (dict(ws=FAKE + 2, nbytes=4), 1), (dict(T=0, k=None), 0)])
def test_cache_write_host_checks(built_lib, over, code):
    over = dict(over)
    kw = {k: over.pop(k) for k in ("h", "ws", "nbytes") if k in over}
    assert _call("moe_lora_cache_write", WriteArgs, WRITE, over, **kw) == code


ATTEND = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, block_tables=FAKE, kv_lens=FAKE, query_offsets=FAKE, out=FAKE, q_t=512, q_h=64,
              o_t=512, o_h=64, kc_p=2048, kc_h=1024, kc_t=64, vc_p=2048, vc_h=1024, vc_t=64, stride=8, T=6, B=3, q_heads=8,
              k_heads=2, head_dim=64, num_pages=9, page=16, width=8, max_query_len=4, shared_len=0, scale=0.125)


@pytest.mark.parametrize("over,code", [
    (dict(h=0), 1), (dict(T=-1), 1), (dict(B=-1), 1), (dict(q_heads=0), 1), (dict(k_heads=0), 1), (dict(k_heads=3), 1),
    (dict(head_dim=0), 1), (dict(head_dim=513), 2), (dict(num_pages=-1), 1), (dict(page=0), 1), (dict(width=-1), 1),
    (dict(max_query_len=-1), 1), (dict(shared_len=-1), 1), (dict(shared_len=129), 1), (dict(stride=7), 1),
    (dict(num_pages=2 ** 20, page=2 ** 11), 1), (dict(width=2 ** 20, page=2 ** 11, stride=2 ** 20), 1),
    (dict(query_offsets=None), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(kv_lens=None), 1), (dict(block_tables=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1),
    (dict(q=FAKE + 1), 1), (dict(out=FAKE + 1), 1), (dict(lse=FAKE + 2), 1), (dict(kv_lens=FAKE + 2), 1),
    (dict(query_offsets=FAKE + 2), 1), (dict(block_tables=FAKE + 2), 1), (dict(ws=0), 1), (dict(ws=FAKE + 8), 1),
    (dict(nbytes=4096), 3), (dict(T=2 ** 28, q_heads=8), 2), (dict(B=65536), 2), (dict(T=0, q=None), 0),
    (dict(B=0, T=4, kv_lens=None), 0)])
def test_attention_host_checks(built_lib, over, code):
    over = dict(over)
    kw = dict(h=over.pop("h", FAKE), ws=over.pop("ws", FAKE), nbytes=over.pop("nbytes", 1 << 32))
    assert _call("moe_lora_attention", AttentionArgs, ATTEND, over, **kw) == code


@pytest.mark.parametrize("over", [dict(q_t=1024), dict(q_h=128, o_t=1024, q_t=1024), dict(o_t=520)])
def test_attention_in_place_takes_its_strides(built_lib, over):
    """`out` that is q has its strides."""
    assert _call("moe_lora_attention", AttentionArgs, ATTEND, over, ws=FAKE, nbytes=1 << 32) == 1


def test_attention_workspace_never_less_for_more_rows(built_lib):
    for Hq, Hk, D in ((32, 4, 128), (7, 1, 96), (16, 16, 64), (64, 1, 128)):
        sizes = [B.moe_lora_attention_workspace_size(T, Hq, Hk, D)
                 for T in list(range(0, 300)) + [511, 512, 513, 1000, 5000, 8192, 100000]]
        assert sizes == sorted(sizes) and sizes[0] >= 256
    n = ctypes.c_size_t()
    size = B.lib().moe_lora_attention_workspace_size
    assert size(-1, 8, 2, 64, ctypes.byref(n)) == 1 and size(1, 8, 3, 64, ctypes.byref(n)) == 1
    assert size(1, 0, 1, 64, ctypes.byref(n)) == 1 and size(1, 8, 2, 0, ctypes.byref(n)) == 1 and size(1, 8, 2, 64, None) == 1


def test_python_side_refuses_cpu_tensors_and_wrong_types(built_lib):
    class H:
        address = FAKE
    z, i = torch.zeros(2, 3, 8).bfloat16(), torch.zeros(2, dtype=torch.int32)
    for bad, what in ((lambda: B.moe_lora_page_tables(H, i[None], i, i, 16, i, i[:1], 4), "block_tables"),
                      (lambda: B.moe_lora_page_tables(H, [1], i, i, 16, i, i[:1], 4), "block_tables"),
                      (lambda: B.moe_lora_cache_write(H, z, z, z, z, i), "k must"),
                      (lambda: B.moe_lora_attention(H, z, z, z, i, i), "q must")):
        with pytest.raises(ValueError, match=what):
            bad()


# ------------------------------------------------------------------------------------ the reference itself
def test_reference_tables_by_hand():
    # two requests on pages of 4: one with 3 tokens that gets 3 more, one with 4 that gets 1
    got = ref.page_tables([[7, -1, -1], [5, -1, -1]], [3, 4], [3, 1], 4, [9, 8, 6], 1, 6)
    assert got == ([[7, 8, -1], [5, 6, -1]], [6, 5], [0, 3, 4], [31, 32, 33, 24, -1, -1], [3, 4, 5, 4, 0, 0], 3)
    # the list ends: the second request's token has no page
    got = ref.page_tables([[7, -1], [5, -1]], [3, 4], [3, 1], 4, [9], 0, 4)
    assert got == ([[7, 9], [5, -1]], [6, 4], [0, 3, 4], [31, 36, 37, -1], [3, 4, 5, 4], 1)


def test_reference_attention_by_hand():
    """Two keys that a row sees with scores 0 and log 3: weights 1/4 and 3/4; a row in front sees the first alone."""
    q = torch.tensor([[[1.0, 0.0]], [[math.log(3.0), 0.0]]])
    k = torch.tensor([[[[0.0, 5.0], [1.0, -2.0]]]])
    v = torch.tensor([[[[4.0, 8.0], [0.0, 16.0]]]])
    out, lse, tol, lse_tol = ref.attention(q, k, v, [[0]], [2], [0, 2], 1.0, ref.PLAIN)
    assert torch.allclose(out, torch.tensor([[[4.0, 8.0]], [[1.0, 14.0]]], dtype=torch.float64))
    assert torch.allclose(lse, torch.tensor([[0.0], [math.log(4.0)]], dtype=torch.float64))
    assert (tol >= 0).all() and (lse_tol >= 0).all()
    # a request of no keys: zeros, and -inf
    out, lse, tol, _ = ref.attention(q, k, v, [[0]], [0], [0, 2], 1.0, ref.PLAIN)
    assert (out == 0).all() and (lse == -math.inf).all() and (tol == 0).all()
