"""moe_lora_linear with infinities and NaN among the adapters: they reach the tokens of their own slot,
as the formula says, and no other token, whichever tokens share a tile."""
import math

import numpy as np
import pytest
import torch

import block_reference as ref
import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# token counts and widths of the three kernels: clusters, narrow tiles, CTA pairs (whole and sliced
# shrinks, two pairs per tile, several tiles per pair), stacks with and without spare columns
SHAPES = [(2, 136, 128, (8, 16)), (24, 200, 520, (64,)), (24, 200, 520, (64, 48)), (32, 4096, 2048, (64, 64)),
          (100, 264, 512, (8, 16, 64, 40)), (128, 384, 1024, (16,) * 12), (300, 8000, 512, (16, 40)),
          (512, 2048, 2048, (16, 5)), (777, 1536, 2048, (16, 48)), (1281, 384, 4104, (64, 64, 64)),
          (2500, 2050, 136, (16, 40, 64, 5)), (5000, 1792, 264, (40, 24))]


@pytest.fixture(scope="module")
def handle():
    return pkg.Handle(0)


def _case(T, N, K, ranks, seed):
    g = torch.Generator().manual_seed(seed)
    S, R = len(ranks), max(ranks) + 2
    r = lambda shape, std: (torch.randn(shape, generator=g) * std).bfloat16()
    c = dict(x=r((T, K), 1.0), w=r((N, K), 1 / math.sqrt(K)), A=r((S, R, K), 1 / math.sqrt(K)), B=r((S, N, R), 0.3),
             ranks=list(ranks), scalings=[[2.0, 0.5, 1.0, -0.25][s % 4] for s in range(S)],
             slots=((torch.arange(T) * 7) % (S + 1) - 1).to(torch.int32))
    return c


def _run(handle, c, f32):
    ad = pkg.moe_lora_linear_adapters(handle, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
    ws = pkg.alloc_linear_workspace(c["x"].shape[0], ad)
    ws.fill_(255)
    y = pkg.moe_lora_linear(handle, c["x"].cuda(), c["w"].cuda(), ad, c["slots"].cuda(),
                            out_dtype=torch.float32 if f32 else torch.bfloat16, workspace=ws)
    assert pkg.moe_lora_check_status(ws)[0] == 0
    return ref.f64(y)


def _finite_part(c, f32):
    """The 64-bit result and bound with 0 in the place of what is not finite."""
    B = torch.where(torch.isfinite(c["B"]), c["B"], torch.zeros_like(c["B"]))
    A = torch.where(torch.isfinite(c["A"]), c["A"], torch.zeros_like(c["A"]))
    return ref.linear(c["x"], c["w"], None, A, B, c["slots"].numpy(), c["ranks"], c["scalings"], f32)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K,ranks", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_nonfinite_b_stays_with_its_slot(handle, T, N, K, ranks, f32):
    c = _case(T, N, K, ranks, N + T)
    S = len(ranks)
    # one value of a row, so that the sign of its infinity is the sign of one product
    at = {}
    for s in range(S):
        for i, v in enumerate((INF, -INF, NAN)):
            n = (37 * s + 11 * i + 5) % N
            if (s, n) not in at:
                at[s, n] = (5 * i + s) % ranks[s], v
                c["B"][s, n, at[s, n][0]] = v
    got = _run(handle, c, f32)
    y, tol = _finite_part(c, f32)
    sl, x = c["slots"].numpy(), ref.f64(c["x"])
    own = np.zeros_like(y, dtype=bool)
    for (s, n), (r, v) in at.items():
        rows = np.nonzero(sl == s)[0]
        own[rows, n] = True
        u = c["scalings"][s] * (x[rows] @ ref.f64(c["A"][s, r]))
        sure = np.abs(u) > 1e-3 * np.abs(u).max() if rows.size else u > 0     # whose sign no rounding turns
        g = got[rows, n]
        assert (np.isnan(g[sure]) if math.isnan(v) else g[sure] == np.sign(u[sure]) * v).all(), (s, n, v)
        assert not np.isfinite(g).any()
    bad = ~(np.abs(got - y) <= tol) & ~own
    assert not bad.any(), f"{bad.sum()} values of other tokens or rows are off, first at {np.argwhere(bad)[:4].tolist()}"


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K,ranks", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_a_slot_switched_off_and_never_filled_adds_nothing(handle, T, N, K, ranks, f32):
    """Factor 0 with NaN in all of the slot's memory: its own tokens take the projection alone."""
    c = _case(T, N, K, ranks, N + T)
    off = len(ranks) - 1
    c["scalings"][off] = 0.0
    c["A"][off] = NAN
    c["B"][off] = NAN
    got = _run(handle, c, f32)
    y, tol = _finite_part(c, f32)
    assert (np.abs(got - y) <= tol).all()


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K,ranks", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_many_nonfinite_values_of_one_slot(handle, T, N, K, ranks, f32):
    """A slot of NaN alone, in A and in B: its tokens are NaN, the others' values are what they are
    without that slot's weights."""
    c = _case(T, N, K, ranks, N + T)
    c["A"][0] = NAN
    c["B"][0] = NAN
    got = _run(handle, c, f32)
    y, tol = _finite_part(c, f32)
    own = c["slots"].numpy() == 0
    assert np.isnan(got[own]).all()
    assert (np.abs(got - y) <= tol)[~own].all()


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K", [(3, 136, 128), (100, 264, 512), (777, 1536, 2048), (2500, 2050, 136), (512, 2048, 2048)])
def test_an_infinite_shrunk_value_keeps_its_sign(handle, T, N, K, f32):
    """One rank whose A holds an infinity: u is +-infinite, and so is every value of the token's row, by
    the sign of u and of B; nothing is subtracted from an infinity on the way."""
    c = _case(T, N, K, (1, 8), T)
    c["A"][0, 0, 3] = INF
    got = _run(handle, c, f32)
    y, tol = _finite_part(c, f32)
    own = c["slots"].numpy() == 0
    sign = np.sign(c["scalings"][0] * ref.f64(c["x"])[own, 3])[:, None] * np.sign(ref.f64(c["B"][0, :, 0]))[None]
    assert (got[own] == sign * INF)[sign != 0].all()
    assert (np.abs(got - y) <= tol)[~own].all()


@pytest.mark.parametrize("T,N,K", [(3, 136, 128), (100, 264, 512), (777, 1536, 2048), (2500, 2050, 136)])
def test_a_shrunk_value_past_the_largest_bf16_stays_finite_in_float32(handle, T, N, K):
    """u = 3.4e38 is a float32, but rounds to an infinite bf16; times 2^-40 it is 3.1e26."""
    c = _case(T, N, K, (1, 8), T)
    c["A"][0] = 0.0
    c["A"][0, 0, 3] = 1.0
    c["x"][:, 3] = 1.0
    c["B"][0] = 2.0 ** -40
    c["scalings"][0] = 3.4e38
    got = _run(handle, c, True)
    own = c["slots"].numpy() == 0
    # u is a product of exact values rounded once to 24 bits, in pieces that lose nothing; then one sum
    np.testing.assert_allclose(got[own], float(np.float32(3.4e38)) * 2.0 ** -40, rtol=2.0 ** -22)


@pytest.mark.parametrize("ranks", [(16, 8), (64,), (64, 64), (40, 0, 16)], ids=str)
def test_a_stack_is_the_same_whatever_its_memory_held(handle, ranks):
    """Every byte of it is written, spare columns and marks among them."""
    import ctypes
    S, N, K, R = len(ranks), 256, 256, max(ranks)     # (sizes without a gap between the parts)
    g = torch.Generator(device="cuda").manual_seed(1)
    A, B = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((S, R, K), (S, N, R)))
    r, n = (ctypes.c_int32 * S)(*ranks), ctypes.c_size_t()
    L = pkg.lib()
    assert L.moe_lora_linear_adapters_size(S, N, K, r, ctypes.byref(n)) == 0
    stacks = []
    for fill in (0, 255):
        t = torch.full((n.value,), fill, dtype=torch.uint8, device="cuda")
        assert L.moe_lora_linear_pack_adapters(handle.ptr, A.data_ptr(), B.data_ptr(), S, N, K, R, r, t.data_ptr(),
                                               torch.cuda.current_stream().cuda_stream) == 0
        stacks.append(t if sum(ranks) % 64 else t[:n.value - 240])    # (the last word's 256 bytes hold 16)
    assert torch.equal(*stacks)
