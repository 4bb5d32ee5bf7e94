"""moe_lora_attention with its result over the queries where a value that some rows do not see is not finite: those rows
are worked out again from their queries, which are to be there still."""
import math

import pytest
import torch

import paged_reference as ref
import routed_moe_expert_gb300 as pkg
from test_gpu_paged import I32, handle, ints, status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk,D", [(4, 2, 64), (4, 2, 128), (8, 1, 96)])
@pytest.mark.parametrize("m", [2, 4, 10, 16, 20, 40, 64, 100, 150])
@pytest.mark.parametrize("cols", [(3,), (-2,), (3, -2)])       # of the lower half, the upper, and both
def test_spoilt_rows_in_place(handle, Hq, Hk, D, m, cols):  # noqa: F811
    g = torch.Generator().manual_seed(m + D)
    n = 290 + m
    q = torch.randn((m, Hq, D), generator=g).bfloat16()
    kc, vc = (torch.randn((40, Hk, 16, D), generator=g).bfloat16() for _ in range(2))
    table = torch.randperm(40, generator=g).tolist()[:32]
    for at, bad in ((n - m // 2, math.inf), (n - 1, math.nan)):   # the rows in front of these keys do not see them
        for c in cols:
            vc[table[at // 16], :, at % 16, c] = bad
    want, want_lse, tol, lse_tol = ref.attention(q, kc, vc, [table], [n], [0, m], D ** -0.5, ref.TILES)
    kc, vc, tables, lens, offsets = kc.cuda(), vc.cuda(), ints([table]), ints([n]), ints([0, m])
    ws = pkg.alloc_attention_workspace(m, Hq, Hk, D)
    finite = torch.isfinite(want)
    assert 0 < (~finite).sum() < finite.numel() // 2
    for _ in range(20):
        got = q.cuda()
        lse = torch.empty((m, Hq), device="cuda")
        assert pkg.moe_lora_attention(handle, got, kc, vc, tables, lens, offsets, m, out=got, lse=lse, workspace=ws)[0] is got
        assert status(ws) == 0
        o = got.double().cpu()
        assert torch.equal(torch.isfinite(o), finite)
        assert ((o - want).abs()[finite] <= tol[finite]).all()
        assert ((lse.double().cpu() - want_lse).abs() <= lse_tol).all()
