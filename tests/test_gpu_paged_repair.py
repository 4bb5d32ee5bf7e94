"""moe_lora_attention on long requests where a value is not finite: rows that do not see it are worked out again, which
may take a while but not hundreds of times the call's time, and no wait of the kernel runs out meanwhile."""
import math

import pytest
import torch

import routed_moe_expert_gb300 as pkg
from test_gpu_paged import I32, handle, ints, status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,m,at", [(8192, 8192, 8190), (8192, 8192, 100), (8192, 8192, 4095), (30000, 40, 29990), (30000, 4, 29998)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_rows_in_front_of_a_bad_value_of_a_long_request(handle, n, m, at, bad):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(n + m)
    Hq, Hk, D, page = 32, 4, 128, 64
    pages = -(-n // page)
    q = torch.randn((m, Hq, D), generator=g, device="cuda").bfloat16()
    kc, vc = (torch.randn((pages, Hk, page, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    vc[at // page, :, at % page, 77] = bad
    ws = pkg.alloc_attention_workspace(m, Hq, Hk, D)
    args = (handle, q, kc, vc, torch.arange(pages, dtype=I32, device="cuda")[None], ints([n]), ints([0, m]), m)
    out = pkg.moe_lora_attention(*args, workspace=ws)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    out = pkg.moe_lora_attention(*args, workspace=ws)
    end.record()
    assert status(ws) == 0
    # A warp's 32 rows one after another, 32 keys a step: table, scores and values are five reads from the L2 in turn, about a
    # microsecond each, and the scores' reads take 16 x 32 lines of eight warps through the first-level cache, 4096 cycles or
    # 2 us: n / 32 steps of 32 rows, 7 us each, and twice that.
    assert start.elapsed_time(end) < 2 * n * 7e-3
    k, v = (t.transpose(1, 2).reshape(-1, Hk, D)[:n].double() for t in (kc, vc))
    first = n - m                                     # the key of the first row
    rows = sorted({0, max(0, at - first - 40), *range(max(0, at - first - 6), min(m, at - first + 6)), m - 1})
    for i in rows:
        sees = first + i + 1
        x = torch.einsum("hgd,nhd->hgn", q[i].double().view(Hk, Hq // Hk, D), k[:sees]) / math.sqrt(D)
        p = x.softmax(2)
        want = torch.einsum("hgn,nhd->hgd", p, v[:sees]).reshape(Hq, D)
        size = torch.einsum("hgn,nhd->hgd", p, v[:sees].abs()).reshape(Hq, D)
        finite = torch.isfinite(want)
        assert finite.all() == (sees <= at)
        assert torch.equal(torch.isfinite(out[i]), finite)
        off = (out[i].double() - want).abs()
        assert (off <= 2.0 ** -8 * want.abs() + 1.01 * (2.0 ** -8 + 2.0 ** -10) * size)[finite].all()
