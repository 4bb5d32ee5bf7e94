"""moe_lora_attention on batches with rows of no request, as a captured step pads them, and rows that see nothing, beside
keys that all requests share."""
import math

import pytest
import torch

import routed_moe_expert_gb300 as pkg
from test_gpu_paged import I32, _attention, handle, ints, status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (4, 2, 64)])
@pytest.mark.parametrize("behind", [5, 300])
def test_padding_beside_shared_keys(handle, Hq, Hk, D, behind):  # noqa: F811
    lens = [(256 + 9 * i, i % 3) for i in range(7)] + [(0, 4), (1, 3), (200, 2)]
    _attention(handle, lens, Hq, Hk, D, 16, seed=behind, shared=256, behind=behind, front=behind // 2)
    _attention(handle, [(3, 40), (300, 1), (0, 9)], Hq, Hk, D, 16, seed=behind, behind=behind)


def _graph_us(call):
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            call()
    best = math.inf
    for _ in range(8):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        graph.replay()
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) * 100)
    return best


def test_padding_costs_no_more_than_requests(handle):  # noqa: F811
    """128 requests and as many rows of padding on 8192 shared keys: no more than 256 requests take."""
    shared, B, Hq, Hk, D, page = 8192, 256, 32, 4, 128, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    pages = shared // page
    q = torch.randn((B, Hq, D), generator=g, device="cuda").bfloat16()
    kc, vc = (torch.randn((pages + B, Hk, page, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    own = pages + torch.arange(B, device="cuda", dtype=I32)[:, None]
    table = torch.cat([torch.arange(pages, device="cuda", dtype=I32).expand(B, -1), own], 1).contiguous()
    lens, offsets = ints([shared + 1 + i % page for i in range(B)]), ints(list(range(B + 1)))
    ws = pkg.alloc_attention_workspace(B, Hq, Hk, D)
    out = torch.empty_like(q)

    def us(n):
        return _graph_us(lambda: pkg.moe_lora_attention(handle, q, kc, vc, table[:n], lens[:n], offsets[:n + 1], 1, shared_len=shared,
                                                        out=out, workspace=ws))

    padded, full = us(B // 2), us(B)
    assert status(ws) == 0
    assert padded <= 1.1 * full, (padded, full)
