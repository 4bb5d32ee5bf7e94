"""moe_lora_attention with a workspace that starts on any 16-byte boundary, as one cut out of a larger buffer does."""
import pytest
import torch

import routed_moe_expert_gb300 as pkg
from test_gpu_paged import I32, handle, ints, status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (4, 2, 64), (6, 2, 96)])
@pytest.mark.parametrize("m,shared", [(1, 0), (40, 0), (300, 0), (1, 1024), (30, 1024), (200, 1040)])
def test_workspace_on_any_boundary(handle, Hq, Hk, D, m, shared):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(m + D)
    lens = [2000, 1100 + m, 3900, 1400]
    T, pages, width = m * len(lens), 700, 250
    q = torch.randn((T, Hq, D), generator=g, device="cuda").bfloat16()
    kc, vc = (torch.randn((pages, Hk, 16, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randint(0, pages, (len(lens), width), generator=g, device="cuda").to(I32)
    table[:, :shared // 16] = table[0, :shared // 16]
    offsets = ints([m * i for i in range(len(lens) + 1)])
    size = pkg.moe_lora_attention_workspace_size(T, Hq, Hk, D)
    room = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    start = -room.data_ptr() % 64
    outs = []
    for off in (0, 16, 32, 48):
        room.fill_(255)
        ws = room[start + off:start + off + size]
        assert ws.data_ptr() % 64 == off
        outs.append(pkg.moe_lora_attention(handle, q, kc, vc, table, ints(lens), offsets, m, shared_len=shared, return_lse=True,
                                           workspace=ws))
        assert status(ws) == 0
        assert (room[:start + off] == 255).all() and (room[start + off + size:] == 255).all()
    for o, e in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(e, outs[0][1])
