"""moe_lora_page_tables where a request's length would pass 32 bits."""
import pytest
import torch

import routed_moe_expert_gb300 as pkg
from test_gpu_paged import I32, handle, ints, status  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("cached,new,kv,code", [(MOST, 5, MOST, 6), (MOST - 3, 5, MOST, 6), (MOST - 5, 5, MOST, 0), (MOST, 0, MOST, 0)])
def test_lengths_stay_in_32_bits(handle, cached, new, kv, code):  # noqa: F811
    page, width = 64, 2 ** 25 + 2          # tables of 134 MB, room for 2^31 + 128 tokens
    table = torch.zeros((2, width), dtype=I32, device="cuda")
    ws = pkg.alloc_cache_workspace()
    o = pkg.moe_lora_page_tables(handle, table, ints([cached, 3]), ints([new, 1]), page, ints([5, 6, 7]), ints([0]), new + 1, workspace=ws)
    assert status(ws) == code
    assert o["kv_lens"].tolist() == [kv, 4]
    assert o["query_offsets"].tolist() == [0, new, new + 1]
    positions = o["positions"].tolist()
    assert positions[-1] == 3 and positions[:-1] == [min(cached + i, MOST) for i in range(new)]
    assert o["slot_map"].tolist()[-1] == 3
