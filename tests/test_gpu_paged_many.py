"""moe_lora_attention on batches of hundreds of requests, whose plans take other ways than few requests' do, caches past
2^31 values, pages that are named twice, offsets out of order, calls side by side, and workspaces that graphs share."""
import math
import random

import pytest
import torch

import paged_reference as ref
import routed_moe_expert_gb300 as pkg
from test_gpu_paged import I32, _attention, handle, ints, status  # noqa: F401

pytestmark = pytest.mark.gpu


def _lens(B, most_keys, most_rows, seed, long=()):
    """Ragged requests, some without rows, some without keys; `long` in the middle."""
    r = random.Random(seed)
    lens = []
    for _ in range(B):
        m = r.choice([0, 1, 1, r.randint(1, most_rows)])
        lens.append((r.choice([0, m, m, m + r.randint(0, most_keys - most_rows)]), m))
    lens[B // 2:B // 2 + len(long)] = long
    return lens


@pytest.mark.parametrize("B", [31, 32, 33, 160, 256, 257, 321, 700])
@pytest.mark.parametrize("most", [200, 900])      # tables of up to 512 keys, and longer ones
def test_single_tokens_of_many_requests(handle, B, most):  # noqa: F811
    r = random.Random(B)
    lens = [(r.choice([0, 1, 16, 64, 65, r.randint(0, most // 8), r.randint(0, most // 8)]), 1) for _ in range(B)]
    lens[B // 3] = (most, 1)
    lens[B - 1] = (most - 7, 1)
    _attention(handle, lens, 4, 2, 64, 16, seed=B, one=True, behind=0)


@pytest.mark.parametrize("B,long", [(33, ()), (257, ()), (400, ()), (900, ()), (33, [(300, 270)]), (40, [(700, 300), (280, 280)]),
                                    (400, [(300, 300)]), (800, [(257, 257), (1, 1), (600, 260)])])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 64), (2, 2, 128)])
def test_ragged_batches_of_many_requests(handle, B, long, Hq, Hk, D):  # noqa: F811
    _attention(handle, _lens(B, 150, 9, B, long), Hq, Hk, D, 16, seed=B + Hq, front=1)


@pytest.mark.parametrize("B,rows", [(33, 3), (300, 3), (300, 1)])
def test_shared_keys_of_many_requests(handle, B, rows):  # noqa: F811
    r = random.Random(B)
    lens = [(256 + r.randint(rows, 90), r.randint(0, rows)) for _ in range(B)]
    _attention(handle, lens, 8, 2, 64, 32, seed=B, shared=256)


@pytest.mark.parametrize("B,long", [(200, 40), (300, 300)])
def test_shared_keys_of_many_requests_beside_a_long_one(handle, B, long):  # noqa: F811
    r = random.Random(B)
    lens = [(256 + r.randint(1, 60), r.randint(0, 1)) for _ in range(B)]
    lens[7] = (256 + long + 9, long)
    _attention(handle, lens, 8, 2, 64, 32, seed=B, shared=256)


@pytest.mark.parametrize("lens", [[(1024, 1024)], [(1280, 1280)], [(1281, 700)], [(700, 400)] * 3, [(1100, 130)] * 5 + [(0, 0)] * 30])
@pytest.mark.parametrize("wide", [0, 70])
def test_whole_items_by_length(handle, lens, wide):  # noqa: F811
    """Prompts about the length up to which items are not cut, in tables as long as they are, and longer ones."""
    _attention(handle, lens + [(wide * 32, 0)], 16, 8, 64, 32, seed=wide)


def test_pages_named_twice(handle):  # noqa: F811
    """Requests that share pages without saying so, and one whose table names a page again and again."""
    g = torch.Generator().manual_seed(8)
    for m, Hq in ((1, 4), (20, 8)):
        kc, vc = (torch.randn((6, 2, 16, 64), generator=g).bfloat16() for _ in range(2))
        q = torch.randn((3 * m, Hq, 64), generator=g).bfloat16()
        tables, lens, offsets = [[1, 1, 1, 1], [1, 2, 2, 1], [5, 2, 0, 1]], [60, 64, 50], [0, m, 2 * m, 3 * m]
        out = pkg.moe_lora_attention(handle, q.cuda(), kc.cuda(), vc.cuda(), ints(tables), ints(lens), ints(offsets), m)
        want, _, tol, _ = ref.attention(q, kc, vc, tables, lens, offsets, 0.125, ref.TILES)
        assert ((out.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("Hq,m,page,D", [(8, 1, 16, 128), (16, 33, 16, 128), (8, 2, 12, 128)])
def test_cache_past_32_bits(handle, Hq, m, page, D):  # noqa: F811
    """Pages whose values lie more than 2^31 values into the cache, written and read."""
    Hk = 8
    pages = (2 ** 31 // (Hk * page * D)) + 12
    kc, vc = (torch.empty((pages, Hk, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(m)
    n, used = 100, -(-100 // page)
    table = [pages - 1 - i if i % 2 == 0 else i for i in range(used)]
    k, v = (torch.randn((n, Hk, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    slots = ints([table[i // page] * page + i % page for i in range(n)])
    pkg.moe_lora_cache_write(handle, k, v, kc, vc, slots)
    at, place = torch.tensor(table, device="cuda")[torch.arange(n) // page], torch.arange(n, device="cuda") % page
    assert torch.equal(kc[at, :, place], k) and torch.equal(vc[at, :, place], v)
    q = torch.randn((m, Hq, D), generator=g, device="cuda").bfloat16()
    ws = pkg.alloc_attention_workspace(m, Hq, Hk, D)
    out = pkg.moe_lora_attention(handle, q, kc, vc, ints([table]), ints([n]), ints([0, m]), m, workspace=ws)
    assert status(ws) == 0
    small = [t[torch.tensor(table, device="cuda")].cpu() for t in (kc, vc)]
    want, _, tol, _ = ref.attention(q, *small, [list(range(used))], [n], [0, m], D ** -0.5, ref.TILES)
    assert ((out.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("B", [6, 33, 2048])
@pytest.mark.parametrize("ask", [1, 4096])
def test_offsets_out_of_order_are_reported(handle, B, ask):  # noqa: F811
    """Every other request claims all rows: the weights of what they would have to do pass 32 bits at the largest."""
    T, width, page = 4096, 8192, 256
    q = torch.randn((T, 16, 64), device="cuda").bfloat16()
    kc = torch.randn((3, 1, page, 64), device="cuda").bfloat16()
    offsets = ints([T * (i & 1) for i in range(B + 1)])
    table = torch.zeros((B, width), dtype=I32, device="cuda")
    ws = pkg.alloc_attention_workspace(T, 16, 1, 64)
    pkg.moe_lora_attention(handle, q, kc, kc, table, torch.full((B,), width * page, dtype=I32, device="cuda"), offsets, ask, workspace=ws)
    assert status(ws) == 6
    # the next call of the handle and workspace is as any
    a = pkg.moe_lora_attention(handle, q[:2], kc, kc, table[:2], ints([70, 3]), workspace=ws)
    assert status(ws) == 0
    assert torch.equal(a, pkg.moe_lora_attention(handle, q[:2], kc, kc, table[:2], ints([70, 3])))


def _call(h, g, m, B, ws=None, out=None):
    kc, vc = (torch.randn((200, 2, 16, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B * m, 8, 128), generator=g, device="cuda").bfloat16()
    table = torch.randint(0, 200, (B, 90), generator=g, device="cuda").to(I32)
    lens = ints([m + 37 * i % 1400 for i in range(B)])
    offsets = ints([m * i for i in range(B + 1)])
    return lambda **kw: pkg.moe_lora_attention(h, q, kc, vc, table, lens, offsets, m, **kw)


def test_two_handles_side_by_side():
    """Calls of two handles on two streams, over and over, give what each gives alone."""
    g = torch.Generator(device="cuda").manual_seed(2)
    handles, streams = [pkg.Handle(0) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    calls = [_call(h, g, m, B) for h, (m, B) in zip(handles, ((1, 40), (50, 9)))]
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])
    for h in handles:
        h.close()


def test_two_graphs_of_one_workspace(handle):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(6)
    ws = pkg.alloc_attention_workspace(400, 8, 2, 128)
    calls = [_call(handle, g, m, B) for m, B in ((1, 33), (40, 10), (3, 5))]
    alone = [c() for c in calls]
    outs = [torch.empty_like(a) for a in alone]
    graphs = []
    for c, o in zip(calls, outs):
        c(out=o, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            c(out=o, workspace=ws)
        graphs.append(graph)
    for order in ((0, 1, 2), (2, 0, 1), (1, 1, 0, 2)):
        for o in outs:
            o.fill_(math.nan)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert status(ws) == 0 and all(torch.equal(o, a) for o, a in zip(outs, alone))
