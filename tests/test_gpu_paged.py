"""moe_lora_page_tables, moe_lora_cache_write and moe_lora_attention against their definitions in 64 bits:
lengths of zero and one, odd sizes, strides, rows that see nothing, pages that end anywhere, garbage behind
them, shared prefixes, streams, graphs, and the run of them together."""
import math
import random

import pytest
import torch

import paged_reference as ref
import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu
I32 = torch.int32
NAN = float("nan")


@pytest.fixture(scope="module")
def handle():
    return pkg.Handle(0)


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def status(ws):
    return pkg.moe_lora_check_status(ws)[0]


# ------------------------------------------------------------------------------------ page tables
def _batch(B, page, width, seed, empty=0.1):
    r = random.Random(seed)
    cached, new = [], []
    for _ in range(B):
        c = r.choice([0, 1, page - 1, page, page + 1, r.randint(0, width * page // 2)])
        n = 0 if r.random() < empty else r.choice([1, 1, 2, page, r.randint(1, width * page - c)])
        cached.append(c)
        new.append(min(n, width * page - c))
    ids = list(range(10000))
    r.shuffle(ids)
    held = [-(-c // page) for c in cached]
    tables, at = [], 0
    for h in held:
        tables.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    return cached, new, tables, ids[at:at + B * width + 5]


def _check_tables(handle, cached, new, tables, free, page, taken, T, code=0, strided=False, alias=False, stream=None):
    want = ref.page_tables(tables, cached, new, page, free, taken, T)
    B, width = len(cached), len(tables[0]) if tables else 3
    wide = torch.full((max(B, 1), width + (3 if strided else 0)), 77, dtype=I32, device="cuda")[:B]
    table = wide[:, :width]
    if B:
        table.copy_(ints(tables))
    ws = pkg.alloc_cache_workspace()
    ws.fill_(255)
    lens, cursor = ints(cached), ints([taken])
    given = {"kv_lens": lens, "taken": cursor} if alias else None
    o = pkg.moe_lora_page_tables(handle, table, lens, ints(new), page, ints(free), cursor, T, outputs=given, workspace=ws)
    assert status(ws) == code
    assert table.tolist() == want[0]
    assert o["kv_lens"].tolist() == want[1] and o["query_offsets"].tolist() == want[2]
    assert o["slot_map"].tolist() == want[3] and o["positions"].tolist() == want[4]
    assert o["taken"].tolist() == [want[5]]
    if strided and B:
        assert (wide[:, width:] == 77).all()
    if alias:
        assert o["kv_lens"] is lens and o["taken"] is cursor
    return o


@pytest.mark.parametrize("B,page,width", [(1, 16, 4), (3, 1, 9), (64, 16, 12), (129, 7, 5), (1000, 16, 3), (1025, 32, 3),
                                          (2500, 16, 2)])
@pytest.mark.parametrize("alias", [False, True])
def test_page_tables(handle, B, page, width, alias):
    cached, new, tables, free = _batch(B, page, width, B + page)
    pad = 0 if alias else 13
    _check_tables(handle, cached, new, tables, free, page, 5, sum(new) + pad, strided=True, alias=alias)


def test_page_tables_long_prompts_and_none(handle):
    _check_tables(handle, [0, 5000, 0], [20011, 0, 3], [[-1] * 200, list(range(40)) + [-1] * 160, [-1] * 200],
                  list(range(100, 400)), 128, 0, 20020)
    _check_tables(handle, [0, 7], [0, 0], [[-1] * 2, [3, -1]], [9], 16, 1, 0)     # nothing new at all
    _check_tables(handle, [], [], [], [1, 2], 16, 1, 5)                          # no request


@pytest.mark.parametrize("cached,new,width,free,taken,T", [
    ([10, 20, 3], [40, 40, 1], 8, 3, 0, 100),        # the free list ends within a request
    ([10, 20, 3], [40, 40, 1], 8, 4, 4, 100),        # it has ended
    ([10, 20], [40, 400], 4, 50, 0, 500),            # a table is too narrow
    ([100, 1], [1, 1], 4, 50, 0, 2),                 # also for what is cached
    ([-5, 20], [3, -7], 4, 50, 0, 20),               # negative lengths count as 0
    ([10, 20, 3], [40, 40, 1], 8, 50, 0, 50)])       # more tokens than rows
def test_page_tables_reports_what_does_not_fit(handle, cached, new, width, free, taken, T):
    tables = [[100 + 10 * b + i if i < -(-max(c, 0) // 16) else -1 for i in range(width)] for b, c in enumerate(cached)]
    _check_tables(handle, cached, new, tables, list(range(free)), 16, taken, T, code=6)


def test_page_tables_cursor_outside_the_list(handle):
    ws = pkg.alloc_cache_workspace()
    for taken in (-1, 4):
        table = ints([[-1, -1]])
        o = pkg.moe_lora_page_tables(handle, table, ints([0]), ints([3]), 16, ints([7, 8, 9]), ints([taken]), 3, workspace=ws)
        assert status(ws) == 6
        assert o["slot_map"].tolist() == ([112, 113, 114] if taken < 0 else [-1, -1, -1])


# ------------------------------------------------------------------------------------ cache write


def _cuda_view(t, layout, D):
    """The same values on the GPU with the layout's strides."""
    if layout == "heads":
        return t.cuda()
    if layout == "tokens":
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    wide = torch.full((*t.shape[:3], 2 * D + 8), NAN, dtype=t.dtype, device="cuda")
    wide[..., D:2 * D] = t.cuda()
    return wide[..., D:2 * D]


@pytest.mark.parametrize("T,H,D,page", [(0, 2, 64, 16), (1, 4, 128, 16), (5, 1, 1, 3), (33, 3, 72, 16), (257, 8, 96, 32),
                                        (1000, 2, 36, 7), (9000, 4, 128, 64)])
@pytest.mark.parametrize("layout", ["heads", "tokens", "apart"])
def test_cache_write(handle, T, H, D, page, layout):
    g = torch.Generator().manual_seed(T + D)
    pages = 2 * T // page + 3
    kc, vc = (torch.randn((pages, H, page, D), generator=g).bfloat16() for _ in range(2))
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.2] = -1
    rows = torch.randn((T, 3 * H * D + 8), generator=g).bfloat16()
    k, v = rows[:, 8:8 + H * D].view(T, H, D), rows[:, 8 + 2 * H * D:].view(T, H, D)
    gk, gv = _cuda_view(kc, layout, D), _cuda_view(vc, layout, D)
    grows = rows.cuda()
    ws = pkg.alloc_cache_workspace()
    pkg.moe_lora_cache_write(handle, grows[:, 8:8 + H * D].view(T, H, D), grows[:, 8 + 2 * H * D:].view(T, H, D), gk, gv,
                             slots.to(I32).cuda(), workspace=ws)
    assert status(ws) == 0
    at = slots[slots >= 0]
    for c, x, got in ((kc, k, gk), (vc, v, gv)):
        c[at // page, :, at % page] = x[slots >= 0]
        assert torch.equal(c.view(torch.int16), got.cpu().contiguous().view(torch.int16))


def test_cache_write_past_the_cache_and_not_finite(handle):
    k = torch.full((3, 2, 64), float("inf"), device="cuda").bfloat16()
    k[1] = NAN
    kc, vc = (torch.zeros((2, 2, 16, 64), device="cuda").bfloat16() for _ in range(2))
    ws = pkg.alloc_cache_workspace()
    pkg.moe_lora_cache_write(handle, k, k, kc, vc, ints([31, 32, 2 ** 31 - 1]), workspace=ws)
    assert status(ws) == 6
    assert torch.isinf(kc[1, :, 15]).all() and (kc == 0).sum() == kc.numel() - 128 and torch.equal(kc, vc)


# ------------------------------------------------------------------------------------ attention
def _attention(handle, lens, Hq, Hk, D, page, seed=0, layout="heads", shared=0, garbage=True, behind=3, front=0, one=False,
               big=1.0, ask=None, scale=None, stream=None, tamper=None, weights=None):
    """A batch [(keys, query rows)] run and held to its bounds; returns (out, lse)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    width = max([-(-n // page) for n, _ in lens] + [1]) + 1
    pages = sum(-(-n // page) for n, _ in lens) + 3
    order = torch.randperm(pages, generator=g).tolist()
    kc, vc = (torch.randn((pages, Hk, page, D), generator=g).bfloat16() for _ in range(2))
    tables, at = [], shared // page
    for n, _ in lens:
        need = max(-(-n // page), 0)
        mine = min(shared // page, need)
        tables.append(order[:mine] + order[at:at + need - mine] + [-1] * (width - need))
        at += need - mine
    offsets = [front]
    for _, n in lens:
        offsets.append(offsets[-1] + n)
    T = offsets[-1] + behind
    q = (torch.randn((T, Hq, D), generator=g) * big).bfloat16()
    if garbage:   # whatever no request's keys occupy
        used = torch.zeros((pages, page), dtype=torch.bool)
        for row, (n, _) in zip(tables, lens):
            for i in range(n):
                used[row[i // page], i % page] = True
        gone = (~used)[:, None, :, None].expand_as(kc)
        kc[gone], vc[gone] = NAN, float("inf")
    if tamper:
        tamper(q, kc, vc, tables)
    gkc, gvc = _cuda_view(kc, layout, D), _cuda_view(vc, layout, D)
    rows = torch.full((T, Hq * D + (8 if layout == "apart" else 0)), NAN).bfloat16()
    rows[:, :Hq * D] = q.view(T, Hq * D)
    gq = rows.cuda()[:, :Hq * D].view(T, Hq, D)
    out = torch.full((T, Hq, D), 7.0, device="cuda").bfloat16()
    lse = torch.full((T, Hq), 7.0, device="cuda")
    ws = pkg.alloc_attention_workspace(T, Hq, Hk, D)
    ws.fill_(255)
    longest = max([n for _, n in lens] + [0])
    gt = ints(tables).view(B, width)
    got = pkg.moe_lora_attention(handle, gq, gkc, gvc, gt, ints([n for n, _ in lens]),
                                 query_offsets=None if one else ints(offsets), max_query_len=longest if ask is None else ask,
                                 scale=scale, shared_len=shared, out=out, lse=lse, workspace=ws, stream=stream)
    assert got[0] is out and got[1] is lse
    torch.cuda.synchronize()
    assert status(ws) == 0
    if weights is None:
        fast = D % 8 == 0 and D <= 128 and page >= 16 and page & (page - 1) == 0
        m = longest if ask is None else ask
        weights = ref.PLAIN if not fast else ref.TILES if Hq // Hk * m > 16 or shared else ref.FEW
    want, want_lse, tol, lse_tol = ref.attention(q, kc, vc, tables, [n for n, _ in lens], offsets,
                                                 D ** -0.5 if scale is None else scale, weights)
    o, e = out.double().cpu(), lse.double().cpu()
    free = torch.isnan(want_lse) & torch.isnan(tol[..., 0]) & torch.isnan(lse_tol)
    rowless = torch.ones(T, dtype=torch.bool)
    rowless[offsets[0]:offsets[-1]] = False
    assert free[rowless].all()
    assert (o[rowless] == 7.0).all() and (e[rowless] == 7.0).all()      # rows of no request
    o, e, want, want_lse, tol, lse_tol = (t[~rowless] for t in (o, e, want, want_lse, tol, lse_tol))
    empty = want_lse == -math.inf
    assert (o[empty] == 0).all() and (e[empty] == -math.inf).all()
    nan = ~torch.isfinite(want)   # (infinite or NaN, whatever comes of a value that is not finite)
    assert torch.equal(nan, ~torch.isfinite(o))
    off = (o - want).abs()[~nan] - tol[~nan]
    assert off.numel() == 0 or off.max() <= 0, f"{off.max():.3g} past the bound, {(off > 0).sum()} values"
    ok = ~empty & ~torch.isnan(want_lse)
    off = (e - want_lse).abs()[ok] - lse_tol[ok]
    assert off.numel() == 0 or off.max() <= 0, f"lse {off.max():.3g} past the bound"
    return out, lse


HEADS = [(8, 1, 128), (4, 4, 64), (7, 1, 128), (6, 2, 96), (3, 1, 80), (5, 5, 8), (24, 1, 128), (32, 4, 64)]


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("page,layout", [(16, "heads"), (64, "tokens"), (256, "heads"), (32, "apart")])
def test_attention_single_tokens(handle, Hq, Hk, D, page, layout):
    lens = [(n, 1) for n in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 300, 511, 700)]
    _attention(handle, lens, Hq, Hk, D, page, seed=D, layout=layout, one=True, behind=0)


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("page,layout", [(16, "tokens"), (128, "heads"), (64, "apart")])
def test_attention_ragged_batches(handle, Hq, Hk, D, page, layout):
    lens = [(200, 200), (5, 1), (0, 0), (333, 17), (64, 64), (0, 3), (128, 130), (129, 1), (400, 2), (1, 1)]
    _attention(handle, lens, Hq, Hk, D, page, seed=D + 1, layout=layout, front=2)


@pytest.mark.parametrize("n,m", [(1, 1), (130, 130), (255, 3), (256, 256), (257, 129), (1000, 600)])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (2, 2, 64), (5, 1, 128)])
def test_attention_prompts(handle, n, m, Hq, Hk, D):
    _attention(handle, [(n, m)], Hq, Hk, D, 16, seed=n)


@pytest.mark.parametrize("Hq,Hk,D,page", [(4, 2, 127, 16), (2, 1, 128, 5), (2, 1, 192, 16), (3, 1, 512, 8), (2, 2, 1, 1),
                                          (8, 2, 20, 48)])
def test_attention_any_layout(handle, Hq, Hk, D, page):
    lens = [(70, 3), (1, 1), (0, 1), (33, 33), (0, 0), (257, 1)]
    _attention(handle, lens, Hq, Hk, D, page, seed=page, layout="apart", shared=0)
    _attention(handle, [(3 * page + 7 * i, 1) for i in range(5)], Hq, Hk, D, page, seed=page, shared=3 * page)


@pytest.mark.parametrize("shared,page", [(16, 16), (128, 16), (144, 16), (1024, 64), (1000 // 32 * 32, 32), (2048, 128)])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (4, 4, 64), (14, 2, 96)])
def test_attention_shared_prefix(handle, shared, page, Hq, Hk, D):
    lens = [(shared + i * 13 + 1, 1) for i in range(19)]
    _attention(handle, lens, Hq, Hk, D, page, seed=shared, shared=shared, one=True, behind=0)
    lens = [(shared + 5, 5), (shared + 70, 2), (shared - 3, 1), (shared, 7), (0, 0), (shared + 200, 3), (2, 2), (0, 1)]
    _attention(handle, lens, Hq, Hk, D, page, seed=shared, shared=shared)


def test_attention_one_long_request_is_split(handle):
    _attention(handle, [(9001, 1)], 8, 1, 128, 32, one=True, behind=0)
    _attention(handle, [(9001, 40)], 8, 1, 128, 32)
    _attention(handle, [(20000, 1), (3, 1)], 2, 2, 64, 128, one=True, behind=0)


@pytest.mark.parametrize("ask", [0, 1, 2, 1000])
def test_attention_max_query_len_only_chooses(handle, ask):
    _attention(handle, [(150, 9), (40, 1), (300, 30)], 8, 2, 128, 16, ask=ask)


@pytest.mark.parametrize("m", [1, 20])
def test_attention_large_scores(handle, m):
    """Scores of several hundred: all the weight lies on single keys."""
    _attention(handle, [(500, m), (90, m)], 8, 1, 128, 16, big=40.0)
    _attention(handle, [(500, m), (90, m)], 8, 1, 128, 16, big=4.0, scale=-0.5)


@pytest.mark.parametrize("m,D", [(1, 128), (20, 128), (1, 100), (3, 100)])
def test_attention_values_that_are_not_finite(handle, m, D):
    """A NaN key reaches the rows that see it and no others; a key whose score is -inf has no weight; a row whose
    every score is -inf is empty."""
    def nan_key(q, kc, vc, tables):
        kc[tables[0][3], 0, 5] = NAN            # key 53 of request 0

    _attention(handle, [(300, m), (300, m)], 4, 1, D, 16, tamper=nan_key)

    def dead(q, kc, vc, tables):
        q[:, :, 0] = 1.0
        for row, n in ((0, 300), (1, 40)):
            for i in range(n):
                if row == 1 or i % 3 == 0:
                    kc[tables[row][i // 16], 0, i % 16, 0] = -math.inf

    _attention(handle, [(300, m), (40, m), (77, m)], 4, 1, D, 16, tamper=dead)


@pytest.mark.parametrize("Hq,Hk,D,m", [(4, 1, 128, 4), (2, 2, 64, 9), (8, 1, 128, 40), (3, 3, 64, 300), (8, 1, 96, 17)])
@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
def test_attention_values_not_finite_stay_with_the_rows_that_see_them(handle, Hq, Hk, D, m, bad):
    """A value that is not finite in the middle of the new tokens: rows in front of it are as without it."""
    def spoil(q, kc, vc, tables):
        for b, at in ((0, 700 - m // 2), (1, 333 - 1)):
            vc[tables[b][at // 16], Hk - 1, at % 16, 5] = bad
            vc[tables[b][at // 16], 0, at % 16, D - 1] = bad

    lens = [(700, m), (333, m), (m + 60, m)]
    _attention(handle, lens, Hq, Hk, D, 16, tamper=spoil)
    _attention(handle, [(n + 1024, k) for n, k in lens], Hq, Hk, D, 16, shared=1024,
               tamper=lambda q, kc, vc, tables: [vc.__setitem__((tables[0][(1724 - m // 2) // 16], 0, (1724 - m // 2) % 16, 3), bad)])
    _attention(handle, [(9000, m)], Hq, Hk, D, 16,
               tamper=lambda q, kc, vc, tables: [vc.__setitem__((tables[0][(9000 - m // 2) // 16], 0, (9000 - m // 2) % 16, 3), bad)])


def test_attention_spoilt_rows_in_place(handle):
    """The same with the result over the queries, which the rows in front of the bad value are worked out from again."""
    g = torch.Generator(device="cuda").manual_seed(4)
    for m in (4, 100):
        q = torch.randn((m, 4, 64), generator=g, device="cuda").bfloat16()
        kc, vc = (torch.randn((40, 2, 16, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
        table = torch.randperm(40, generator=g, device="cuda").to(I32)[None, :20]
        clean = pkg.moe_lora_attention(handle, q, kc, vc, table, ints([300]), ints([0, m]))
        at = 300 - m // 2
        vc[int(table[0, at // 16]), :, at % 16, 7] = math.inf
        got = pkg.moe_lora_attention(handle, q, kc, vc, table, ints([300]), ints([0, m]), out=q)
        assert got is q
        near = (got[:m // 2].float() - clean[:m // 2].float()).abs() <= 2.0 ** -6 * clean[:m // 2].float().abs() + 2.0 ** -7
        assert near.all() and not torch.isfinite(got[m // 2:, :, 7].float()).any()


def test_attention_bad_pages_are_reported(handle):
    """A page outside the cache is read as zeros and reported; nothing outside is touched."""
    for m, Hq in ((1, 4), (30, 8)):
        q = torch.randn((m, Hq, 128), device="cuda").bfloat16()
        kc = torch.randn((4, 1, 16, 128), device="cuda").bfloat16()
        for bad in (-1, 4, 2 ** 31 - 1, -2 ** 31):
            ws = pkg.alloc_attention_workspace(m, Hq, 1, 128)
            out = pkg.moe_lora_attention(handle, q, kc, kc, ints([[0, bad, 2]]), ints([40]), query_offsets=ints([0, m]),
                                         max_query_len=m, workspace=ws)
            assert status(ws) == 6
            keys = torch.cat([kc[0, 0], torch.zeros_like(kc[0, 0]), kc[2, 0]])[:40].double()
            s = torch.einsum("thd,nd->htn", q.double(), keys) / math.sqrt(128)
            s = s.masked_fill(torch.ones((m, 40), dtype=torch.bool, device="cuda").triu(40 - m + 1), -math.inf)
            want = torch.einsum("htn,nd->thd", s.softmax(2), keys)
            assert (out.double() - want).abs().max() < 0.05


@pytest.mark.parametrize("kv,offsets", [([41], [0, 3]), ([-1], [0, 3]), ([30], [2, 1]), ([30], [-1, 2]), ([30], [0, 4])])
def test_attention_bad_lengths_are_reported(handle, kv, offsets):
    kc = torch.randn((4, 1, 16, 128), device="cuda").bfloat16()
    for Hq in (1, 16):
        ws = pkg.alloc_attention_workspace(3, Hq, 1, 128)
        pkg.moe_lora_attention(handle, torch.randn((3, Hq, 128), device="cuda").bfloat16(), kc, kc, ints([[0, 1]]), ints(kv),
                               query_offsets=ints(offsets), max_query_len=3, workspace=ws)
        assert status(ws) == 6


def test_attention_in_place_and_repeated(handle):
    g = torch.Generator(device="cuda").manual_seed(3)
    for m in (1, 40):
        q = torch.randn((3 * m, 8, 128), generator=g, device="cuda").bfloat16()
        kc, vc = (torch.randn((400, 2, 16, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
        table = torch.randperm(390, generator=g, device="cuda").to(I32).view(3, 130)
        args = (kc, vc, table, ints([2000, 77, 500]), ints([0, m, 2 * m, 3 * m]), m)
        a = pkg.moe_lora_attention(handle, q, *args)
        b = pkg.moe_lora_attention(handle, q, *args)
        assert torch.equal(a, b)
        c = pkg.moe_lora_attention(handle, q, *args, out=q)
        assert c is q and torch.equal(a, q)


def test_attention_larger_workspace_of_a_larger_call(handle):
    sizes = [pkg.moe_lora_attention_workspace_size(T, 32, 4, 128) for T in (0, 1, 3, 16, 17, 100, 1000, 10000, 100000)]
    assert sizes == sorted(sizes)


def test_on_another_stream_and_captured(handle):
    """The operators of a step captured once and replayed with other lengths, on a stream of their own."""
    side = torch.cuda.Stream()
    h = pkg.Handle(0)
    page, width, B, T, Hq, Hk, D = 16, 40, 5, 24, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = (torch.zeros((300, Hk, page, D), device="cuda").bfloat16() for _ in range(2))
    table = torch.full((B, width), -1, dtype=I32, device="cuda")
    free = torch.randperm(300, generator=g, device="cuda").to(I32)
    lens, new, taken = ints([0] * B), ints([0] * B), ints([0])
    qkv = torch.empty((T, (Hq + 2 * Hk) * D), device="cuda").bfloat16()
    out = torch.empty((T, Hq, D), device="cuda").bfloat16()
    ws, ws2 = pkg.alloc_cache_workspace(), pkg.alloc_attention_workspace(T, Hq, Hk, D)
    o = {"kv_lens": lens, "taken": taken}

    def step():
        pkg.moe_lora_page_tables(h, table, lens, new, page, free, taken, T, outputs=o, workspace=ws)
        k, v = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D), qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
        pkg.moe_lora_cache_write(h, k, v, kc, vc, o["slot_map"])
        pkg.moe_lora_attention(h, qkv[:, :Hq * D].view(T, Hq, D), kc, vc, table, lens, o["query_offsets"], T, out=out,
                               workspace=ws2)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    keys = [[] for _ in range(B)]
    r = random.Random(1)
    for _ in range(6):
        add = [r.randint(0, 6) for _ in range(B)]
        add[r.randrange(B)] = 0
        while sum(add) > T:
            add[add.index(max(add))] -= 1
        rows = torch.randn(qkv.shape, generator=g, device="cuda").bfloat16()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            new.copy_(ints(add))
            qkv.copy_(rows)
            out.fill_(7.0)
            graph.replay()
        side.synchronize()
        assert status(ws) == 0 and status(ws2) == 0
        t = 0
        for b, n in enumerate(add):
            for i in range(n):
                keys[b].append(rows[t + i, Hq * D:].view(2, Hk, D).double())
            for i in range(n):
                seen = torch.stack(keys[b][:len(keys[b]) - n + i + 1])     # [keys, 2, Hk, D]
                q = rows[t + i, :Hq * D].view(Hk, Hq // Hk, D).double()
                p = torch.einsum("hgd,nhd->hgn", q, seen[:, 0]).div(math.sqrt(D)).softmax(2)
                want = torch.einsum("hgn,nhd->hgd", p, seen[:, 1]).reshape(Hq, D)
                size = torch.einsum("hgn,nhd->hgd", p, seen[:, 1].abs()).reshape(Hq, D)
                assert ((out[t + i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1.1 * 2.0 ** -8 * size).all()
            t += n
        assert (out[t:] == 7.0).all()
        assert lens.tolist() == [len(k) for k in keys]
    h.close()


def test_tensors_of_a_named_stream(handle):
    side = torch.cuda.Stream()
    kc = torch.randn((8, 1, 16, 128), device="cuda").bfloat16()
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    table, lens = ints([[0, 1, 2], [3, 4, 5]]), ints([40, 3])
    torch.cuda.synchronize()
    a = pkg.moe_lora_attention(handle, q, kc, kc, table, lens, stream=side)
    side.synchronize()
    assert torch.equal(a, pkg.moe_lora_attention(handle, q, kc, kc, table, lens))
