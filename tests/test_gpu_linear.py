"""moe_lora_linear against its definition in 64 bits: token counts around the tile sizes, odd
widths, ragged ranks, strides, types, streams, graphs, and what it refuses."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_reference as ref
import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    return pkg.Handle(0)


def _rand(shape, std, g):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def _case(T, N, K, ranks, seed=0, bias=False, slots="mixed", nan_tail=True):
    g = torch.Generator().manual_seed(seed)
    S, R = len(ranks), max(ranks, default=0)
    c = dict(x=_rand((T, K), 1.0, g), w=_rand((N, K), 1 / math.sqrt(K), g),
             bias=torch.randn(N, generator=g) if bias else None, A=None, B=None, slots=None, ranks=list(ranks))
    if S:
        c["A"] = _rand((S, max(R, 1), K), 1 / math.sqrt(K), g)
        c["B"] = _rand((S, N, max(R, 1)), 0.3, g)
        if nan_tail:
            for s, r in enumerate(ranks):
                c["A"][s, r:] = float("nan")
                c["B"][s, :, r:] = float("nan")
        if slots == "mixed":
            c["slots"] = torch.randint(-1, S, (T,), generator=g, dtype=torch.int32)
        elif slots == "none":
            c["slots"] = torch.full((T,), -1, dtype=torch.int32)
        else:   # runs of 50 tokens
            c["slots"] = ((torch.arange(T) // 50) % (S + 1) - 1).to(torch.int32)
    c["scalings"] = [[2.0, 0.5, 1.0, -0.25][s % 4] for s in range(S)]
    return c


def _dev(t):
    return None if t is None else t.cuda()


def _run(h, c, f32=False, out=None, x=None, w=None, workspace=None):
    ad = None
    if c["A"] is not None:
        ad = pkg.moe_lora_linear_adapters(h, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
    return pkg.moe_lora_linear(h, _dev(c["x"]) if x is None else x, _dev(c["w"]) if w is None else w, adapters=ad,
                               slot_idx=_dev(c["slots"]), bias=_dev(c["bias"]), out=out,
                               out_dtype=torch.float32 if f32 else torch.bfloat16, workspace=workspace)


def _check(got, c, f32=False):
    sl = None if c["slots"] is None else c["slots"].numpy()
    y, tol = ref.linear(c["x"], c["w"], c["bias"], c["A"], c["B"], sl, c["ranks"], c["scalings"], f32)
    err = np.abs(ref.f64(got) - y)
    assert np.isfinite(ref.f64(got)).all()
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} times the bound at {np.argwhere(err > tol)[:4].tolist()}"


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 300])
def test_token_counts(handle, T, f32):
    c = _case(T, 200, 328, (8, 16, 5), seed=T, bias=True)
    got = _run(handle, c, f32)
    assert got.shape == (T, 200) and got.dtype == (torch.float32 if f32 else torch.bfloat16)
    _check(got, c, f32)


@pytest.mark.parametrize("N,K", [(1, 8), (7, 8), (128, 64), (129, 72), (130, 520), (384, 2048), (1001, 136), (4100, 1024)])
@pytest.mark.parametrize("T", [3, 70])
def test_widths(handle, T, N, K):
    _check(_run(handle, c := _case(T, N, K, (16, 3), seed=N + T)), c)
    _check(_run(handle, c := _case(T, N, K, (), seed=N + T, bias=True), True), c, True)


@pytest.mark.parametrize("T,N,K", [(2500, 2050, 136), (2560, 2048, 512), (5121, 1000, 72), (19500, 130, 64), (1281, 4096, 264),
                                   (3066, 1551, 136), (400, 1536, 2048), (1536, 3008, 328)])
@pytest.mark.parametrize("slots", ["mixed", "runs", "none", None])
def test_long_batches(handle, T, N, K, slots):
    """Enough tokens for the widest tiles: ragged in every direction, rows of y on and off 16-byte
    boundaries, adapters of several 64-column blocks."""
    for f32 in (False, True):
        c = _case(T, N, K, (16, 40, 64, 5) if slots else (), seed=T, bias=N % 2 == 0, slots=slots or "none")
        _check(_run(handle, c, f32), c, f32)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("ranks", [(16, 40), (64, 48)], ids=["64", "128"])
@pytest.mark.parametrize("T,N,K", [(777, 1536, 2048), (2450, 1560, 1640), (2304, 1000, 520), (300, 8000, 512), (513, 3200, 776)])
def test_shrinks_shared_by_several_pairs(handle, T, N, K, ranks, f32):
    """At most one product tile for each pair of SMs, with pairs to spare and without; run twice for the
    same bits, and once more after a call without adapters."""
    c = _case(T, N, K, ranks, seed=N, slots="runs", bias=True)
    got = _run(handle, c, f32)
    _check(got, c, f32)
    assert torch.equal(got, _run(handle, c, f32))
    _run(handle, dict(c, A=None, slots=None), f32)
    assert torch.equal(got, _run(handle, c, f32))


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("ranks", [(16, 40), (64, 48)], ids=["64", "128"])
@pytest.mark.parametrize("T,N,K", [(4000, 2300, 1040), (6000, 1800, 1104), (5000, 1792, 7168)])
def test_shrinks_dealt_out_over_several_tiles_per_pair(handle, T, N, K, ranks, f32):
    c = _case(T, N, K, ranks, seed=K, slots="runs", bias=True)
    ad = pkg.moe_lora_linear_adapters(handle, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
    ws = pkg.alloc_linear_workspace(T, ad)
    ws.fill_(255)
    got = _run(handle, c, f32, workspace=ws)
    _check(got, c, f32)
    assert torch.equal(got, _run(handle, c, f32, workspace=ws))


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("ranks", [(), (16, 40), (64, 64, 64)], ids=["none", "64", "192"])
@pytest.mark.parametrize("T,N,K", [(300, 1000, 2056), (777, 1536, 2048), (600, 641, 2304), (1281, 384, 4104), (200, 2400, 3080)])
def test_products_shared_by_several_pairs(handle, T, N, K, ranks, f32):
    """So few tiles that pairs of SMs share a tile's K; again for the same bits, and into a column range
    of a wider tensor, of which nothing else is written."""
    c = _case(T, N, K, ranks, seed=N + 1, slots="runs", bias=True)
    got = _run(handle, c, f32)
    _check(got, c, f32)
    buf = torch.full((T + 2, N + 11), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    assert torch.equal(got, _run(handle, c, f32, out=buf[1:T + 1, 3:N + 3]))
    buf[1:T + 1, 3:N + 3] = 77.0
    assert (buf == 77.0).all()


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("ranks", [(16,), (64, 64, 64), (40,) * 20], ids=["64", "192", "800"])
@pytest.mark.parametrize("T,N,K", [(1, 200, 512), (40, 384, 1024), (100, 384, 2048), (250, 384, 4104), (1281, 384, 4104),
                                   (777, 1536, 1024), (5000, 1536, 264)])
def test_what_the_workspace_held_does_not_matter(handle, T, N, K, ranks, f32):
    """NaN in every byte of it, and slots in runs, so that neighbouring tokens need different blocks of
    the stacked adapters."""
    c = _case(T, N, K, ranks, seed=T, slots="runs")
    ad = pkg.moe_lora_linear_adapters(handle, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
    ws = pkg.alloc_linear_workspace(T, ad)
    ws.fill_(255)
    _check(_run(handle, c, f32, workspace=ws), c, f32)


@pytest.mark.parametrize("T,N,K", [(3, 130, 7168), (200, 384, 7168), (1500, 384, 7168), (900, 200, 4104)])
def test_long_sums_in_float32(handle, T, N, K):
    """The tensor cores truncate as they accumulate; in parts of 1024 the error of a float32 result
    over a long K stays that of a float32 sum of such parts: at most 64 steps of 16 products each
    truncated to 24 bits (2^-23 of the running sum, which stays below the part's largest sum of
    |terms| / sqrt of their count times 4 for these zero-mean terms), half of it on average: 32 * 2^-23
    relative to the result's size, here held in the 2-norm."""
    c = _case(T, N, K, (), seed=T)
    got = ref.f64(_run(handle, c, True))
    y = ref.f64(c["x"]) @ ref.f64(c["w"]).T
    assert np.linalg.norm(got - y) <= 32 * 2.0 ** -23 * np.linalg.norm(y)


@pytest.mark.parametrize("ranks", [(1,), (128,), (0, 8), (64, 64, 64), (8, 16, 32, 64), (16,) * 40, (64,) * 64],
                         ids=lambda r: f"{len(r)}x{max(r)}")
@pytest.mark.parametrize("T,slots", [(5, "mixed"), (200, "mixed"), (500, "runs"), (40, "none")])
def test_ranks(handle, ranks, T, slots):
    for f32 in (False, True):
        c = _case(T, 264, 256, ranks, seed=len(ranks) + T, slots=slots)
        _check(_run(handle, c, f32), c, f32)


def test_factors_of_zero_and_all_ranks_zero(handle):
    c = _case(30, 136, 128, (8, 16))
    c["scalings"] = [0.0, 1.5]
    _check(_run(handle, c), c)
    c["scalings"] = [0.0, 0.0]
    base = _run(handle, dict(c, A=None, slots=None))
    assert torch.equal(_run(handle, c), base)
    c = _case(30, 136, 128, (0, 0))
    _check(_run(handle, c), c)


@pytest.mark.parametrize("T", [1, 20, 150, 700, 19700])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
def test_strided_rows_and_nothing_else_written(handle, T, f32):
    """Rows of x and w inside wider tensors, the result as a column range of a wider tensor, from
    an offset that leaves it aligned to its elements alone."""
    N, K = 141, 200
    c = _case(T, N, K, (8, 24), seed=T)
    xw = torch.full((T + 1, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:T, 16:16 + K] = c["x"].cuda()
    ww = torch.full((N + 2, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    ww[1:N + 1, :K] = c["w"].cuda()
    for lead, width in ((3, N + 10), (4, 152), (8, 160)):
        buf = torch.full((T + 2, width), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        got = _run(handle, c, f32, out=buf[1:T + 1, lead:lead + N], x=xw[:T, 16:16 + K], w=ww[1:N + 1, :K])
        _check(got, c, f32)
        rest = buf.clone()
        rest[1:T + 1, lead:lead + N] = 77.0
        assert (rest == 77.0).all()


def test_large_values_infinities_and_nan_pass_through(handle):
    c = _case(40, 130, 64, (8,), seed=3)
    c["slots"][:] = 0
    c["slots"][5] = -1
    c["x"][2, 3] = float("inf")
    c["x"][9, 1] = float("nan")
    got = _run(handle, c).float().cpu()
    bad = ~torch.isfinite(got).all(1)
    assert bad.nonzero()[:, 0].tolist() == [2, 9]      # no other token sees them


def test_same_bits_every_time_and_on_other_streams(handle):
    c = _case(90, 640, 2048, (8, 16, 32), seed=1)
    ad = pkg.moe_lora_linear_adapters(handle, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
    x, w, slots = c["x"].cuda(), c["w"].cuda(), c["slots"].cuda()
    a = pkg.moe_lora_linear(handle, x, w, ad, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = pkg.moe_lora_linear(handle, x, w, ad, slots)
    d = pkg.moe_lora_linear(handle, x, w, ad, slots, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, d)
    _check(a, c)


def test_graph_replay_on_new_inputs(handle):
    for T in (4, 600, 10000):
        c = _case(T, 264, 512, (8, 16), seed=T)
        ad = pkg.moe_lora_linear_adapters(handle, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
        x, w, slots = c["x"].cuda(), c["w"].cuda(), c["slots"].cuda()
        ws, out = pkg.alloc_linear_workspace(T, ad), torch.empty((T, 264), dtype=torch.bfloat16, device="cuda")
        pkg.moe_lora_linear(handle, x, w, ad, slots, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.moe_lora_linear(handle, x, w, ad, slots, out=out, workspace=ws)
        for seed in (5, 6):
            c2 = _case(T, 264, 512, (8, 16), seed=seed)
            x.copy_(c2["x"])
            slots.copy_(c2["slots"])
            graph.replay()
            torch.cuda.synchronize()
            _check(out, dict(c, x=c2["x"], slots=c2["slots"]))


def test_slot_out_of_range_is_reported_and_adds_nothing(handle):
    c = _case(33, 136, 128, (8, 16), seed=2)
    ad = pkg.moe_lora_linear_adapters(handle, c["A"].cuda(), c["B"].cuda(), c["ranks"], c["scalings"])
    ws = pkg.alloc_linear_workspace(33, ad)
    for bad in (2, -2, 2 ** 30):
        s = c["slots"].clone()
        s[7] = bad
        got = pkg.moe_lora_linear(handle, c["x"].cuda(), c["w"].cuda(), ad, s.cuda(), workspace=ws)
        st, word = pkg.moe_lora_check_status(ws)
        assert st == 6 and (word & 0xff) == 6
        s[7] = -1
        _check(got, dict(c, slots=s))
        pkg.moe_lora_linear(handle, c["x"].cuda(), c["w"].cuda(), ad, s.cuda(), workspace=ws)
        assert pkg.moe_lora_check_status(ws)[0] == 0
    pkg.moe_lora_linear(handle, c["x"].cuda(), c["w"].cuda(), workspace=ws)
    assert pkg.moe_lora_check_status(ws)[0] == 0


def test_empty_batch(handle):
    n = handle.launch_count()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((32, 64), dtype=torch.bfloat16, device="cuda")
    assert pkg.moe_lora_linear(handle, x, w).shape == (0, 32)
    assert handle.launch_count() == n


def test_refusals(handle):
    c = _case(8, 32, 64, (8, 4))
    x, w, A, B, slots = c["x"].cuda(), c["w"].cuda(), c["A"].cuda(), c["B"].cuda(), c["slots"].cuda()
    ad = pkg.moe_lora_linear_adapters(handle, A, B, c["ranks"], c["scalings"])
    n = handle.launch_count()
    f = lambda *a, **k: pkg.moe_lora_linear(handle, *a, **k)
    for bad in (lambda: f(x.float(), w), lambda: f(x[:, :32], w), lambda: f(x.cpu(), w), lambda: f(x, w, ad),
                lambda: f(x, w, ad, slots.long()), lambda: f(x, w, ad, slots[:4]), lambda: f(x, w[:16], ad, slots),
                lambda: f(x, w, bias=torch.zeros(31, device="cuda")), lambda: f(x, w, out_dtype=torch.float16),
                lambda: f(x, w, out=torch.empty((8, 31), dtype=torch.bfloat16, device="cuda")),
                lambda: f(x.t().contiguous().t(), w), lambda: f(x[0], w),
                lambda: pkg.moe_lora_linear_adapters(handle, A, B[:, :, :4], c["ranks"], c["scalings"]),
                lambda: pkg.moe_lora_linear_adapters(handle, A, B, [8], c["scalings"])):
        with pytest.raises(ValueError):
            bad()
    codes = []
    for bad in (lambda: f(torch.empty((8, 68), dtype=torch.bfloat16, device="cuda")[:, 1:65], w),       # alignment
                lambda: f(torch.empty((8, 68), dtype=torch.bfloat16, device="cuda")[:, :64], w),        # row stride
                lambda: f(torch.empty((8, 12), dtype=torch.bfloat16, device="cuda"),
                          torch.empty((4, 12), dtype=torch.bfloat16, device="cuda")),                   # K % 8
                lambda: f(x, w, ad, slots, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                lambda: pkg.moe_lora_linear_adapters(handle, A, B, [9, 4], c["scalings"]),              # rank above R
                lambda: pkg.moe_lora_linear_adapters(
                    handle, torch.empty((64, 128, 8), dtype=torch.bfloat16, device="cuda"),
                    torch.empty((64, 8, 128), dtype=torch.bfloat16, device="cuda"), [128] * 64, [1.0] * 64)):
        with pytest.raises(pkg.MoELoRAError) as e:
            bad()
        codes.append(e.value.status)
    assert codes == [1, 1, 1, 3, 1, 2]
    nan = pkg.moe_lora_linear_adapters(handle, A, B, c["ranks"], [float("nan"), 1.0])
    with pytest.raises(pkg.MoELoRAError):
        f(x, w, nan, slots)
    assert handle.launch_count() == n + 1   # the NaN-factor stack alone


def test_large_offsets(handle):
    """Rows past 2^31 elements of x, w and y: only the strides are large."""
    T, N, K = 3, 140, 64
    c = _case(T, N, K, (8,), seed=4)
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    pitch = (1 << 30) + 8
    xb = torch.empty(2 * pitch + K, dtype=torch.bfloat16, device="cuda")
    x = xb.as_strided((T, K), (pitch, 1))
    x.copy_(c["x"])
    yb = torch.empty(2 * pitch + N, dtype=torch.float32, device="cuda")
    out = yb.as_strided((T, N), (pitch, 1))
    _check(_run(handle, c, True, out=out, x=x), c, True)
