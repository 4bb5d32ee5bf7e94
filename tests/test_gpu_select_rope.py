"""moe_lora_select_experts and moe_lora_qk_norm_rope against their definitions in 64 bits: ties,
groups, ruled-out experts, odd sizes, strides, types, streams, and what they refuse."""
import numpy as np
import pytest
import torch

import block_reference as ref
import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def handle():
    return pkg.Handle(0)


# ------------------------------------------------------------------------------------- select
def _logits(T, E, seed, dtype, masked=0.0):
    """Logits on a coarse grid, so that equal keys are exact ties and others lie well apart."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randint(-16, 17, (T, E), generator=g) / 8.0
    if masked:
        z[torch.rand((T, E), generator=g) < masked] = -INF
    return z.to(dtype)


def _bias(E, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    return torch.randint(-8, 9, (E,), generator=g) / 64.0


def _apart(keys):
    """Distinct 64-bit keys of a token differ by more than float32 can blur."""
    for row in keys:
        v = np.unique(row[row > -np.inf])
        gap = np.diff(v)
        if gap.size and (gap[gap > 1e-13] < 2e-6).any():
            return False
    return True


# Relative error of a weight: a score is a quotient and an exponential of an exact difference (2 ulp),
# the sum of 32 at most, the quotient, the factor: 64 roundings of 2^-24 hold it amply.
W_RTOL = 64 * 2.0 ** -24


def _select(handle, z, k, sigmoid, bias=None, **kw):
    o = pkg.moe_lora_select_experts(handle, z if z.is_cuda else z.cuda(), k,
                                    scoring=pkg.SCORE_SIGMOID if sigmoid else pkg.SCORE_SOFTMAX,
                                    bias=None if bias is None else bias.cuda(), packed=True, **kw)
    ids, w = o["topk_ids"].cpu().numpy(), o["topk_weights"].cpu().numpy()
    pk = o["packed_topk_ids"].cpu().numpy()
    np.testing.assert_array_equal(pk >> 16, ids)
    bits = o["topk_weights"].to(torch.bfloat16).view(torch.int16).cpu().numpy().astype(np.int32) & 0xFFFF
    np.testing.assert_array_equal(pk & 0xFFFF, bits)
    return ids, w


def _compare(handle, z, k, sigmoid, bias=None, n_group=1, topk_group=1, top2=False, renormalize=True, factor=1.0):
    ids, w = _select(handle, z, k, sigmoid, bias, n_group=n_group, topk_group=topk_group,
                     group_score=pkg.GROUP_TOP2 if top2 else pkg.GROUP_MAX, renormalize=renormalize,
                     routed_scaling_factor=factor)
    rids, rw, keys = ref.select(z, k, sigmoid, bias, n_group, topk_group, top2, renormalize, factor)
    assert _apart(keys), "the test's inputs leave keys too close to tell apart in float32"
    np.testing.assert_array_equal(ids, rids)
    np.testing.assert_allclose(w, rw, rtol=W_RTOL, atol=1e-30)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 5, 5), (3, 33, 7), (9, 64, 8), (33, 128, 8), (2, 130, 32), (40, 256, 8),
                                   (17, 257, 3), (9, 384, 8), (5, 500, 10), (1100, 64, 4), (2, 1023, 32), (2, 1024, 32)])
def test_sizes(handle, T, E, k, dtype, sigmoid):
    _compare(handle, _logits(T, E, E + T, dtype), k, sigmoid, factor=2.5)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("top2", [False, True], ids=["max", "top2"])
@pytest.mark.parametrize("E,n_group,topk_group,k", [(16, 4, 2, 8), (256, 8, 4, 8), (384, 8, 3, 6), (60, 4, 3, 6), (96, 32, 9, 8),
                                                    (20, 10, 10, 5), (1024, 32, 1, 32), (14, 2, 1, 7)])
def test_groups(handle, E, n_group, topk_group, k, top2, sigmoid):
    for masked in (0.0, 0.3):
        _compare(handle, _logits(21, E, E, torch.float32, masked), k, sigmoid, None, n_group, topk_group, top2,
                 renormalize=masked == 0.0)


@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (8, 3)])
def test_bias_chooses_and_does_not_weigh(handle, n_group, topk_group):
    _compare(handle, _logits(50, 64, 5, torch.float32), 6, True, _bias(64, 1), n_group, topk_group, False)
    # a bias that lifts the last expert over all others
    b = torch.zeros(64)
    b[63] = 100.0
    ids, w = _select(handle, _logits(50, 64, 5, torch.float32), 1, True, b)
    assert (ids == 63).all()
    np.testing.assert_allclose(w, 1.0)


def test_all_equal_logits_choose_the_lowest_ids(handle):
    for sigmoid in (False, True):
        ids, w = _select(handle, torch.zeros(4, 200), 8, sigmoid)
        assert (ids == np.arange(8)).all()
        np.testing.assert_allclose(w, 1 / 8, rtol=W_RTOL)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_ruled_out_experts(handle, sigmoid):
    z = _logits(6, 40, 7, torch.float32)
    z[0] = -INF                         # nothing left
    z[1, 1:] = -INF                     # one left, fewer than k
    z[1, 0] = 0.5
    z[2] = float("nan")
    z[3, ::2] = float("nan")
    z[4] = torch.finfo(torch.float32).min          # the type's lowest value masks nothing: all equal
    z[5, 3] = INF
    z[5, 9] = INF
    bias = torch.zeros(40)
    bias[39] = 50.0                     # lifts no ruled-out expert
    for b in (None, bias):
        ids, w = _select(handle, z, 4, sigmoid, b)
        assert np.isfinite(w).all()
        rids, rw, _ = ref.select(z, 4, sigmoid, b)
        np.testing.assert_array_equal(ids, rids)
        np.testing.assert_allclose(w, rw, rtol=W_RTOL, atol=1e-30)
    ids, w = _select(handle, z, 4, sigmoid)
    assert ids[0].tolist() == [0, 1, 2, 3] and (w[0] == 0).all() and (w[2] == 0).all()
    assert ids[1].tolist() == [0, 1, 2, 3] and w[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert ids[5, :2].tolist() == [3, 9]
    low = torch.full((2, 64), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16)
    low[:, 5] = 1.0
    ids, w = _select(handle, low, 2, sigmoid)
    assert ids[0].tolist() == [5, 0] and w[0, 0] == 1.0 and w[0, 1] == 0.0


@pytest.mark.parametrize("spread", [1.0, 8.0, 60.0])
@pytest.mark.parametrize("E", [128, 200, 384])
def test_softmax_scores_are_the_correctly_rounded_quotients(handle, E, spread):
    """The kernel's quotient (a reciprocal and one residual) against IEEE division of the same
    exponentials by the same sum, bit for bit; at the largest spread the small terms underflow."""
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.randn((400, E), generator=g, device="cuda") * spread
    e = torch.exp(z - z.amax(1, keepdim=True))
    p = e / e.double().sum(1, keepdim=True).float()
    o = pkg.moe_lora_select_experts(handle, z, 32, renormalize=False)
    assert torch.equal(o["topk_weights"], p.gather(1, o["topk_ids"].long()))


@pytest.mark.parametrize("spread", [1.0, 8.0, 60.0])
def test_sigmoid_scores_are_the_correctly_rounded_reciprocals(handle, spread):
    """The kernel's reciprocal against IEEE division, bit for bit; the largest spread has scores that
    are subnormal or 0."""
    g = torch.Generator(device="cuda").manual_seed(9)
    z = torch.randn((20000, 32), generator=g, device="cuda") * spread
    s = 1.0 / (1.0 + torch.exp(-z))
    o = pkg.moe_lora_select_experts(handle, z, 32, scoring=pkg.SCORE_SIGMOID, renormalize=False)
    assert torch.equal(o["topk_weights"], s.gather(1, o["topk_ids"].long()))
    assert torch.equal(o["topk_ids"].long(), torch.sort(s, dim=1, descending=True, stable=True).indices)


@pytest.mark.parametrize("scale", [1e-38, 1e-3, 1.0, 40.0])
@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (8, 3)])
def test_softmax_ties_of_the_quotients_go_to_the_lower_id(handle, scale, n_group, topk_group):
    """Neighbouring numerators can have one quotient; the choice is by the quotient, then by the id."""
    g = torch.Generator(device="cuda").manual_seed(17)
    z = torch.randn((3000, 256), generator=g, device="cuda") * scale * 2.0 ** torch.randint(
        -20, 1, (3000, 1), generator=g, device="cuda")
    e = torch.exp(z - z.amax(1, keepdim=True))
    s = e / e.double().sum(1, keepdim=True).float()
    if n_group > 1:
        best = torch.sort(s.view(3000, n_group, -1).amax(2), dim=1, descending=True, stable=True).indices
        keep = torch.zeros((3000, n_group), dtype=torch.bool, device="cuda").scatter(1, best[:, :topk_group], True)
        s = torch.where(keep.repeat_interleave(256 // n_group, 1), s, -1.0)
    o = pkg.moe_lora_select_experts(handle, z, 8, n_group=n_group, topk_group=topk_group, renormalize=False)
    ids = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :8]
    assert torch.equal(o["topk_ids"].long(), ids)
    assert torch.equal(o["topk_weights"], s.gather(1, ids))


def test_strided_and_unaligned_logits(handle):
    wide = torch.full((30, 300), float("nan"), dtype=torch.float32, device="cuda")
    for lead, E, dtype in ((3, 256, torch.float32), (4, 256, torch.float32), (1, 129, torch.bfloat16), (2, 128, torch.bfloat16)):
        z = _logits(30, E, lead, dtype)
        buf = wide.to(dtype)
        buf[:, lead:lead + E] = z.cuda()
        ids, w = _select(handle, buf[:, lead:lead + E], 8, True)
        rids, rw, _ = ref.select(z, 8, True)
        np.testing.assert_array_equal(ids, rids)
        np.testing.assert_allclose(w, rw, rtol=W_RTOL)


def test_select_on_another_stream_and_into_given_outputs(handle):
    z = _logits(64, 128, 3, torch.bfloat16).cuda()
    a = pkg.moe_lora_select_experts(handle, z, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = dict(topk_ids=torch.zeros((64, 8), dtype=torch.int32, device="cuda"),
             topk_weights=torch.zeros((64, 8), device="cuda"))
    b = pkg.moe_lora_select_experts(handle, z, 8, outputs=o, stream=side)
    torch.cuda.synchronize()
    assert b["topk_ids"] is o["topk_ids"] and "packed_topk_ids" not in b
    assert torch.equal(a["topk_ids"], b["topk_ids"]) and torch.equal(a["topk_weights"], b["topk_weights"])
    empty = pkg.moe_lora_select_experts(handle, z[:0], 8)
    assert empty["topk_ids"].shape == (0, 8)


def test_select_feeds_the_routed_layer(handle):
    """The packed words are what the externally routed layer takes: its own record of the routing
    weights is the bf16 rounding of the weights chosen here."""
    import gpu_helpers as gh
    from routed_moe_expert_gb300 import workloads as wl
    cfg = wl.LayerConfig("sel", T=40, H=128, I=64, E=16, top_k=4, ranks=(8,), scalings=(1.0,))
    g = gh.to_dev(wl.make_inputs(cfg, seed=2))
    o = pkg.moe_lora_select_experts(handle, g["router_logits"], 4, packed=True)
    r = pkg.moe_lora_forward_routed(handle, g["hidden"], o["packed_topk_ids"], g["w1"], g["w2"], 4, 16, do_finalize=False,
                                    lora_A_gu=g["lora_A_gu"], lora_B_gu=g["lora_B_gu"], lora_A_dn=g["lora_A_dn"],
                                    lora_B_dn=g["lora_B_dn"], slot_idx=g["slot_idx"], ranks=g["ranks"],
                                    scalings=g["scalings"])
    torch.cuda.synchronize()
    assert torch.equal(r["expert_weights"], o["topk_weights"].to(torch.bfloat16).float())


def test_select_refusals(handle):
    z = torch.zeros((4, 64), device="cuda")
    f = lambda *a, **k: pkg.moe_lora_select_experts(handle, *a, **k)
    n = handle.launch_count()
    for bad in (lambda: f(z.half(), 4), lambda: f(z[0], 4), lambda: f(z.t(), 4), lambda: f(z.cpu(), 4),
                lambda: f(z, 4, bias=torch.zeros(63, device="cuda")), lambda: f(z, 4, bias=torch.zeros(64)),
                lambda: f(z, 4, outputs=dict(topk_ids=torch.zeros((4, 4), device="cuda")))):
        with pytest.raises(ValueError):
            bad()
    codes = []
    for bad in (lambda: f(z, 0), lambda: f(z, 33), lambda: f(z, 4, scoring=2), lambda: f(z, 4, n_group=3, topk_group=1),
                lambda: f(z, 4, n_group=8, topk_group=9), lambda: f(z, 9, n_group=8, topk_group=1),
                lambda: f(z, 4, n_group=64, topk_group=8), lambda: f(z, 4, group_score=5),
                lambda: f(torch.zeros((2, 32), device="cuda"), 4, n_group=32, topk_group=8, group_score=pkg.GROUP_TOP2),
                lambda: f(torch.zeros((1, 1025), device="cuda"), 4),
                lambda: f(z, 4, routed_scaling_factor=float("nan"))):
        with pytest.raises(pkg.MoELoRAError) as e:
            bad()
        codes.append(e.value.status)
    assert codes == [1, 1, 1, 1, 1, 1, 2, 1, 1, 1, 1]
    assert handle.launch_count() == n


# --------------------------------------------------------------------------------------- rope
def _table(P, R, seed=0):
    a = torch.rand((P, R // 2), generator=torch.Generator().manual_seed(seed)) * 6.3
    return torch.cat([a.cos(), a.sin()], 1)


def _qk(T, Hq, Hk, D, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    return (r(T, Hq, D).to(torch.bfloat16), r(T, Hk, D).to(torch.bfloat16), 1 + 0.2 * r(D), 1 + 0.2 * r(D),
            torch.randint(0, 50, (T,), generator=g))


def _near(got, want):
    y, tol = want
    err = np.abs(ref.f64(got) - y)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} times the bound at {np.argwhere(err > tol)[:4].tolist()}"


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1, 1, 1, 2, 2), (1, 32, 4, 128, 128), (3, 5, 2, 64, 64), (7, 4, 4, 80, 40),
                                         (7, 4, 4, 80, 80), (2, 3, 1, 96, 48), (5, 2, 2, 192, 64), (9, 8, 1, 256, 256),
                                         (4, 2, 1, 512, 512), (4, 2, 1, 512, 508), (3, 2, 1, 6, 4), (3, 7, 3, 33, 2),
                                         (3, 3, 3, 511, 510), (6, 2, 2, 128, 0), (700, 6, 2, 64, 32)])
def test_rope_sizes(handle, T, Hq, Hk, D, R, interleaved):
    for wt, pt in ((torch.bfloat16, torch.int32), (torch.float32, torch.int64)):
        q, k, wq, wk, pos = _qk(T, Hq, Hk, D, D + T)
        wq, wk, pos, table = wq.to(wt), wk.to(wt), pos.to(pt), _table(50, R)
        qo, ko = pkg.moe_lora_qk_norm_rope(handle, q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), table.cuda(), pos.cuda(),
                                           eps=1e-5, interleaved=interleaved)
        _near(qo, ref.norm_rope(q, wq, table, pos, 1e-5, interleaved))
        _near(ko, ref.norm_rope(k, wk, table, pos, 1e-5, interleaved))


@pytest.mark.parametrize("lead,D,R", [(0, 128, 128), (3, 128, 128), (4, 64, 32), (2, 48, 16)])
@pytest.mark.parametrize("T", [1, 65])
def test_rope_on_slices_of_merged_rows_in_place(handle, T, lead, D, R):
    """q and k as slices of merged rows, from offsets down to one element, written where they are;
    the values between and after them stay."""
    Hq, Hk = 6, 2
    q, k, wq, wk, pos = _qk(T, Hq, Hk, D, T)
    table = _table(50, R)
    buf = torch.full((T, lead + (Hq + 2 * Hk) * D + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    qs = buf[:, lead:lead + Hq * D].view(T, Hq, D)
    ks = buf[:, lead + Hq * D:lead + (Hq + Hk) * D].view(T, Hk, D)
    qs.copy_(q)
    ks.copy_(k)
    a, b = pkg.moe_lora_qk_norm_rope(handle, qs, ks, wq.cuda(), wk.cuda(), table.cuda(), pos.cuda(), q_out=qs, k_out=ks)
    assert a is qs and b is ks
    _near(qs, ref.norm_rope(q, wq, table, pos, 1e-6, False))
    _near(ks, ref.norm_rope(k, wk, table, pos, 1e-6, False))
    assert (buf[:, :lead] == 9).all() and (buf[:, lead + (Hq + Hk) * D:] == 9).all()


def test_rope_heads_in_another_order_and_wide_table_rows(handle):
    """Head-major storage ([H, T, D] seen as [T, H, D]) on both sides, table rows of a wider table."""
    q, k, wq, wk, pos = _qk(20, 4, 2, 64, 1)
    wide = torch.full((50, 70), float("nan"))
    wide[:, 3:67] = _table(50, 64)
    qh = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    kh = k.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    qo = torch.empty((4, 20, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ko = torch.empty((2, 20, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    pkg.moe_lora_qk_norm_rope(handle, qh, kh, wq.cuda(), wk.cuda(), wide.cuda()[:, 3:67], pos.cuda(), q_out=qo, k_out=ko)
    _near(qo, ref.norm_rope(q, wq, wide[:, 3:67], pos, 1e-6, False))
    _near(ko, ref.norm_rope(k, wk, wide[:, 3:67], pos, 1e-6, False))


def test_rope_zero_heads_rows_and_values(handle):
    q, k, wq, wk, pos = _qk(5, 3, 2, 64, 1)
    table = _table(50, 64)
    dev = [t.cuda() for t in (q, k, wq, wk, table, pos)]
    qo, ko = pkg.moe_lora_qk_norm_rope(handle, dev[0][:, :0], dev[1], *dev[2:])
    assert qo.shape == (5, 0, 64)
    _near(ko, ref.norm_rope(k, wk, table, pos, 1e-6, False))
    qo, ko = pkg.moe_lora_qk_norm_rope(handle, dev[0][:0], dev[1][:0], *dev[2:5], dev[5][:0])
    assert qo.shape == (0, 3, 64) and ko.shape == (0, 2, 64)
    qo, _ = pkg.moe_lora_qk_norm_rope(handle, torch.zeros_like(dev[0]), *dev[1:])      # eps keeps a zero head at zero
    assert (qo == 0).all()
    dev[0][2, 1, 3] = float("nan")                                                     # stays in its own head
    qo, _ = pkg.moe_lora_qk_norm_rope(handle, *dev)
    bad = torch.isnan(qo).any(2).nonzero().tolist()
    assert bad == [[2, 1]]


def test_rope_position_out_of_range_is_reported_and_not_rotated(handle):
    q, k, wq, wk, pos = _qk(70, 3, 2, 64, 8)
    table = _table(50, 64)
    ws = pkg.alloc_qk_norm_rope_workspace()
    for pt, bad in ((torch.int32, 50), (torch.int32, -1), (torch.int64, 2 ** 40)):
        p = pos.to(pt)
        p[66] = bad
        qo, ko = pkg.moe_lora_qk_norm_rope(handle, q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), table.cuda(), p.cuda(), workspace=ws)
        assert pkg.moe_lora_check_status(ws)[0] == 6
        _near(qo, ref.norm_rope(q, wq, table, p, 1e-6, False))
        p[66] = 1
        pkg.moe_lora_qk_norm_rope(handle, q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), table.cuda(), p.cuda(), workspace=ws)
        assert pkg.moe_lora_check_status(ws)[0] == 0


def test_rope_large_offsets(handle):
    """Tokens past 2^31 elements of the input."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    q, k, wq, wk, pos = _qk(3, 2, 1, 64, 4)
    table = _table(50, 64)
    pitch = (1 << 30) + 8
    buf = torch.empty(2 * pitch + 128, dtype=torch.bfloat16, device="cuda")
    qs = buf.as_strided((3, 2, 64), (pitch, 64, 1))
    qs.copy_(q)
    qo, _ = pkg.moe_lora_qk_norm_rope(handle, qs, k.cuda(), wq.cuda(), wk.cuda(), table.cuda(), pos.cuda())
    _near(qo, ref.norm_rope(q, wq, table, pos, 1e-6, False))


def test_rope_graph_replay(handle):
    q, k, wq, wk, pos = _qk(11, 4, 2, 64, 2)
    table = _table(50, 64)
    d = [t.cuda() for t in (q, k, wq, wk, table, pos)]
    outs = torch.empty_like(d[0]), torch.empty_like(d[1])
    pkg.moe_lora_qk_norm_rope(handle, *d, q_out=outs[0], k_out=outs[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.moe_lora_qk_norm_rope(handle, *d, q_out=outs[0], k_out=outs[1])
    q2, _, _, _, pos2 = _qk(11, 4, 2, 64, 3)
    d[0].copy_(q2)
    d[5].copy_(pos2)
    graph.replay()
    torch.cuda.synchronize()
    _near(outs[0], ref.norm_rope(q2, wq, table, pos2, 1e-6, False))


def test_rope_refusals(handle):
    q, k, wq, wk, pos = (t.cuda() for t in _qk(4, 2, 1, 64, 1))
    table = _table(50, 64).cuda()
    f = lambda *a, **kw: pkg.moe_lora_qk_norm_rope(handle, *a, **kw)
    n = handle.launch_count()
    for bad in (lambda: f(q.float(), k, wq, wk, table, pos), lambda: f(q, k[:3], wq, wk, table, pos),
                lambda: f(q, k[:, :, :32], wq, wk, table, pos), lambda: f(q, k, wq[:32], wk, table, pos),
                lambda: f(q, k, wq.bfloat16(), wk, table, pos), lambda: f(q, k, wq, wk, table.half(), pos),
                lambda: f(q, k, wq, wk, table, pos.float()), lambda: f(q, k, wq, wk, table, pos[:2]),
                lambda: f(q.cpu(), k, wq, wk, table, pos), lambda: f(q.transpose(1, 2), k, wq, wk, table, pos),
                lambda: f(q, k, wq, wk, table, pos, q_out=torch.empty_like(k))):
        with pytest.raises(ValueError):
            bad()
    codes = []
    big = torch.zeros((1, 1, 514), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(514, device="cuda")
    for bad in (lambda: f(q, k, wq, wk, table[:, :63], pos), lambda: f(q, k, wq, wk, _table(50, 66).cuda(), pos),
                lambda: f(big, big, w, w, table, pos[:1]), lambda: f(q, k, wq, wk, table, pos, eps=-1.0),
                lambda: f(q, k, wq, wk, table, pos, workspace=torch.zeros(2, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pkg.MoELoRAError) as e:
            bad()
        codes.append(e.value.status)
    assert codes == [1, 1, 2, 1, 3]
    assert handle.launch_count() == n
