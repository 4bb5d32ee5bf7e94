"""Every instance of moe_lora_linear's kernels, each by the shapes that the choice of tiles gives it."""
import numpy as np
import pytest
import torch

import block_reference as ref
import routed_moe_expert_gb300 as pkg
from test_gpu_linear import _case, _check, _run
from test_linear_choice import choice

RANKS = {0: (), 64: (16, 40), 128: (64, 48), 192: (64, 64, 64), 512: (64,) * 8}

# (kernel, token tile or weight rows, 64-row blocks of the stacked A (cluster), float32, adapters, K shared by several
# CTAs or pairs, several accumulators (narrow, cluster) or shrink slices (wide)), (T, N, K, float32, stacked ranks)
INSTANCES = [
    (('cluster', 16, 1, False, True, False, False), (1217, 9, 136, False, 64)),
    (('cluster', 16, 1, False, True, True, False), (5, 81, 1408, False, 64)),
    (('cluster', 16, 1, True, True, False, False), (1257, 11, 136, True, 64)),
    (('cluster', 16, 1, True, True, True, False), (3, 459, 280, True, 64)),
    (('cluster', 16, 1, True, True, True, True), (3, 13, 8416, True, 64)),
    (('cluster', 16, 2, False, True, False, False), (1255, 9, 144, False, 128)),
    (('cluster', 16, 2, False, True, True, False), (97, 29, 552, False, 128)),
    (('cluster', 16, 2, True, True, False, False), (1283, 9, 144, True, 128)),
    (('cluster', 16, 2, True, True, True, False), (1131, 13, 72, True, 128)),
    (('cluster', 16, 2, True, True, True, True), (147, 13, 8808, True, 128)),
    (('cluster', 32, 1, False, True, False, False), (4931, 9, 72, False, 64)),
    (('cluster', 32, 1, False, True, True, False), (1217, 9, 712, False, 64)),
    (('cluster', 32, 1, True, True, False, False), (4971, 9, 8, True, 64)),
    (('cluster', 32, 1, True, True, True, False), (611, 9, 1352, True, 64)),
    (('cluster', 32, 1, True, True, True, True), (309, 9, 8264, True, 64)),
    (('cluster', 32, 2, False, True, False, False), (6009, 9, 8, False, 128)),
    (('cluster', 32, 2, False, True, True, False), (635, 9, 792, False, 128)),
    (('cluster', 32, 2, True, True, False, False), (5667, 11, 8, True, 128)),
    (('cluster', 32, 2, True, True, True, False), (617, 9, 784, True, 128)),
    (('cluster', 32, 2, True, True, True, True), (307, 9, 8400, True, 128)),
    (('narrow', 128, 0, False, False, False, False), (6471, 589, 72, False, 0)),
    (('narrow', 128, 0, False, False, True, False), (5007, 9, 656, False, 0)),
    (('narrow', 128, 0, False, True, True, False), (997, 9, 4992, False, 512)),
    (('narrow', 128, 0, True, False, False, False), (6731, 261, 72, True, 0)),
    (('narrow', 128, 0, True, False, True, False), (5007, 11, 656, True, 0)),
    (('narrow', 128, 0, True, False, True, True), (2159, 9, 8744, True, 0)),
    (('narrow', 128, 0, True, True, False, False), (1303, 3155, 352, True, 64)),
    (('narrow', 128, 0, True, True, True, False), (443, 9, 4264, True, 512)),
    (('narrow', 128, 0, True, True, True, True), (417, 11, 8728, True, 512)),
    (('narrow', 16, 0, False, False, False, False), (9, 1093, 88, False, 0)),
    (('narrow', 16, 0, False, False, True, False), (1, 75, 1880, False, 0)),
    (('narrow', 16, 0, False, True, False, False), (9, 765, 128, False, 192)),
    (('narrow', 16, 0, False, True, True, False), (5, 25, 4136, False, 192)),
    (('narrow', 16, 0, True, False, False, False), (901, 17, 80, True, 0)),
    (('narrow', 16, 0, True, False, True, False), (59, 21, 1048, True, 0)),
    (('narrow', 16, 0, True, False, True, True), (1, 15, 8960, True, 0)),
    (('narrow', 16, 0, True, True, False, False), (1131, 13, 72, True, 192)),
    (('narrow', 16, 0, True, True, True, False), (1, 25, 5504, True, 512)),
    (('narrow', 16, 0, True, True, True, True), (1, 11, 11952, True, 128)),
    (('narrow', 32, 0, False, False, False, False), (2465, 9, 72, False, 0)),
    (('narrow', 32, 0, False, False, True, False), (1207, 9, 200, False, 0)),
    (('narrow', 32, 0, False, True, False, False), (97, 5067, 80, False, 512)),
    (('narrow', 32, 0, False, True, True, False), (253, 11, 648, False, 512)),
    (('narrow', 32, 0, True, False, False, False), (2561, 9, 72, True, 0)),
    (('narrow', 32, 0, True, False, True, False), (1187, 9, 232, True, 0)),
    (('narrow', 32, 0, True, False, True, True), (309, 9, 8592, True, 0)),
    (('narrow', 32, 0, True, True, False, False), (67, 7763, 72, True, 512)),
    (('narrow', 32, 0, True, True, True, False), (255, 9, 704, True, 512)),
    (('narrow', 32, 0, True, True, True, True), (181, 9, 8400, True, 192)),
    (('narrow', 64, 0, False, False, False, False), (5013, 9, 328, False, 0)),
    (('narrow', 64, 0, False, False, True, False), (711, 9, 784, False, 0)),
    (('narrow', 64, 0, False, True, False, False), (6903, 9, 528, False, 128)),
    (('narrow', 64, 0, False, True, True, False), (143, 9, 1416, False, 512)),
    (('narrow', 64, 0, True, False, False, False), (4959, 9, 336, True, 0)),
    (('narrow', 64, 0, True, False, True, False), (619, 13, 784, True, 0)),
    (('narrow', 64, 0, True, False, True, True), (611, 11, 8968, True, 0)),
    (('narrow', 64, 0, True, True, False, False), (6415, 15, 152, True, 192)),
    (('narrow', 64, 0, True, True, True, False), (131, 9, 1408, True, 512)),
    (('narrow', 64, 0, True, True, True, True), (97, 9, 8456, True, 512)),
    (('wide', 128, 0, False, False, False, False), (4941, 141, 200, False, 0)),
    (('wide', 128, 0, False, False, True, False), (5007, 9, 11192, False, 0)),
    (('wide', 128, 0, False, True, False, False), (985, 15, 80, False, 512)),
    (('wide', 128, 0, False, True, False, True), (4869, 9, 536, False, 128)),
    (('wide', 128, 0, False, True, True, False), (6519, 11, 1376, False, 512)),
    (('wide', 128, 0, False, True, True, True), (2541, 9, 2584, False, 128)),
    (('wide', 128, 0, True, False, False, False), (5125, 153, 200, True, 0)),
    (('wide', 128, 0, True, False, True, False), (4497, 9, 4384, True, 0)),
    (('wide', 128, 0, True, True, False, False), (1351, 9, 72, True, 512)),
    (('wide', 128, 0, True, True, False, True), (5021, 11, 520, True, 128)),
    (('wide', 128, 0, True, True, True, False), (951, 9, 6144, True, 512)),
    (('wide', 128, 0, True, True, True, True), (1105, 9, 4128, True, 64)),
    (('wide', 192, 0, False, False, False, False), (6869, 261, 80, False, 0)),
    (('wide', 192, 0, False, True, False, False), (4185, 9, 72, False, 512)),
    (('wide', 192, 0, False, True, False, True), (5187, 129, 584, False, 128)),
    (('wide', 256, 0, False, False, False, False), (265, 7743, 80, False, 0)),
    (('wide', 256, 0, False, False, True, False), (5021, 131, 2472, False, 0)),
    (('wide', 256, 0, False, True, False, False), (5869, 9, 8, False, 512)),
    (('wide', 256, 0, False, True, False, True), (5251, 201, 520, False, 64)),
    (('wide', 256, 0, False, True, True, False), (6847, 175, 1480, False, 512)),
    (('wide', 256, 0, False, True, True, True), (2809, 131, 3760, False, 64)),
]


def _instance(T, N, K, f32, Rs):
    c = choice(T, N, K, f32, Rs)
    kind = ("narrow", "wide", "cluster")[c["kernel"]]
    return (kind, c["rows"] if kind == "wide" else c["tokens"], 1 + (Rs > 64) if kind == "cluster" else 0, f32, Rs > 0,
            c["split"] > 1, c["accs"] > 1 or c["slices"] > 1)


def test_the_shapes_reach_their_instances(built_lib):
    """A change of the choice's constants that moves a shape has to bring another shape for the instance."""
    off = [(want, shape, _instance(*shape)) for want, shape in INSTANCES if _instance(*shape) != want]
    assert not off, off
    kernels = {k[:4] + k[6:] for k, _ in INSTANCES}
    assert len(INSTANCES) == len({k for k, _ in INSTANCES}) and len(kernels) >= 30


@pytest.fixture(scope="module")
def handle():
    h = pkg.Handle(0)
    yield h
    h.close()


def _id(v):
    return "-".join(str(int(x) if isinstance(x, bool) else x) for x in v)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [s for _, s in INSTANCES], ids=_id)
def test_against_the_definition(handle, shape):
    T, N, K, f32, Rs = shape
    c = _case(T, N, K, RANKS[Rs], seed=T + N + K, bias=N % 3 == 0)
    got = _run(handle, c, f32)
    _check(got, c, f32)
    assert torch.equal(got, _run(handle, c, f32))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [s for _, s in INSTANCES if s[3] and s[4]], ids=_id)
def test_all_24_bits_of_a_shrunk_value(handle, shape):
    """Rows of x and of A with one nonzero value each, so that u is a product of 16 bits times a factor,
    rounded to a float32; w is 0 and a row of B has one power of two.  A float32 result is that u times it, to
    the bit: a lost piece of u would show at 2^-8 or 2^-16."""
    T, N, K, _, Rs = shape
    ranks = RANKS[Rs]
    g = torch.Generator().manual_seed(K)
    S, R = len(ranks), max(ranks)
    k0 = min(K - 1, 5 + K // 2)
    x = torch.zeros((T, K), dtype=torch.bfloat16)
    A = torch.zeros((S, R, K), dtype=torch.bfloat16)
    B = torch.zeros((S, N, R), dtype=torch.bfloat16)
    x[:, k0] = (1 + torch.rand(T, generator=g)).bfloat16()
    A[:, :, k0] = (1 + torch.rand((S, R), generator=g)).bfloat16() * torch.randint(0, 2, (S, R), generator=g).mul(2).sub(1).bfloat16()
    at = torch.stack([torch.arange(N) % r for r in ranks])
    power = 2.0 ** torch.randint(-6, 7, (S, N), generator=g)
    B.scatter_(2, at[:, :, None], power[:, :, None].bfloat16())
    scalings = [float(np.float32(1 / 3 + s)) for s in range(S)]
    slots = torch.randint(-1, S, (T,), generator=g, dtype=torch.int32)
    ad = pkg.moe_lora_linear_adapters(handle, A.cuda(), B.cuda(), list(ranks), scalings)
    got = pkg.moe_lora_linear(handle, x.cuda(), torch.zeros((N, K), dtype=torch.bfloat16, device="cuda"), ad, slots.cuda(),
                              out_dtype=torch.float32).cpu().numpy()
    want = np.zeros((T, N), np.float32)
    for s in range(S):
        rows = np.nonzero(slots.numpy() == s)[0]
        product = x[rows, k0].float().numpy()[:, None] * A[s, :, k0].float().numpy()[None]      # exact: 16 bits
        u = np.float32(scalings[s]) * product
        want[rows] = u[:, at[s].numpy()] * power[s].numpy()[None]
    np.testing.assert_array_equal(got, want)
