"""moe_lora_qk_norm_rope with infinities and NaN: a value that is not rotated depends on itself and on
the head's scale alone."""
import numpy as np
import pytest
import torch

import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def handle():
    return pkg.Handle(0)


def _definition(x, w, table, pos, interleaved):
    """In 64 bits; 1 / sqrt(inf) is 0."""
    x, w, table = x.double().numpy(), w.double().numpy(), table.double().numpy()
    R = table.shape[1]
    with np.errstate(all="ignore"):
        n = x / np.sqrt((x * x).mean(2, keepdims=True) + 1e-6) * w
        y = n.copy()
        for t, p in enumerate(pos.tolist()):
            if 0 <= p < table.shape[0]:
                c, s = table[p, :R // 2], table[p, R // 2:]
                a = slice(0, R, 2) if interleaved else slice(0, R // 2)
                b = slice(1, R, 2) if interleaved else slice(R // 2, R)
                y[t, :, a], y[t, :, b] = n[t, :, a] * c - n[t, :, b] * s, n[t, :, b] * c + n[t, :, a] * s
    return y


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,R", [(64, 32), (128, 64), (192, 64), (256, 128), (80, 40), (96, 16), (64, 64), (128, 0), (512, 256)])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_values_that_are_not_rotated_keep_to_themselves(handle, D, R, interleaved, value):
    T, H = 6, 3
    g = torch.Generator().manual_seed(D + R)
    q = torch.randn((T, H, D), generator=g).bfloat16()
    k = torch.randn((T, 1, D), generator=g).bfloat16()
    wq, wk = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    a = torch.rand((20, R // 2), generator=g) * 6.3
    table = torch.cat([a.cos(), a.sin()], 1)
    pos = torch.randint(0, 20, (T,), generator=g, dtype=torch.int32)
    pos[4] = 99                                   # out of range: normed and not rotated
    q[1, 1, D - 3] = value                        # in a head, past its rotated values (R < D)
    q[4, 2, 1] = value
    wq[D - 1] = value                             # in a weight: that value of every head
    if R == D:
        wq[D - 1] = 1.0
    dev = [t.cuda() for t in (q, k, wq, wk, table, pos)]
    for out, x, w in zip(pkg.moe_lora_qk_norm_rope(handle, *dev, interleaved=interleaved), (q, k), (wq, wk)):
        got, want = out.float().cpu().numpy(), _definition(x, w, table, pos, interleaved)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        np.testing.assert_array_equal(np.isinf(got), np.isinf(want))
        fin = np.isfinite(want)
        # a rotated value is a sum of two products of at most 3 roundings each, rounded to bf16
        np.testing.assert_allclose(got[fin], want[fin], rtol=2.0 ** -8, atol=1e-5 + (D + 24) * 2.0 ** -23 * 8)
