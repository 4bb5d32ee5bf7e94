"""moe_lora_attention near float32's end: values of up to 1e37 under scores that rise or fall along the keys, whose
weights relative to the first keys' would be millions."""
import pytest

from test_gpu_paged import _attention, handle  # noqa: F401

pytestmark = pytest.mark.gpu


def _slope(rise, lens, size=3e36):
    """Scores that change by `rise` from a request's first key to its last, and values of about `size`."""
    def tamper(q, kc, vc, tables):
        page = kc.shape[2]
        q.mul_(0.1)
        q[:, :, 0] = 1.0
        for row, (n, _) in zip(tables, lens):
            for i in range(n):
                kc[row[i // page], :, i % page, 0] = rise * i / n
                vc[row[i // page], :, i % page] *= size
    return tamper


@pytest.mark.parametrize("rise", [18.0, 40.0, -30.0])
@pytest.mark.parametrize("Hq,Hk,D,m", [(4, 1, 128, 1), (8, 1, 64, 2), (2, 2, 128, 40), (4, 2, 64, 30), (3, 1, 96, 200), (2, 1, 192, 3)])
def test_large_values_of_rising_scores(handle, rise, Hq, Hk, D, m):  # noqa: F811
    lens = [(700, m), (m + 250, m), (m, m)]
    _attention(handle, lens, Hq, Hk, D, 16, scale=1.0, garbage=False, tamper=_slope(rise, lens))


@pytest.mark.parametrize("m", [1, 40])
def test_large_values_in_pieces(handle, m):  # noqa: F811
    """Cut items: every piece has a reference of its own."""
    lens = [(9000, m)]
    _attention(handle, lens, 4, 1, 64, 32, scale=1.0, garbage=False, tamper=_slope(60.0, lens))


@pytest.mark.parametrize("rise", [25.0, -25.0])
@pytest.mark.parametrize("m", [1, 9])
def test_large_values_behind_a_shared_prefix(handle, rise, m):  # noqa: F811
    lens = [(1024 + 40 * i + m, m) for i in range(5)]

    def tamper(q, kc, vc, tables):
        vc.mul_(3e36)
        _slope(rise, lens, 1.0)(q, kc, vc, tables)   # (the shared pages as the last request has them)

    _attention(handle, lens, 8, 2, 64, 32, shared=1024, scale=1.0, garbage=False, tamper=tamper)
