"""Sizes and scales at the ends of what moe_lora_attention takes, on the host: its checks come before an empty batch
returns, which launches nothing."""
import pytest

from test_paged_abi import ATTEND, FAKE, AttentionArgs, _call


@pytest.mark.parametrize("width,page,code", [
    (2 ** 27 - 512, 16, 0), (2 ** 27 - 511, 16, 1), (2 ** 27 - 1, 16, 1), (1, 2 ** 31 - 8192, 0), (1, 2 ** 31 - 8191, 1),
    (2 ** 31 - 1, 1, 1), (2 ** 23 - 32, 256, 0), (2 ** 23 - 31, 256, 1)])
def test_keys_of_a_table(built_lib, width, page, code):
    """Key indices are rounded up to units and looked ahead of in 32 bits, so tables end 8192 keys below 2^31."""
    over = dict(T=0, B=1, width=width, stride=width, page=page, num_pages=1)
    assert _call("moe_lora_attention", AttentionArgs, ATTEND, over, ws=FAKE, nbytes=1 << 32) == code


@pytest.mark.parametrize("scale,code", [(2.3e38, 0), (-2.3e38, 0), (2.4e38, 1), (-3.4e38, 1), (0.0, 0), (1e-45, 0)])
def test_scale_times_log2_e_is_finite(built_lib, scale, code):
    """Weights are powers of two of scores times scale * log2(e)."""
    assert _call("moe_lora_attention", AttentionArgs, ATTEND, dict(T=0, scale=scale), ws=FAKE, nbytes=1 << 32) == code
