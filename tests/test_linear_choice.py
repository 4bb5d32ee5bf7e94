"""The choice of kernel and tiles of moe_lora_linear, on the host alone."""
import ctypes

import pytest

from routed_moe_expert_gb300 import binding as B

SMS, PAIRS_BY_TWO = 152, 72     # a GB300: its SMs, and the pairs that run at a time in clusters of two
NARROW, WIDE, CLUSTER = 0, 1, 2


def choice(T, N, K, f32=False, Rs=0, sms=SMS, by_two=PAIRS_BY_TWO):
    out = (ctypes.c_int32 * 6)()
    B.lib().mlk_linear_choice(T, N, K, int(f32), Rs, sms, by_two, out)
    return dict(zip(("kernel", "tokens", "rows", "split", "accs", "slices"), out))


def test_the_device_of_the_call_decides(built_lib):
    """Two pairs share a tile where the call's own device has the pairs for it, whatever devices other
    handles of the process are on."""
    small = choice(512, 4096, 7168, by_two=30)
    assert choice(512, 4096, 7168)["split"] == 2 and small["split"] == 1 and small["kernel"] == WIDE
    assert choice(512, 4096, 7168) == choice(512, 4096, 7168)
