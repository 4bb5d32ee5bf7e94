"""Calls of the operators around the layer on a stream of the caller's naming: what they allocate is
not memory that the current stream's work still uses."""
import pytest
import torch

import routed_moe_expert_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = pkg.Handle(0)
    yield h
    h.close()


def _calls(handle):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    T = 512
    x, w = r(T, 256).bfloat16(), (r(384, 256) / 16).bfloat16()
    A, B = (r(2, 16, 256) / 16).bfloat16(), r(2, 384, 16).bfloat16()
    ad = pkg.moe_lora_linear_adapters(handle, A, B, [16, 8], [1.0, 2.0])
    slots = torch.randint(-1, 2, (T,), generator=g, device="cuda").int()
    z, q = r(T, 64), r(T, 6, 64).bfloat16()
    table, pos = r(T, 64), torch.arange(T, device="cuda", dtype=torch.int32)
    one = torch.ones(64, device="cuda")
    return {
        "select": lambda **k: [pkg.moe_lora_select_experts(handle, z, 8, packed=True, **k)[n]
                               for n in ("topk_ids", "topk_weights", "packed_topk_ids")],
        "linear": lambda **k: [pkg.moe_lora_linear(handle, x, w, ad, slots, **k)],
        "adapters": lambda **k: [pkg.moe_lora_linear_adapters(handle, A, B, [16, 8], [1.0, 2.0], **k).packed],
        "rope": lambda **k: list(pkg.moe_lora_qk_norm_rope(handle, q, q[:, :2], one, one, table, pos, **k))}


@pytest.mark.parametrize("what", ["select", "linear", "adapters", "rope"])
@pytest.mark.parametrize("as_number", [False, True])
def test_memory_freed_on_the_current_stream_is_not_taken(handle, what, as_number):
    call = _calls(handle)[what]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of every size that the call asks for, still to be written by the current stream when they are freed
    sizes = [512, 1 << 14, 1 << 15, 1 << 16, 1 << 17, 1 << 18, 1 << 19, 1 << 20, 1 << 21, 1 << 22]
    sizes += [t.numel() * t.element_size() for t in want]
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda._sleep(40_000_000)
    for t in held:
        t.fill_(255)
    del held, t
    got = call(stream=side.cuda_stream if as_number else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_are_the_callers_after_a_wait(handle):
    """The current stream may go on with a result once it has waited; freed, it is not handed out again
    before that is done."""
    call = _calls(handle)["linear"]
    want = call()[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(40_000_000)
    copy = y.clone()
    del y
    with torch.cuda.stream(side):
        other = [torch.full_like(want, 9.0) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(other) == 8


@pytest.mark.parametrize("named", [False, True])
def test_adapters_let_go_of_while_another_stream_reads_them(handle, named):
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, w = r(64, 256).bfloat16(), (r(384, 256) / 16).bfloat16()
    A, B = (r(2, 16, 256) / 16).bfloat16(), r(2, 384, 16).bfloat16()
    slots = torch.randint(-1, 2, (64,), generator=g, device="cuda").int()
    make = lambda: pkg.moe_lora_linear_adapters(handle, A, B, [16, 8], [1.0, 2.0])
    want = pkg.moe_lora_linear(handle, x, w, make(), slots).clone()
    ad, side = make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
        if not named:
            got = pkg.moe_lora_linear(handle, x, w, ad, slots)
    if named:
        got = pkg.moe_lora_linear(handle, x, w, ad, slots, stream=side)
    n = ad.packed.numel()
    del ad
    torch.cuda._sleep(1_000_000)
    others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(others) == 4
