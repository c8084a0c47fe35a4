"""GPU tests of the row quantisers in buffers of more rows than the experts have: the
other rows are not read (a call takes as long as on a buffer of the experts' rows
alone), and rows past the first that each workgroup takes are right."""

import pytest
import torch

import _experts_8bit as E8
import mixture_experts_token_amd as moe
from _parity import POISON, poisoned

pytestmark = pytest.mark.gpu

QUANTIZE = {"int8": moe.moe_quantize_rows_int8, "fp8": moe.moe_quantize_rows_fp8}
CODE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}


def least_us(call):
    """Least time of a call among others, of five times ten."""
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        call()
        a.record()
        for _ in range(10):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("rows,n,dtype", [(65536, 7168, torch.bfloat16), (32768, 16384, torch.bfloat16),
                                          (200000, 1024, torch.float32)])
def test_other_rows_cost_nothing(hip_device, kind, rows, n, dtype):
    """A buffer of some 0.8 GB or more, which takes at least 100 us to read at the card's 8 TB/s, with 64
    rows of experts: within 30 us of what these rows take alone."""
    dev, live = hip_device, 64
    assert rows * n * torch.empty(0, dtype=dtype).element_size() / 8e12 > 100e-6
    x = torch.ones((rows, n), dtype=dtype, device=dev)
    codes, scale = torch.empty((rows, n), dtype=CODE[kind], device=dev), torch.empty(rows, device=dev)
    off = torch.arange(0, live + 1, 2, device=dev)
    whole = least_us(lambda: QUANTIZE[kind](x, codes, scale, expert_first_token_offset=off))
    alone = least_us(lambda: QUANTIZE[kind](x[:live], codes[:live], scale[:live], expert_first_token_offset=off))
    print("[case] %s %d x %d: %.1f us, alone %.1f us" % (kind, rows, n, whole, alone), flush=True)
    assert whole < alone + 30


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("rows,live,n", [(20000, 17001, 4104), (30000, 8193, 16384), (9000, 9000, 32768),
                                         (30000, 200, 16384)])
def test_rows_behind_the_first_of_a_workgroup(hip_device, kind, rows, live, n):
    dev = hip_device
    print("[case] %s %d of %d x %d" % (kind, live, rows, n), flush=True)
    g = torch.Generator(device=dev).manual_seed(live)
    x = torch.randn((rows, n), generator=g, device=dev, dtype=torch.bfloat16)
    x *= torch.exp(torch.randn((rows, 1), generator=g, device=dev)).to(torch.bfloat16)
    codes, scale = poisoned((rows, n), torch.uint8, dev), poisoned((rows,), torch.float32, dev)
    off = torch.tensor([0, live // 3, live // 3, live], device=dev)
    QUANTIZE[kind](x, codes.view(CODE[kind]), scale, expert_first_token_offset=off)
    torch.cuda.synchronize()
    for lo, hi in ((0, 20), (8182, 8202), (16380, 16390), (live - 20, live)):
        lo, hi = min(lo, live), min(hi, live)
        if lo == hi:
            continue
        want, want_scale = E8.codes_of(x[lo:hi].cpu(), kind)
        assert torch.equal(codes[lo:hi].cpu(), want.view(torch.uint8)) and torch.equal(scale[lo:hi].cpu(), want_scale)
    for t in (codes[live:], scale[live:]):
        assert bool((t.view(torch.uint8) == POISON).all())
