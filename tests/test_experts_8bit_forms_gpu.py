"""GPU parity of the 8-bit layers where large tiles run many steps, where light
remainders are taken by a launch of small tiles of their own or stay with the large
ones, and where the buffers have at most a row per expert.  Which form a shape takes
is checked on the host (test_experts_8bit_tiles_host.py)."""

import pytest
import torch

import _experts_8bit as E8
from _parity import poisoned
from test_experts_8bit_gpu import (BF16, LAYER, assert_untouched, offsets, rand_codes, rand_scale, randn, row_codes)

pytestmark = pytest.mark.gpu

# (rows of each expert, rows of the buffers, n, k)
FORMS = [
    ([1024, 1025, 1134, 1023], 4209, 3960, 2064),   # remainders apart: a third of the experts' in small tiles
    ([1024, 768, 1024, 1280], 5000, 2000, 2064),    # asked for, but no remainder
    ([1024, 1025, 1134, 1023], 4209, 2200, 2064),   # asked for, but the large ones have room
    ([3000], 3000, 4096, 4112),                     # one expert, 33 steps
    ([1700, 40, 0, 1900, 256], 3899, 3000, 4624),   # few rows per expert on average, long tiles
    # up to one row per expert in the buffers (single tokens), also where one has more
    ([1], 1, 8, 16),
    ([1, 0, 1, 0, 0, 2, 1, 0], 8, 520, 2064),
    ([1] * 8, 8, 1032, 8208),
    ([0, 9, 0, 0, 1, 0, 5, 0, 0, 0, 0, 0, 0, 0, 1, 0], 16, 200, 528),
    ([0, 1, 0] + [0] * 20 + [17] + [0] * 40, 64, 72, 1104),
    ([1] * 1024, 1024, 40, 64),
]


def _id(v):
    return "rows%d-%dx%d" % (sum(v[0]), v[2], v[3])


def buffers(counts, rows, k, kind, seed, dev):
    """Codes and scales of `rows` rows; those behind the experts' have NaN scales."""
    x, xs = row_codes([rows], k, kind, seed, dev)
    xs[sum(counts):] = float("nan")
    return x[:rows], xs[:rows]


@pytest.mark.parametrize("shape", FORMS, ids=_id)
@pytest.mark.parametrize("kind,act", [("int8", "none"), ("fp8", "silu")])
def test_gated(hip_device, shape, kind, act):
    counts, rows, n, k = shape
    dev, m, e = hip_device, sum(shape[0]), len(shape[0])
    print("[case] gated %s %s" % (kind, _id(shape)), flush=True)
    off = offsets(counts, dev)
    x, xs = buffers(counts, rows, k, kind, 1, dev)
    w, ws = rand_codes((e, 2 * n, k), kind, 3, dev), rand_scale((e, 2 * n), 4, dev, 0.02 * k**-0.5)
    h = poisoned((rows, n), BF16, dev)
    LAYER["gated", kind](x, xs, w, ws, off, h, activation=act)
    torch.cuda.synchronize()
    E8.check_gated(x, xs, w, ws, off, kind, act, h)
    assert_untouched(h[m:], "h behind the last expert")


@pytest.mark.parametrize("shape", FORMS, ids=_id)
@pytest.mark.parametrize("kind,act,whole", [("int8", "gelu_tanh", True), ("fp8", "none", False)])
def test_linear(hip_device, shape, kind, act, whole):
    counts, rows, n, k = shape
    dev, m, e = hip_device, sum(shape[0]), len(shape[0])
    print("[case] linear %s %s" % (kind, _id(shape)), flush=True)
    off = offsets(counts, dev)
    x, xs = buffers(counts, rows, k, kind, 5, dev)
    w, ws = rand_codes((e, n, k), kind, 7, dev), rand_scale((e, n), 8, dev, 0.02 * k**-0.5)
    b = randn((e, n), 9, dev) if whole else None
    r = randn((rows, n), 10, dev) if whole else None
    y = poisoned((rows, n), BF16, dev)
    LAYER["linear", kind](x, xs, w, ws, off, y, bias=b, residual=r, activation=act)
    torch.cuda.synchronize()
    E8.check_linear(x, xs, w, ws, b, r, off, kind, act, y)
    assert_untouched(y[m:], "y behind the last expert")


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_every_sum_is_whole(hip_device, kind):
    """Codes up to 8 with scales of one: sums that fp32 holds exactly in both launches."""
    counts, rows, n, k = FORMS[0]
    dev, m, e = hip_device, sum(counts), len(counts)
    off = offsets(counts, dev)
    g = torch.Generator(device="cpu").manual_seed(11)
    code = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    x = torch.randint(-8, 9, (rows, k), generator=g, dtype=torch.int32).float()
    w = torch.randint(-8, 9, (e, n, k), generator=g, dtype=torch.int32).float()
    y = poisoned((rows, n), BF16, dev)
    LAYER["linear", kind](x.to(code).to(dev), torch.ones(rows, device=dev), w.to(code).to(dev),
                          torch.ones((e, n), device=dev), off, y)
    torch.cuda.synchronize()
    lo = 0
    for i, c in enumerate(counts):
        want = x[lo:lo + c] @ w[i].t()  # whole numbers up to 64 k < 2^18, exact in any order
        assert torch.equal(y[lo:lo + c].cpu(), want.to(BF16)), i
        lo += c
    assert_untouched(y[m:], "y behind the last expert")
