"""The longest rows of the 8-bit layers: sums that cancel to -1, 0 or 1, so that a code
or a step of codes lost, read twice or taken from elsewhere shows in outputs that bf16
holds exactly.  (Sums near half the row's length do not show it: bf16's step there is
thousands.)  That such mistakes show is checked on the host.
"""

import pytest
import torch

import mixture_experts_token_amd as moe
from _parity import poisoned

LONGEST = {"int8": 131056, "fp8": 2**20}
CODE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
LINEAR = {"int8": moe.moe_grouped_linear_int8, "fp8": moe.moe_grouped_linear_fp8}
N = 40


def cancelling(kind):
    """(x [k], w [N, k]) of -1, 0 and 1: x has ones, then minus ones; w's halves are equal but for one code of a column."""
    k = LONGEST[kind]
    x = torch.ones(k, dtype=torch.int8)
    x[k // 2:] = -1
    g = torch.Generator(device="cpu").manual_seed(k)
    half = torch.randint(0, 2, (N, k // 2), generator=g, dtype=torch.int8)
    w = torch.cat([half, half], dim=1)
    ends = [0, 1, 15, 16, 31, 63, 64, 127, 128, 255, 256, 511, 512, 1023, 2047]
    at = ends + [k // 2 - 1, k // 2] + [k - 1 - i for i in ends] + [k // 4, k // 4 * 3]
    for c, i in enumerate(at):
        w[c, i] ^= 1  # the columns after these sum to 0
    return x, w


def sums(x, w):
    return (w.to(torch.int64) * x.to(torch.int64)).sum(1)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_mistakes_show(kind):
    x, w = cancelling(kind)
    k = x.numel()
    want = sums(x, w)
    assert int(want.abs().max()) == 1 and int((want == 0).sum()) == N - 34
    for length in (1, 8, 16, 32, 64, 128, 256, 512, 2048):
        for at in (0, k // 2 - length, k // 2, k - length):
            lost = w.clone()
            lost[:, at:at + length] = 0
            assert not torch.equal(sums(x, lost), want), ("lost", at, length)
        if length == 1:
            continue  # a neighbour's code may be the same
        for at, other in ((0, length), (k - length, k - 2 * length), (k // 2, k // 2 + length)):
            twice = w.clone()
            twice[:, at:at + length] = w[:, other:other + length]
            assert not torch.equal(sums(x, twice), want), ("read twice", at, length)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,rows", [([1], 1), ([1, 0, 1], 3), ([1, 2, 0, 1], 8), ([10, 0, 3], 30), ([40, 60], 100),
                                         ([300], 300), ([700, 0, 520], 1300)], ids=str)
@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_longest_rows(hip_device, kind, counts, rows):
    """Streamed in every form, small tiles, large tiles."""
    dev, e, m = hip_device, len(counts), sum(counts)
    print("[case] %s rows=%s of %d" % (kind, counts, rows), flush=True)
    x, w = cancelling(kind)
    k = x.numel()
    sign = torch.where(torch.arange(rows) % 3 == 1, -1.0, 1.0)
    codes = x.float().to(CODE[kind]).to(dev), (-x).float().to(CODE[kind]).to(dev)
    xs = torch.empty((rows, k), dtype=torch.uint8, device=dev)
    for j in range(rows):
        xs[j] = codes[int(sign[j] < 0)].view(torch.uint8)
    xs[m:] = 0x7F
    ws = w.float().to(CODE[kind]).to(dev).view(torch.uint8).expand(e, N, k).contiguous()
    shift = torch.arange(e)  # expert i has the columns in another order
    for i in range(e):
        ws[i] = ws[i].roll(int(shift[i]), 0)
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int64, device=dev)
    y = poisoned((rows, N), torch.bfloat16, dev)
    LINEAR[kind](xs.view(CODE[kind]), torch.ones(rows, device=dev), ws.view(CODE[kind]), torch.ones((e, N), device=dev),
                 off, y)
    torch.cuda.synchronize()
    want, lo = sums(x, w).float(), 0
    for i, c in enumerate(counts):
        assert torch.equal(y[lo:lo + c].cpu().float(), sign[lo:lo + c, None] * want.roll(i)), i
        lo += c
    assert bool((y[m:].view(torch.uint8) == 0xFF).all())
