"""GPU tests of what the 8-bit layers' sums hold where experts have few rows: fp8
codes are multiplied and added as the numbers they stand for, in fp32, and no
product is cut beside a larger one.

Every expected output is known exactly and rounded once, and is compared for equality.
"""

import numpy as np
import pytest
import torch

import mixture_experts_token_amd as moe
from _parity import poisoned

pytestmark = pytest.mark.gpu

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn

# (rows of each expert, n, k): the forms for 4, 8 and 16 rows per pass, experts of
# several passes, waves that share a row, rows that end inside a step
STREAMED = [
    ([1], 40, 1104),
    ([1, 0, 1, 4], 200, 272),
    ([2, 1, 2, 3, 0, 2], 264, 2064),
    ([9, 1, 3, 8, 0, 4], 72, 1104),
    ([12] * 20, 136, 528),
    ([30, 1, 0, 1, 2, 1, 0, 1], 40, 16400),
]


def _id(shape):
    return "rows%d-%dx%d" % (sum(shape[0]), shape[1], shape[2])


def offsets(counts, dev):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64, device=dev)


def small_beside_large(counts, columns, k, seed):
    """(x, w, sums): in every eight codes two products of 2^16 that cancel and six of -1, 0 or 1."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randint(-1, 2, (sum(counts), k), generator=g).float()
    w = torch.randint(-1, 2, (len(counts), columns, k), generator=g).float()
    at = torch.arange(0, k, 8)
    a, b = at + torch.randint(0, 4, at.shape, generator=g), at + 4 + torch.randint(0, 4, at.shape, generator=g)
    x[:, a] = x[:, b] = 256.0
    w[:, :, a], w[:, :, b] = 256.0, -256.0
    sums = torch.cat([x[lo:lo + c] @ w[e].t() for e, (lo, c) in enumerate(zip(np.cumsum([0] + counts[:-1]), counts))])
    # a matrix instruction adds whole eights, up to eight of them: its partial sums are whole
    # numbers up to 2^20, and those from instruction to instruction as small as the last one
    assert float(sums.abs().max()) < 2**12  # a product of two of them is exact in fp32
    return x.to(FP8), w.to(FP8), sums


@pytest.mark.parametrize("shape", STREAMED, ids=_id)
def test_small_products_beside_large_ones_linear(hip_device, shape):
    counts, n, k = shape
    dev, m = hip_device, sum(counts)
    print("[case] linear %s" % _id(shape), flush=True)
    x, w, sums = small_beside_large(counts, n, k, 1)
    y = poisoned((m, n), BF16, dev)
    moe.moe_grouped_linear_fp8(x.to(dev), torch.ones(m, device=dev), w.to(dev), torch.ones(len(counts), n, device=dev),
                               offsets(counts, dev), y)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), sums.to(BF16))


@pytest.mark.parametrize("shape", STREAMED, ids=_id)
def test_small_products_beside_large_ones_gated(hip_device, shape):
    counts, n, k = shape
    dev, m = hip_device, sum(counts)
    print("[case] gated %s" % _id(shape), flush=True)
    x, w, sums = small_beside_large(counts, 2 * n, k, 2)
    h = poisoned((m, n), BF16, dev)
    moe.moe_grouped_gated_gemm_fp8(x.to(dev), torch.ones(m, device=dev), w.to(dev),
                                   torch.ones(len(counts), 2 * n, device=dev), offsets(counts, dev), h,
                                   activation="none")
    torch.cuda.synchronize()
    assert torch.equal(h.cpu(), (sums[:, :n] * sums[:, n:]).to(BF16))


@pytest.mark.parametrize("rows", [1, 2, 8])
def test_every_code_times_every_code(hip_device, rows):
    """x row r has code r in one place, w row c code c in every place: a product of two
    4-bit significands, which bf16 holds; a NaN code where either is one."""
    dev, n, k, experts = hip_device, 256, 528, 256 // rows
    x = torch.zeros((256, k), dtype=torch.uint8)
    x[torch.arange(256), torch.arange(256) * 37 % k] = torch.arange(256, dtype=torch.uint8)
    codes = torch.arange(256, dtype=torch.uint8)
    w = codes[None, :, None].repeat(experts, 1, k)
    y = poisoned((256, n), BF16, dev)
    moe.moe_grouped_linear_fp8(x.to(dev), torch.ones(256, device=dev), w.to(dev), torch.ones(experts, n, device=dev),
                               offsets([rows] * experts, dev), y)
    torch.cuda.synchronize()
    v = codes.view(FP8).float()
    want = v[:, None] * v[None, :]
    got = y.cpu().float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])
