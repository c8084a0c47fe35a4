"""Long sums of the expert layers, to the last term.

Inputs are whole numbers between -2 and 2, so every product and, up to a
length of 2^21 (4 * 2^21 < 2^24 with a bias of at most 2), every partial sum
in any order is a whole number below 2^24, which fp32 holds exactly.  The one
rounding left is the output's, to bf16: results have to be equal, and a term
that is left out or taken twice shows (tests/test_experts_host_exact.py plants
such mistakes in the reference).
"""

import numpy as np
import pytest
import torch

from _exact import bf16_of, same, whole
from _parity import POISON, poisoned
import mixture_experts_token_amd as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TAIL = 3


def _say(msg):
    print("[case] " + msg, flush=True)


def rows_of(counts, cols, seed, dev):
    t = whole((sum(counts) + TAIL, cols), seed).to(dev)
    t[sum(counts):] = float("nan")
    return t


def offsets(counts, dev):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64, device=dev)


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == POISON).all())


def product(x, w, counts):
    """x[j] w[e]^T over each expert's rows, in 64 bits on the tensors' device."""
    out = torch.zeros(sum(counts), w.shape[1], dtype=torch.float64, device=x.device)
    at = 0
    for e, c in enumerate(counts):
        if c:
            out[at:at + c] = torch.mm(x[at:at + c].double(), w[e].double().t().contiguous())
        at += c
    return out


def outer(d, x, counts):
    """d[rows of e]^T x[rows of e], in 64 bits, in pieces of rows."""
    out = torch.zeros(len(counts), d.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    at = 0
    for e, c in enumerate(counts):
        for lo in range(at, at + c, 50000):
            rows = slice(lo, min(lo + 50000, at + c))
            out[e] += torch.mm(d[rows].double().t().contiguous(), x[rows].double())
        at += c
    return out


# (rows of each expert, n, k).  k: streamed with eight, four, two and one x row in
# LDS, and past what fits there (tiled); the longest and the shortest rows allowed
SHAPES = [
    ([1, 0, 2, 3, 0, 0, 0, 1], 40, 1096),
    ([1, 0, 2, 3, 0, 0, 0, 1], 72, 4104),
    ([1, 0, 2, 3, 0, 0, 0, 1], 72, 8200),
    ([0, 5, 1, 0, 0, 0, 0, 2], 136, 16392),
    ([0, 5, 1, 0, 0, 0, 0, 2], 136, 32768),
    ([2, 0, 1], 40, 33000),
    ([30, 1, 0], 136, 16392),
    ([300, 0, 270], 264, 8200),
    ([3], 8, 2**20),
    ([2, 1], 2**20, 8),
    ([200, 70], 2**15, 72),
    ([40, 0], 8, 2**20),
    ([40, 0], 2**20, 8),
]


def _id(v):
    return "rows%d-%dx%d" % (sum(v[0]), v[1], v[2])


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_linear(hip_device, shape):
    counts, n, k = shape
    _say("exact linear " + _id(shape))
    dev, m, e = hip_device, sum(counts), len(counts)
    off, x, w, b = offsets(counts, dev), rows_of(counts, k, 1, dev), whole((e, n, k), 2).to(dev), whole((e, n), 3).to(dev)
    y = poisoned((m + TAIL, n), BF16, dev)
    moe.moe_grouped_linear_bf16(x, w, off, y, bias=b)
    torch.cuda.synchronize()
    z = product(x, w, counts) + b.double().repeat_interleave(torch.tensor(counts, device=dev), 0)
    same(y[:m], bf16_of(z), "y")
    assert untouched(y[m:])


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_gated(hip_device, shape):
    counts, n, k = shape
    _say("exact gated " + _id(shape))
    dev, m, e = hip_device, sum(counts), len(counts)
    off, x, w = offsets(counts, dev), rows_of(counts, k, 1, dev), whole((e, 2 * n, k), 2).to(dev)
    h, keep = poisoned((m + TAIL, n), BF16, dev), poisoned((m + TAIL, 2 * n), BF16, dev)
    moe.moe_grouped_gated_gemm_bf16(x, w, off, h, gate_up=keep, activation="relu")
    torch.cuda.synchronize()
    z = product(x, w, counts)
    same(keep[:m], bf16_of(z), "gate_up")
    # h is the one product of two whole numbers in fp32, then bf16: both roundings as the kernel has them
    same(h[:m], (z[:, :n].clamp(min=0).float() * z[:, n:].float()).to(BF16), "h")
    assert untouched(h[m:]) and untouched(keep[m:])


@pytest.mark.parametrize("alone", [False, True], ids=["together", "alone"])
@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_linear_backward(hip_device, shape, alone):
    counts, n, k = shape
    _say("exact linear backward " + _id(shape))
    dev, m, e = hip_device, sum(counts), len(counts)
    off, x, w = offsets(counts, dev), rows_of(counts, k, 1, dev), whole((e, n, k), 2).to(dev)
    d_y = rows_of(counts, n, 4, dev)
    d_x, d_w, d_b = poisoned((m + TAIL, k), BF16, dev), poisoned((e, n, k), BF16, dev), poisoned((e, n), BF16, dev)
    if alone:
        for out in (dict(d_x=d_x), dict(d_w=d_w), dict(d_bias=d_b)):
            moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, **out)
    else:
        moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=d_x, d_w=d_w, d_bias=d_b)
    torch.cuda.synchronize()
    same(d_x[:m], bf16_of(product(d_y, w.transpose(1, 2), counts)), "d_x")
    same(d_w, bf16_of(outer(d_y, x, counts)), "d_w")
    ones = torch.ones(m, 1, dtype=BF16, device=dev)
    same(d_b, bf16_of(outer(d_y, ones, counts)[:, :, 0]), "d_bias")
    assert untouched(d_x[m:])


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_gated_backward(hip_device, shape):
    counts, n, k = shape
    _say("exact gated backward " + _id(shape))
    dev, m, e = hip_device, sum(counts), len(counts)
    off, x, w = offsets(counts, dev), rows_of(counts, k, 1, dev), whole((e, 2 * n, k), 2).to(dev)
    # gate and up between -1 and 1, so that their gradients stay between -2 and 2
    gate_up, d_h = rows_of(counts, 2 * n, 5, dev).clamp(-1, 1), rows_of(counts, n, 6, dev)
    d_gu, d_x = poisoned((m + TAIL, 2 * n), BF16, dev), poisoned((m + TAIL, k), BF16, dev)
    d_w = poisoned((e, 2 * n, k), BF16, dev)
    moe.moe_grouped_gated_gemm_backward_bf16(d_h, gate_up, x, w, off, d_gu, d_x=d_x, d_w=d_w, activation="relu")
    torch.cuda.synchronize()
    d, g, u = d_h[:m].float(), gate_up[:m, :n].float(), gate_up[:m, n:].float()
    want = torch.cat([d * u * (g > 0).float(), d * g.clamp(min=0)], 1).to(BF16)
    same(d_gu[:m], want, "d_gate_up")
    same(d_x[:m], bf16_of(product(want, w.transpose(1, 2), counts)), "d_x")
    same(d_w, bf16_of(outer(want, x, counts)), "d_w")
    assert untouched(d_gu[m:]) and untouched(d_x[m:])


def test_gradients_over_many_rows(hip_device):
    """600001 rows of 4096: elements pass 2^31, bytes 2^32, sums over 300000 rows."""
    counts, n, k, dev = [300000, 300001], 64, 4096, hip_device
    m = sum(counts)
    _say("exact gradients of %d rows of %d" % (m, k))
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randint(-2, 3, (m, k), generator=g, device=dev, dtype=torch.int8).to(BF16)
    d_y = torch.randint(-2, 3, (m, n), generator=g, device=dev, dtype=torch.int8).to(BF16)
    w, off = whole((2, n, k), 2).to(dev), offsets(counts, dev)
    y, d_x = poisoned((m, n), BF16, dev), poisoned((m, k), BF16, dev)
    d_w, d_b = poisoned((2, n, k), BF16, dev), poisoned((2, n), BF16, dev)
    moe.moe_grouped_linear_bf16(x, w, off, y)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=d_x, d_w=d_w, d_bias=d_b)
    torch.cuda.synchronize()
    same(d_w, bf16_of(outer(d_y, x, counts)), "d_w")
    same(d_b, bf16_of(torch.stack([t.double().sum(0) for t in d_y.split(counts)])), "d_bias")
    at = 0
    for e, c in enumerate(counts):
        wd = w[e].double()
        for lo in range(at, at + c, 50000):
            rows = slice(lo, min(lo + 50000, at + c))
            same(y[rows], bf16_of(torch.mm(x[rows].double(), wd.t().contiguous())), "y from row %d" % lo)
            same(d_x[rows], bf16_of(torch.mm(d_y[rows].double(), wd)), "d_x from row %d" % lo)
        at += c
