"""Whole-number inputs and the comparison for sums that fp32 holds exactly."""

import torch


def whole(shape, seed):
    """bf16 whole numbers between -2 and 2."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, dtype=torch.int8).to(torch.bfloat16)


def bf16_of(t):
    """64-bit whole numbers below 2^24, rounded once to bf16 (fp32 holds them, so the first step rounds nothing)."""
    assert float(t.abs().max()) < 2.0**24 if t.numel() else True
    return t.float().to(torch.bfloat16)


def same(got, want, what):
    """Equal elementwise (0 equals -0)."""
    bad = got != want
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d differ; first at %s: got %g, want %g" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i])))
