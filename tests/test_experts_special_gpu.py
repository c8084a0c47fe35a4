"""GPU values and slopes of the expert layers' activations at zero, far out, at infinities and NaN.

An activation at an infinity is its limit (0 or infinity; slopes 0 or 1), in
every form of the forward (tiled, streamed) and of the backward.
"""

import math

import pytest
import torch

import _experts as X
from _parity import poisoned
import mixture_experts_token_amd as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF, NAN = math.inf, math.nan
ACTS = ["none", "relu", "silu", "gelu_tanh"]
VALS = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 3, -3, 12, -12, 29, -29, 31, -31, 90, -90, 1e4, -1e4, 1e20, -1e20,
        3e38, -3e38, INF, -INF, NAN, 1.0, -1.0, INF, NAN, -INF, 2.0, -2.0]


def value(z, act):
    """act(z) in 64 bits, its limit at an infinity."""
    v = X.act_value(torch.nan_to_num(z, nan=0.0, posinf=0.0, neginf=0.0), act)
    v = torch.where(z == INF, z, v)
    v = torch.where(z == -INF, z if act == "none" else torch.zeros_like(z), v)
    return torch.where(torch.isnan(z), z, v)


def slope(z, act):
    s = X.act_slope(torch.nan_to_num(z, nan=0.0, posinf=0.0, neginf=0.0), act)
    s = torch.where(z == INF, torch.ones_like(z), s)
    s = torch.where(z == -INF, torch.full_like(z, 1.0 if act == "none" else 0.0), s)
    if act in ("silu", "gelu_tanh"):  # relu: a NaN is not above 0, so its slope is 0
        s = torch.where(torch.isnan(z), z, s)
    return s


def check(got, ref, tol, what):
    """Equal where ref is an infinity or NaN, within tol elsewhere."""
    got = X.f64(got)
    wrong = int((torch.isnan(got) != torch.isnan(ref)).sum())
    assert wrong == 0, "%s: NaN or not, in the wrong place" % what
    far = torch.isinf(ref)
    wrong = int((got[far] != ref[far]).sum()) + int(torch.isinf(got[~far]).sum())
    assert wrong == 0, "%s: infinities" % what
    near = ~far & ~torch.isnan(ref)
    X.assert_within(got[near], ref[near], tol[near], what)


def zs(rows, dev):
    return torch.stack([torch.tensor(VALS).roll(i) for i in range(rows)]).to(BF16).to(dev)


@pytest.mark.parametrize("act", ACTS)
def test_linear_slopes(hip_device, act):
    z = zs(3, hip_device)
    d_y = torch.full_like(z, 0.75)
    n, off = z.shape[1], torch.tensor([0, 3], dtype=torch.int64, device=hip_device)
    w, d_x = torch.zeros(1, n, 8, dtype=BF16, device=hip_device), poisoned((3, 8), BF16, hip_device)
    if act == "none":  # the slope is 1 whatever z: d_x is the product of d_y itself
        w[0, :, 0] = 1.0
        moe.moe_grouped_linear_backward_bf16(d_y, None, w, off, d_x=d_x)
        torch.cuda.synchronize()
        assert d_x[:, 0].tolist() == [0.75 * n] * 3 and not d_x[:, 1:].any()
        return
    d_z = poisoned((3, n), BF16, hip_device)
    moe.moe_grouped_linear_backward_bf16(d_y, None, w, off, d_x=d_x, pre_activation=z, d_pre_activation=d_z,
                                         activation=act)
    torch.cuda.synchronize()
    ref = 0.75 * slope(X.f64(z), act)
    check(d_z, ref, X.HALF * ref.abs() + X.SLOPE * 0.75, "d_pre_activation")


@pytest.mark.parametrize("act", ACTS)
def test_gated_slopes(hip_device, act):
    g = zs(4, hip_device)
    n = g.shape[1]
    u = torch.tensor([1.5, -0.25, 4.0, -2.0], dtype=BF16, device=hip_device).view(4, 1).expand(4, n)
    gate_up = torch.cat([g, u], 1).contiguous()
    d_h = torch.full((4, n), 0.75, dtype=BF16, device=hip_device)
    off = torch.tensor([0, 4], dtype=torch.int64, device=hip_device)
    w = torch.zeros(1, 2 * n, 8, dtype=BF16, device=hip_device)
    d_gu = poisoned((4, 2 * n), BF16, hip_device)
    moe.moe_grouped_gated_gemm_backward_bf16(d_h, gate_up, None, w, off, d_gu, activation=act)
    torch.cuda.synchronize()
    g64, u64 = X.f64(g), X.f64(u)
    ref = 0.75 * u64 * slope(g64, act)
    check(d_gu[:, :n], ref, X.HALF * ref.abs() + X.SLOPE * (0.75 * u64).abs(), "d_gate")
    ref = 0.75 * value(g64, act)
    check(d_gu[:, n:], ref, (X.HALF + 2 * X.ACT) * ref.abs(), "d_up")


# counts: streamed (a row or two of several experts) and tiled (more rows)
@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [40, 3]], ids=["streamed", "tiled"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_values(hip_device, counts, act):
    """z = bias exactly (x and w are zeros): y = act(bias)."""
    n, e, m = len(VALS), len(counts), sum(counts)
    b = zs(e, hip_device)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int64, device=hip_device)
    x = torch.zeros(m, 64, dtype=BF16, device=hip_device)
    w = torch.zeros(e, n, 64, dtype=BF16, device=hip_device)
    y, pre = poisoned((m, n), BF16, hip_device), poisoned((m, n), BF16, hip_device)
    moe.moe_grouped_linear_bf16(x, w, off, y, bias=b, pre_activation=pre, activation=act)
    torch.cuda.synchronize()
    z = X.f64(b).repeat_interleave(torch.tensor(counts), 0)
    check(pre, z, torch.zeros_like(z), "pre_activation")
    ref = value(z, act)
    check(y, ref, (X.HALF + X.ACT) * ref.abs(), "y")


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [40, 3]], ids=["streamed", "tiled"])
@pytest.mark.parametrize("act", ACTS)
def test_gated_values_at_infinities(hip_device, counts, act):
    """g overflows to an infinity of either sign (3e38 times 3e38), u is 1.5."""
    n, k, e, m = 16, 64, len(counts), sum(counts)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int64, device=hip_device)
    x = torch.zeros(m, k, dtype=BF16, device=hip_device)
    x[:, 0], x[:, 1] = 3e38, 1.0
    w = torch.zeros(e, 2 * n, k, dtype=BF16, device=hip_device)
    w[:, 0:n:2, 0], w[:, 1:n:2, 0] = 3e38, -3e38
    w[:, n:, 1] = 1.5
    h, keep = poisoned((m, n), BF16, hip_device), poisoned((m, 2 * n), BF16, hip_device)
    moe.moe_grouped_gated_gemm_bf16(x, w, off, h, gate_up=keep, activation=act)
    torch.cuda.synchronize()
    g = torch.tensor([INF, -INF], dtype=torch.float64).repeat(n // 2).expand(m, n)
    check(keep[:, :n], g, torch.zeros_like(g), "g")
    ref = 1.5 * value(g, act)
    check(h, ref, torch.zeros_like(ref), "h")
