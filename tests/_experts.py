"""64-bit references of the expert layers and the error bounds their tests use.

Bounds, with the half step of a bf16 rounding taken as 2^-8 of the value:

* a product of T terms accumulated in fp32 is within T 2^-22 of the sum of the
  terms' magnitudes (four times the worst case of any order of summation, as
  the matrix cores' internal order is not documented);
* the logistic function is evaluated in fp32 as 1 / (1 + exp2(a t)): the
  argument carries at most 4 roundings of relative 2^-24, so exp's relative
  error is at most 4 |t| 2^-24 + 2^-23, and |t| < 104 before the result is 0
  or 1 in fp32; value and slope are within 2^-14 of the sum of the magnitudes
  of their terms, at most 2^-14 |act(z)| and 2^-13 (GELU's largest slope term
  is below 2).
"""

import math

import torch

HALF = 2.0**-8    # half a step of bf16
ACT = 2.0**-14    # relative error of an activation's value in fp32
SLOPE = 2.0**-13  # absolute error of its slope
TINY = 1e-30
STEEP = 1.13      # the largest slope of any of the activations


def accumulate(t):
    return t * 2.0**-22


def act_value(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))
    return z


def act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z**3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def f64(t):
    return None if t is None else t.detach().cpu().double()


def segments(off):
    off = [int(v) for v in off]
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def assert_within(got, ref, tol, what):
    """got within tol of ref elementwise (both NaN counts as equal)."""
    err = (f64(got) - ref).abs()
    err = torch.where(torch.isnan(ref) & torch.isnan(f64(got)), torch.zeros_like(err), err)
    bad = ~(err <= tol + TINY)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d outside; first at %s: got %g, want %g, tolerance %g" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(ref[i]), float(tol[i])))


def grouped(x, w, off):
    """(product, sum of magnitudes) of x[j] w[e]^T, rows of all experts."""
    m = int(off[-1])
    z, mag = torch.zeros(m, w.shape[1], dtype=torch.float64), torch.zeros(m, w.shape[1], dtype=torch.float64)
    for e, lo, hi in segments(off):
        z[lo:hi] = x[lo:hi] @ w[e].t()
        mag[lo:hi] = x[lo:hi].abs() @ w[e].abs().t()
    return z, mag


def input_grad(d_z, w, off):
    m = int(off[-1])
    g, mag = torch.zeros(m, w.shape[2], dtype=torch.float64), torch.zeros(m, w.shape[2], dtype=torch.float64)
    for e, lo, hi in segments(off):
        g[lo:hi] = d_z[lo:hi] @ w[e]
        mag[lo:hi] = d_z[lo:hi].abs() @ w[e].abs()
    return g, mag


def weight_grad(d_z, x, off):
    shape = (len(off) - 1, d_z.shape[1], x.shape[1])
    g, mag = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    for e, lo, hi in segments(off):
        g[e] = d_z[lo:hi].t() @ x[lo:hi]
        mag[e] = d_z[lo:hi].abs().t() @ x[lo:hi].abs()
    return g, mag


def bias_grad(d_z, off):
    shape = (len(off) - 1, d_z.shape[1])
    g, mag = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    for e, lo, hi in segments(off):
        g[e] = d_z[lo:hi].sum(0)
        mag[e] = d_z[lo:hi].abs().sum(0)
    return g, mag


def longest(off):
    return max([hi - lo for _, lo, hi in segments(off)], default=0)


def check_gated(x, w, off, act, h, gate_up):
    n = w.shape[1] // 2
    m = int(off[-1])
    z, mag = grouped(f64(x), f64(w), off)
    dz = accumulate(x.shape[1]) * mag
    g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
    a = act_value(g, act)
    ref = a * u
    tol = (HALF + ACT) * ref.abs() + STEEP * dg * (u.abs() + du) + (a.abs() + STEEP * dg) * du
    assert_within(h[:m], ref, tol, "h")
    if gate_up is not None:
        assert_within(gate_up[:m], z, HALF * z.abs() + 2 * dz, "gate_up")


def check_linear(x, w, bias, residual, off, act, y, pre):
    m = int(off[-1])
    z, mag = grouped(f64(x), f64(w), off)
    if bias is not None:
        for e, lo, hi in segments(off):
            z[lo:hi] += f64(bias)[e]
            mag[lo:hi] += f64(bias)[e].abs()
    dz = accumulate(x.shape[1] + 1) * mag
    a = act_value(z, act)
    ref = a if residual is None else a + f64(residual)[:m]
    tol = HALF * ref.abs() + 2.0**-23 * ref.abs() + ACT * a.abs() + STEEP * 2 * dz
    assert_within(y[:m], ref, tol, "y")
    if pre is not None:
        assert_within(pre[:m], z, HALF * z.abs() + 2 * dz, "pre_activation")


def check_products(d_z, x, w, off, d_x, d_w, d_bias=None):
    """The products of a backward pass, from the bf16 d_z that they take."""
    m = int(off[-1])
    dz64 = f64(d_z)[:m]
    if d_x is not None:
        ref, mag = input_grad(dz64, f64(w), off)
        assert_within(d_x[:m], ref, HALF * ref.abs() + 2 * accumulate(w.shape[1]) * mag, "d_x")
    if d_w is not None:
        ref, mag = weight_grad(dz64, f64(x), off)
        assert_within(d_w, ref, HALF * ref.abs() + 2 * accumulate(longest(off)) * mag, "d_w")
    if d_bias is not None:
        ref, mag = bias_grad(dz64, off)
        assert_within(d_bias, ref, HALF * ref.abs() + 2 * accumulate(longest(off)) * mag, "d_bias")


def check_gated_slopes(d_h, gate_up, off, act, d_gate_up):
    m = int(off[-1])
    n = d_h.shape[1]
    d, g, u = f64(d_h)[:m], f64(gate_up)[:m, :n], f64(gate_up)[:m, n:]
    ref = d * u * act_slope(g, act)
    assert_within(d_gate_up[:m, :n], ref, HALF * ref.abs() + SLOPE * (d * u).abs(), "d_gate")
    ref = d * act_value(g, act)
    assert_within(d_gate_up[:m, n:], ref, (HALF + 2 * ACT) * ref.abs(), "d_up")


def check_slopes(d_y, pre, off, act, d_z):
    m = int(off[-1])
    d, z = f64(d_y)[:m], f64(pre)[:m]
    ref = d * act_slope(z, act)
    assert_within(d_z[:m], ref, HALF * ref.abs() + SLOPE * d.abs(), "d_pre_activation")


def unpermute_backward(d_out, y, wts, inv):
    """(d_expanded rows written {j: row}, d_weights, sum of magnitudes); entries of -1 give 0, other bad ones NaN."""
    n, k = wts.shape
    slots = inv.view(-1).tolist()
    rows, d_w, mag = {}, torch.zeros(n * k, dtype=torch.float64), torch.zeros(n * k, dtype=torch.float64)
    d_out, y, wf = f64(d_out), f64(y), f64(wts).view(-1)
    for r, j in enumerate(slots):
        if 0 <= j < n * k:
            rows[j] = wf[r] * d_out[r // k]
            d_w[r] = (d_out[r // k] * y[j]).sum()
            mag[r] = (d_out[r // k] * y[j]).abs().sum()
        elif j != -1:
            d_w[r] = math.nan
    return rows, d_w.view(n, k), mag.view(n, k)
