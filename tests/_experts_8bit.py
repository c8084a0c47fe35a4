"""64-bit references of the 8-bit expert path and the error bounds its tests use.

Codes and scales of the quantisers are compared for equality.  Bounds of the
layers, with the half step of a bf16 rounding taken as 2^-8 of the value:

* a sum of int8 codes is exact in the 32-bit integers; its conversion to fp32
  and the products with two scales are three roundings of relative 2^-24,
  within 2^-22 of the value together;
* the matrix cores add products of fp8 codes eight at a time (the eight codes of
  an aligned 8-byte piece of both rows).  With e the largest exponent of the
  eight, each product is cut, towards zero, to a multiple of 2^(e - 13): one of two
  4-bit significands and exponent e is such a multiple, so at most seven products
  lose less than 2^(e - 13) each, and a piece's sum is off by less than 7 2^-13 2^e <= 7
  2^-13 times its largest product, which is at most the largest |x| times the
  largest |w| of the piece.  (Seen in single products: beside 256 * 256 = 2^16 a
  product of 4 vanishes within the same eight codes and nowhere else, 8 stays, 15
  becomes 8; beside 240 * 240, of exponent 14, 2 stays.)  Sums of pieces are in
  fp32: within T 2^-22 of the sum of the terms' magnitudes (four times the worst
  case of any order of summation);
* activations as in ``_experts``.

No scale in these tests is so small that a product of it is subnormal in fp32.
"""

import numpy as np
import torch

import oracle
from _experts import ACT, HALF, STEEP, accumulate, act_value, assert_within, f64, grouped
from _parity import to_np

SCALED = 2.0**-22


def int8_codes(x):
    """(codes, scale) of rows of finite or special bf16 / f32 values.

    x / scale in 64 bits: x has at most 24 and scale 24 bits, so a quotient that
    is not a tie is at least 2^-33 (relative) away from every tie.
    """
    bits = x.float().abs().view(torch.int32).amax(dim=1)  # NaN above infinity above every number
    scale = (bits.view(torch.float32).double() / 127).float()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = torch.round(x.double() / scale.double()[:, None]).clamp(-127, 127)
    q = torch.where(torch.isfinite(scale)[:, None], q, torch.zeros_like(q))
    return q.to(torch.int8), scale


def fp8_codes(x):
    """(code bytes, scale) by the oracle."""
    codes, scale = oracle.quantize_fp8_rows(to_np(x), "bf16" if x.dtype == torch.bfloat16 else "f32")
    return torch.from_numpy(codes.copy()), torch.from_numpy(np.asarray(scale, np.float32).reshape(-1).copy())


def codes_of(x, kind):
    return int8_codes(x) if kind == "int8" else fp8_codes(x)


def values(codes, kind):
    """The numbers that codes stand for, in 64 bits."""
    if kind == "int8":
        return codes.detach().cpu().double()
    return codes.detach().cpu().view(torch.float8_e4m3fn).float().double()


def scaled(x, x_scale, w, w_scale, off, kind):
    """(z, its error bound): the scaled products of codes, rows of all experts."""
    m = int(off[-1])
    z, mag = grouped(values(x, kind)[:m], values(w, kind), off)
    factor = torch.zeros_like(z)
    bounds = [int(v) for v in off]
    for e in range(len(bounds) - 1):
        lo, hi = bounds[e], bounds[e + 1]
        factor[lo:hi] = f64(x_scale).view(-1)[lo:hi, None] * f64(w_scale)[e]
    z = z * factor
    err = SCALED * z.abs()
    if kind == "fp8":
        cut, _ = grouped(largest_of_eight(values(x, kind)[:m]), largest_of_eight(values(w, kind)), off)
        err = err + (accumulate(x.shape[1]) * mag + 7 * 2.0**-13 * cut) * factor.abs()
    return z, err


def largest_of_eight(v):
    """The largest magnitude of each aligned piece of eight codes of a row."""
    return v.abs().view(*v.shape[:-1], v.shape[-1] // 8, 8).amax(-1)


def check_gated(x, x_scale, w, w_scale, off, kind, act, h):
    m, n = int(off[-1]), w.shape[1] // 2
    z, dz = scaled(x, x_scale, w, w_scale, off, kind)
    g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
    a = act_value(g, act)
    ref = a * u
    tol = (HALF + ACT) * ref.abs() + STEEP * dg * (u.abs() + du) + (a.abs() + STEEP * dg) * du
    assert_within(h[:m], ref, tol, "h")


def check_linear(x, x_scale, w, w_scale, bias, residual, off, kind, act, y):
    m = int(off[-1])
    z, dz = scaled(x, x_scale, w, w_scale, off, kind)
    if bias is not None:
        bounds = [int(v) for v in off]
        for e in range(len(bounds) - 1):
            z[bounds[e]:bounds[e + 1]] += f64(bias)[e]
        dz = dz + SCALED * z.abs()
    a = act_value(z, act)
    ref = a if residual is None else a + f64(residual)[:m]
    tol = HALF * ref.abs() + 2.0**-23 * ref.abs() + ACT * a.abs() + STEEP * 2 * dz
    assert_within(y[:m], ref, tol, "y")
