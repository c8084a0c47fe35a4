"""The expert layers' C ABI and binding on a host without a GPU: what the header
declares is exported, bad arguments are refused before anything touches HIP,
and the 64-bit references that the GPU tests use agree with central
differences of the formulas.
"""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import _experts as X
from mixture_experts_token_amd import binding, experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_experts.h")
OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 3, 4

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only on a host without a GPU")


def addr(i, extra=0):
    """A fake device address, never dereferenced; addresses lie 64 GiB apart."""
    return ctypes.c_void_p((i + 1) * (1 << 36) + extra)


@pytest.fixture(scope="module")
def lib():
    return experts._load()


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def test_header_and_exports(lib):
    names = ["moe_grouped_gated_gemm_backward_bf16", "moe_grouped_gated_gemm_bf16",
             "moe_grouped_linear_backward_bf16", "moe_grouped_linear_bf16", "moe_unpermute_backward"]
    assert declared_functions() == names
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(names) <= set(re.findall(r"\bT (moe_[a-z0-9_]+)\b", out))
    import mixture_experts_token_amd as moe

    for name in names:
        assert callable(getattr(moe, name)) and getattr(lib, name).argtypes


def test_header_compiles_as_c():
    src = '#include "moe_experts.h"\nint main(void) { return MOE_ACT_GELU_TANH; }\n'
    res = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER),
                          "-x", "c", "-"], input=src, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def gated(lib, **kw):
    a = dict(x=addr(0), w=addr(1), off=addr(2), e=4, rows=100, n=64, k=128, act=2, keep=addr(3), h=addr(4))
    a.update(kw)
    return lib.moe_grouped_gated_gemm_bf16(a["x"], a["w"], a["off"], a["e"], a["rows"], a["n"], a["k"], a["act"],
                                           a["keep"], a["h"], None)


def gated_back(lib, **kw):
    a = dict(dh=addr(0), keep=addr(1), x=addr(2), w=addr(3), off=addr(4), e=4, rows=100, n=64, k=128, act=2,
             dgu=addr(5), dx=addr(6), dw=addr(7))
    a.update(kw)
    return lib.moe_grouped_gated_gemm_backward_bf16(a["dh"], a["keep"], a["x"], a["w"], a["off"], a["e"], a["rows"],
                                                    a["n"], a["k"], a["act"], a["dgu"], a["dx"], a["dw"], None)


def linear(lib, **kw):
    a = dict(x=addr(0), w=addr(1), b=addr(2), r=addr(3), off=addr(4), e=4, rows=100, n=64, k=128, act=0,
             pre=addr(5), y=addr(6))
    a.update(kw)
    return lib.moe_grouped_linear_bf16(a["x"], a["w"], a["b"], a["r"], a["off"], a["e"], a["rows"], a["n"], a["k"],
                                       a["act"], a["pre"], a["y"], None)


def linear_back(lib, **kw):
    a = dict(dy=addr(0), pre=addr(1), x=addr(2), w=addr(3), off=addr(4), e=4, rows=100, n=64, k=128, act=2,
             dz=addr(5), dx=addr(6), dw=addr(7), db=addr(8))
    a.update(kw)
    return lib.moe_grouped_linear_backward_bf16(a["dy"], a["pre"], a["x"], a["w"], a["off"], a["e"], a["rows"],
                                                a["n"], a["k"], a["act"], a["dz"], a["dx"], a["dw"], a["db"], None)


def unpermute_back(lib, **kw):
    a = dict(do=addr(0), y=addr(1), dt=binding.MOE_DTYPE_BF16, wts=addr(2), inv=addr(3), n=10, h=64, topk=2,
             dy=addr(4), dw=addr(5))
    a.update(kw)
    return lib.moe_unpermute_backward(a["do"], a["y"], a["dt"], a["wts"], a["inv"], a["n"], a["h"], a["topk"],
                                      a["dy"], a["dw"], None)


@host_only
@pytest.mark.parametrize("call", [gated, gated_back, linear, linear_back], ids=lambda f: f.__name__)
def test_layer_sizes_are_refused(lib, call):
    for kw in (dict(e=0), dict(e=1025), dict(rows=-1), dict(rows=2**31), dict(n=0), dict(k=0), dict(n=-8),
               dict(n=2**20 + 8), dict(k=2**20 + 8), dict(act=-1), dict(act=4), dict(off=None)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(n=60), dict(k=12), dict(off=addr(9, 4)), dict(x=addr(9, 8)), dict(w=addr(9, 2))):
        assert call(lib, **kw) == MISALIGNED, kw


@host_only
def test_missing_buffers_are_refused(lib):
    for kw in (dict(x=None), dict(w=None), dict(h=None)):
        assert gated(lib, **kw) == INVALID, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None)):
        assert linear(lib, **kw) == INVALID, kw
    for kw in (dict(dh=None), dict(keep=None), dict(dgu=None), dict(x=None), dict(w=None)):
        assert gated_back(lib, **kw) == INVALID, kw
    for kw in (dict(dy=None), dict(pre=None), dict(dz=None), dict(x=None), dict(w=None)):
        assert linear_back(lib, **kw) == INVALID, kw
    # without an activation there is no pre-activation, and some output has to be given
    assert linear_back(lib, act=0) == INVALID
    assert linear_back(lib, act=0, pre=None) == INVALID
    assert linear_back(lib, act=0, dz=None) == INVALID
    assert linear_back(lib, act=0, pre=None, dz=None, dx=None, dw=None, db=None) == INVALID


@host_only
def test_overlaps_are_refused(lib):
    assert gated(lib, h=addr(0)) == INVALID
    assert gated(lib, keep=addr(4, 100 * 64 * 2 - 16)) == INVALID  # the last vector of h
    assert gated(lib, h=addr(1, 4 * 128 * 128 * 2 - 16)) == INVALID  # the last vector of w
    assert linear(lib, y=addr(3)) == INVALID  # in place over the residual
    assert linear(lib, pre=addr(2)) == INVALID
    assert gated_back(lib, dgu=addr(1)) == INVALID
    assert gated_back(lib, dx=addr(2)) == INVALID
    assert gated_back(lib, dw=addr(6, 16)) == INVALID
    assert linear_back(lib, dz=addr(0)) == INVALID
    assert linear_back(lib, db=addr(7, 4 * 64 * 128 * 2 - 16)) == INVALID
    assert unpermute_back(lib, dy=addr(1)) == INVALID
    assert unpermute_back(lib, dw=addr(2)) == INVALID


@host_only
def test_unpermute_backward_arguments(lib):
    for kw in (dict(n=-1), dict(topk=0), dict(topk=1025), dict(n=2**30, topk=2), dict(h=0), dict(do=None),
               dict(inv=None), dict(y=None), dict(wts=None), dict(dy=None, dw=None), dict(dt=7)):
        assert unpermute_back(lib, **kw) == INVALID, kw
    assert unpermute_back(lib, dt=binding.MOE_DTYPE_FP8_E4M3) == UNSUPPORTED
    for kw in (dict(h=60), dict(do=addr(9, 8)), dict(y=addr(9, 8)), dict(dy=addr(9, 8)), dict(wts=addr(9, 2)),
               dict(dw=addr(9, 2)), dict(inv=addr(9, 2))):
        assert unpermute_back(lib, **kw) == MISALIGNED, kw
    assert unpermute_back(lib, n=0) == OK  # nothing to do
    assert gated(lib, rows=0, x=None, h=None, keep=None) == OK
    assert linear(lib, rows=0, x=None, y=None, pre=None, r=None) == OK


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refuses_bad_tensors():
    off = torch.zeros(4, dtype=torch.int64)
    x, w, h = bf(10, 64), bf(3, 32, 64), bf(10, 16)
    call = experts.moe_grouped_gated_gemm_bf16
    with pytest.raises(ValueError, match="activation"):
        call(x, w, off, h, activation="tanh")
    with pytest.raises(ValueError, match="gate rows"):
        call(x, bf(3, 33, 64), off, h)
    with pytest.raises(ValueError, match="w must"):
        call(x, bf(32, 64), off, h)
    with pytest.raises(ValueError):
        call(bf(10, 72), w, off, h)  # k differs from w's
    with pytest.raises(ValueError):
        call(x, w, off, bf(9, 16))
    with pytest.raises(ValueError):
        call(x, w, off, bf(16, 10))  # as many elements, another shape
    with pytest.raises(TypeError):
        call(x.float(), w, off, h)
    with pytest.raises(TypeError):
        call(x, w, off.int(), h)
    with pytest.raises(ValueError):
        call(x, w, off[:3], h)
    with pytest.raises(ValueError, match="contiguous"):
        call(bf(64, 10).t(), w, off, h)
    with pytest.raises(ValueError):
        call(x, w, off, h, gate_up=bf(10, 16))
    with pytest.raises(TypeError, match="GPU"):
        call(x, w, off, h)


def test_binding_refuses_bad_backward_tensors():
    off = torch.zeros(4, dtype=torch.int64)
    x, w, dy = bf(10, 64), bf(3, 32, 64), bf(10, 32)
    back = experts.moe_grouped_linear_backward_bf16
    with pytest.raises(ValueError, match="go with"):
        back(dy, x, w, off, d_x=bf(10, 64), pre_activation=dy)
    with pytest.raises(ValueError, match="required"):
        back(dy, x, w, off, d_x=bf(10, 64), activation="silu")
    with pytest.raises(ValueError, match="x is required"):
        back(dy, None, w, off, d_w=bf(3, 32, 64))
    with pytest.raises(ValueError):
        back(dy, x, w, off, d_bias=bf(32, 3))
    with pytest.raises(TypeError):
        back(dy, x, w, off, d_w=torch.zeros(3, 32, 64))
    with pytest.raises(TypeError, match="GPU"):
        back(dy, None, w, off, d_x=bf(10, 64))
    gback = experts.moe_grouped_gated_gemm_backward_bf16
    with pytest.raises(ValueError):
        gback(bf(10, 16), bf(10, 16), x, w, off, bf(10, 32))
    with pytest.raises(TypeError, match="GPU"):
        gback(bf(10, 16), bf(10, 32), x, w, off, bf(10, 32))
    up = experts.moe_unpermute_backward
    wts, inv = torch.zeros(5, 2), torch.zeros(10, dtype=torch.int32)
    with pytest.raises(ValueError):
        up(bf(4, 64), bf(10, 64), wts, inv, d_topk_weights=torch.zeros(5, 2))
    with pytest.raises(ValueError, match="expanded_output is required"):
        up(bf(5, 64), None, wts, inv, d_topk_weights=torch.zeros(5, 2))
    with pytest.raises(TypeError):
        up(bf(5, 64), bf(10, 64).float(), wts, inv, d_topk_weights=torch.zeros(5, 2))
    with pytest.raises(TypeError):
        up(bf(5, 64).half(), bf(10, 64).half(), wts, inv, d_topk_weights=torch.zeros(5, 2))
    with pytest.raises(TypeError, match="GPU"):
        up(bf(5, 64), None, wts, inv, d_expanded_output=bf(10, 64))


@pytest.mark.parametrize("act", sorted(experts.ACTIVATIONS))
def test_reference_gradients_agree_with_differences(act):
    """The 64-bit references: central differences of sum(out * cotangent) along
    random directions.  With a step of 1e-6 the truncation is of order 1e-12
    and the cancellation 1e-16 / 1e-6, times sums of magnitudes around 1e2."""
    g = torch.Generator().manual_seed(5)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    off = torch.tensor([0, 3, 3, 8])
    x, w, bias, cot = rnd(8, 6), rnd(3, 10, 6), rnd(3, 10), rnd(8, 10)

    def layer(x, w, b):
        z, _ = X.grouped(x, w, off)
        for e, lo, hi in X.segments(off):
            z[lo:hi] += b[e]
        return z

    def gated(x, w):
        z, _ = X.grouped(x, w, off)
        return X.act_value(z[:, :5], act) * z[:, 5:]

    z = layer(x, w, bias)
    d_z = cot * X.act_slope(z, act)
    grads = [X.input_grad(d_z, w, off)[0], X.weight_grad(d_z, x, off)[0], X.bias_grad(d_z, off)[0]]
    at, step = [x, w, bias], 1e-6
    for i in range(3):
        v = rnd(*at[i].shape)

        def f(t):
            moved = [a + t * v if j == i else a for j, a in enumerate(at)]
            return float((X.act_value(layer(*moved), act) * cot).sum())

        assert abs((f(step) - f(-step)) / (2 * step) - float((grads[i] * v).sum())) < 1e-6

    z, _ = X.grouped(x, w, off)
    gz, u, c = z[:, :5], z[:, 5:], cot[:, :5]
    d_gu = torch.cat([c * u * X.act_slope(gz, act), c * X.act_value(gz, act)], 1)
    grads = [X.input_grad(d_gu, w, off)[0], X.weight_grad(d_gu, x, off)[0]]
    for i, a in enumerate((x, w)):
        v = rnd(*a.shape)

        def f(t):
            return float((gated(x + t * v if i == 0 else x, w + t * v if i == 1 else w) * c).sum())

        assert abs((f(step) - f(-step)) / (2 * step) - float((grads[i] * v).sum())) < 1e-6
