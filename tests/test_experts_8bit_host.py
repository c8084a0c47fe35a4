"""The 8-bit expert path's C ABI and binding on a host without a GPU: what the
header declares is exported, bad arguments are refused before anything touches
HIP, and the int8 reference that the GPU tests use is the nearest integer by
rational arithmetic.
"""

import ctypes
import os
import re
import subprocess
from fractions import Fraction

import pytest
import torch

import _experts_8bit as E8
from mixture_experts_token_amd import binding, experts_8bit as X8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_experts_8bit.h")
OK, INVALID, SMALL, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3, 4
F32, BF16, FP8 = binding.MOE_DTYPE_F32, binding.MOE_DTYPE_BF16, binding.MOE_DTYPE_FP8_E4M3

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only on a host without a GPU")
KINDS = ["int8", "fp8"]


def addr(i, extra=0):
    """A fake device address, never dereferenced; addresses lie 64 GiB apart."""
    return ctypes.c_void_p((i + 1) * (1 << 36) + extra)


@pytest.fixture(scope="module")
def lib():
    return X8._load()


def test_header_and_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert names == ["moe_grouped_gated_gemm_fp8", "moe_grouped_gated_gemm_int8", "moe_grouped_linear_fp8",
                     "moe_grouped_linear_int8", "moe_permute_quant_int8", "moe_quantize_rows_fp8",
                     "moe_quantize_rows_int8"]
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(names) <= set(re.findall(r"\bT (moe_[a-z0-9_]+)\b", out))
    import mixture_experts_token_amd as moe

    for name in names:
        assert callable(getattr(moe, name)) and getattr(lib, name).argtypes


def test_header_compiles_as_c():
    src = '#include "moe_experts_8bit.h"\nint main(void) { return MOE_ACT_SILU; }\n'
    res = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER),
                          "-x", "c", "-"], input=src, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def gated(lib, kind, **kw):
    a = dict(x=addr(0), xs=addr(1), w=addr(2), ws=addr(3), off=addr(4), e=4, rows=100, n=64, k=128, act=2, y=addr(5))
    a.update(kw)
    return getattr(lib, "moe_grouped_gated_gemm_" + kind)(
        a["x"], a["xs"], a["w"], a["ws"], a["off"], a["e"], a["rows"], a["n"], a["k"], a["act"], a["y"], None)


def linear(lib, kind, **kw):
    a = dict(x=addr(0), xs=addr(1), w=addr(2), ws=addr(3), b=addr(6), r=addr(7), off=addr(4), e=4, rows=100, n=64,
             k=128, act=0, y=addr(5))
    a.update(kw)
    return getattr(lib, "moe_grouped_linear_" + kind)(
        a["x"], a["xs"], a["w"], a["ws"], a["b"], a["r"], a["off"], a["e"], a["rows"], a["n"], a["k"], a["act"],
        a["y"], None)


def quantize(lib, kind, **kw):
    a = dict(x=addr(0), dt=BF16, off=addr(1), e=4, rows=100, n=64, codes=addr(2), s=addr(3))
    a.update(kw)
    return getattr(lib, "moe_quantize_rows_" + kind)(a["x"], a["dt"], a["off"], a["e"], a["rows"], a["n"], a["codes"],
                                                     a["s"], None)


def permute(lib, **kw):
    a = dict(x=addr(0), dt=BF16, ids=addr(1), idt=binding.MOE_DTYPE_INT32, n=100, h=64, topk=2, e=4, map=None, local=0,
             codes=addr(2), s=addr(3), off=addr(4), perm=addr(5), inv=addr(6), ws=addr(7), wsb=1 << 20)
    a.update(kw)
    return lib.moe_permute_quant_int8(a["x"], a["dt"], a["ids"], a["idt"], a["n"], a["h"], a["topk"], a["e"], a["map"],
                                      a["local"], a["codes"], a["s"], a["off"], a["perm"], a["inv"], a["ws"],
                                      a["wsb"], None)


@host_only
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", [gated, linear], ids=lambda f: f.__name__)
def test_layer_arguments(lib, kind, call):
    for kw in (dict(e=0), dict(e=1025), dict(rows=-1), dict(rows=2**31), dict(n=0), dict(k=0), dict(n=-8),
               dict(n=2**20 + 8), dict(k=2**20 + 16), dict(act=-1), dict(act=4), dict(off=None), dict(x=None),
               dict(xs=None), dict(w=None), dict(ws=None), dict(y=None)):
        assert call(lib, kind, **kw) == INVALID, kw
    for kw in (dict(n=60), dict(k=24), dict(off=addr(9, 4)), dict(x=addr(9, 8)), dict(w=addr(9, 2)),
               dict(xs=addr(9, 2)), dict(ws=addr(9, 1)), dict(y=addr(9, 8))):
        assert call(lib, kind, **kw) == MISALIGNED, kw
    # the last bytes of every input
    for kw in (dict(y=addr(0)), dict(y=addr(0, 100 * 128 - 16)), dict(y=addr(1, 4 * 100 - 16)),
               dict(y=addr(2, 4 * 64 * 128 - 16)), dict(y=addr(3, 4 * 4 * 64 - 16)), dict(y=addr(4, 32))):
        assert call(lib, kind, **kw) == INVALID, kw
    assert call(lib, kind, rows=0, x=None, xs=None, y=None) == OK
    assert call(lib, kind, k=2**17) == (INVALID if kind == "int8" else 5)  # 5: no device here
    assert call(lib, kind, k=2**17 - 16) == 5


@host_only
@pytest.mark.parametrize("kind", KINDS)
def test_linear_epilogue_arguments(lib, kind):
    for kw in (dict(b=addr(9, 8)), dict(r=addr(9, 8))):
        assert linear(lib, kind, **kw) == MISALIGNED, kw
    for kw in (dict(y=addr(7)), dict(y=addr(6, 4 * 64 * 2 - 16)), dict(y=addr(7, 100 * 64 * 2 - 16))):
        assert linear(lib, kind, **kw) == INVALID, kw


@host_only
@pytest.mark.parametrize("kind", KINDS)
def test_quantize_arguments(lib, kind):
    assert quantize(lib, kind, dt=FP8) == UNSUPPORTED
    for kw in (dict(e=0), dict(e=1025), dict(off=None), dict(off=None, e=0, rows=-1), dict(rows=-1), dict(rows=2**31),
               dict(n=0), dict(n=2**20 + 8), dict(x=None), dict(codes=None), dict(s=None), dict(codes=addr(0)),
               dict(codes=addr(0, 100 * 64 * 2 - 16)), dict(s=addr(2, 100 * 64 - 4)), dict(s=addr(1, 36))):
        assert quantize(lib, kind, **kw) == INVALID, kw
    for kw in (dict(n=60), dict(n=62, dt=F32), dict(x=addr(9, 8)), dict(codes=addr(9, 8)), dict(s=addr(9, 2)),
               dict(off=addr(9, 4))):
        assert quantize(lib, kind, **kw) == MISALIGNED, kw
    assert quantize(lib, kind, rows=0, x=None, codes=None, s=None) == OK
    assert quantize(lib, kind, off=None, e=0, rows=0) == OK


@host_only
def test_permute_arguments(lib):
    for kw in (dict(dt=FP8),):
        assert permute(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(n=-1), dict(h=0), dict(h=8200), dict(h=4100, dt=F32), dict(topk=0), dict(topk=5), dict(e=0),
               dict(e=1025), dict(n=2**30, topk=2), dict(x=None), dict(ids=None), dict(codes=None), dict(s=None),
               dict(off=None), dict(perm=None), dict(inv=None), dict(local=2), dict(idt=F32), dict(map=addr(8)),
               dict(codes=addr(0)), dict(s=addr(1)), dict(codes=addr(5, 200 * 4 - 16)), dict(s=addr(2, 200 * 64 - 4))):
        assert permute(lib, **kw) == INVALID, kw
    for kw in (dict(h=60), dict(x=addr(9, 8)), dict(codes=addr(9, 4)), dict(s=addr(9, 2)), dict(off=addr(9, 4))):
        assert permute(lib, **kw) == MISALIGNED, kw
    assert permute(lib, n=100000, topk=4, wsb=16) == SMALL


def test_binding_refuses_bad_tensors():
    off = torch.zeros(4, dtype=torch.int64)
    i8, f8 = torch.int8, torch.float8_e4m3fn

    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape).to(dtype)

    x, xs, w, ws, h = t(10, 64, dtype=i8), torch.ones(10), t(3, 32, 64, dtype=i8), torch.ones(3, 32), t(10, 16)
    call = X8.moe_grouped_gated_gemm_int8
    with pytest.raises(ValueError, match="activation"):
        call(x, xs, w, ws, off, h, activation="tanh")
    with pytest.raises(ValueError, match="gate rows"):
        call(x, xs, t(3, 33, 64, dtype=i8), torch.ones(3, 33), off, h)
    for bad in ((t(10, 72, dtype=i8), xs, w, ws, off, h), (x, torch.ones(9), w, ws, off, h),
                (x, torch.ones(10, 2), w, ws, off, h), (x, xs, w, torch.ones(3, 16), off, h),
                (x, xs, w, ws, off[:3], h), (x, xs, w, ws, off, t(9, 16)), (x, None, w, ws, off, h)):
        with pytest.raises(ValueError):
            call(*bad)
    for bad in ((x.to(f8), xs, w, ws, off, h), (x, xs.double(), w, ws, off, h), (x, xs, w.to(f8), ws, off, h),
                (x, xs, w, ws, off.int(), h), (x, xs, w, ws, off, h.float())):
        with pytest.raises(TypeError):
            call(*bad)
    with pytest.raises(TypeError, match="GPU"):
        call(x, xs[:, None], w, ws, off, h)
    linear = X8.moe_grouped_linear_fp8
    xf, wf, y = x.to(f8), w.to(f8), t(10, 32)
    with pytest.raises(ValueError):
        linear(xf, xs, wf, ws, off, y, bias=t(32))
    with pytest.raises(ValueError):
        linear(xf, xs, wf, ws, off, y, residual=t(10, 16))
    with pytest.raises(TypeError):
        linear(x, xs, wf, ws, off, y)
    with pytest.raises(TypeError, match="GPU"):
        linear(xf.view(torch.uint8), xs, wf, ws, off, y)
    quantize = X8.moe_quantize_rows_int8
    for bad in ((t(10, 64), t(10, 64, dtype=f8), xs), (t(10, 64, dtype=torch.float16), x, xs)):
        with pytest.raises(TypeError):
            quantize(*bad)
    for bad in ((t(10, 64), t(10, 32, dtype=i8), xs), (t(10, 64), x, torch.ones(11)), (t(64), x, xs)):
        with pytest.raises(ValueError):
            quantize(*bad)
    with pytest.raises(TypeError, match="GPU"):
        quantize(t(10, 64), x, xs, expert_first_token_offset=off)
    ids, idx, offs = torch.zeros(5, 2, dtype=torch.int32), torch.zeros(10, dtype=torch.int32), torch.zeros(
        5, dtype=torch.int64)
    permute = X8.moe_permute_quant_int8
    for bad in ((t(4, 64), ids, 4, x, xs, offs, idx, idx), (t(5, 64), ids, 4, x[:, :32].contiguous(), xs, offs, idx, idx),
                (t(5, 64), ids, 5, x, xs, offs, idx, idx), (t(5, 64), ids, 4, x, xs, offs, idx[:9], idx)):
        with pytest.raises(ValueError):
            permute(*bad)
    for bad in ((t(5, 64), ids.short(), 4, x, xs, offs, idx, idx), (t(5, 64), ids, 4, x.to(f8), xs, offs, idx, idx),
                (t(5, 64, dtype=torch.float16), ids, 4, x, xs, offs, idx, idx)):
        with pytest.raises(TypeError):
            permute(*bad)
    with pytest.raises(TypeError, match="GPU"):
        permute(t(5, 64), ids, 4, x, xs, offs, idx, idx)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_int8_reference_is_the_nearest_integer(dtype):
    """Against rational arithmetic: x = (q + 1/2) scale and its neighbours, and random values, for many scales."""
    g = torch.Generator().manual_seed(11)
    rows = []
    for e in (-100, -3, 0, 7, 60):
        amax = (torch.rand(1, generator=g) + 1) * 2.0**e
        scale = (amax.double() / 127).float()
        q = torch.randint(-127, 127, (64,), generator=g).double() + 0.5
        x = (q * scale.double()).float()
        x = torch.cat([amax, x, torch.nextafter(x, torch.tensor(float("inf"))), torch.randn(63, generator=g) * amax / 3])
        rows.append(x.clamp(-float(amax), float(amax)))
    x = torch.stack(rows + [torch.arange(192).float().remainder(127.5).div(0.5).floor().mul(0.5).clamp(max=127)])
    x = x.to(dtype)
    codes, scale = E8.int8_codes(x)
    for i in range(x.shape[0]):
        s = Fraction(float(scale[i]))
        for v, c in zip(x[i].tolist(), codes[i].tolist()):
            r = Fraction(v) / s
            want = max(-127, min(127, round(r)))  # of a Fraction: nearest, ties to even
            assert c == want, (i, v, float(s), c, want)
