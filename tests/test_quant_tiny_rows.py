"""fp8 quantisation of finite f32 rows whose largest magnitude over 448 rounds to 0 in
fp32: the scale is 1 and every code a zero, as for a row of zeros, and not a scale of
0, over which a zero of the same row is a NaN.

448 * 2^-150 = 224 of the smallest subnormals, 2^-149, is the last such magnitude
(half a subnormal rounds to the even 0); 225 of them have the scale 2^-149.
"""

import numpy as np
import pytest
import torch

import mixture_experts_token_amd as moe
import oracle
from _parity import poisoned, to_np
from mixture_experts_token_amd import binding

TINIEST = 2.0**-149


def tiny_rows(h):
    """f32 [7, h]: rows below, at and past the border, beside zeros; an ordinary row."""
    x = np.zeros((7, h), np.float64)
    x[0, 1] = TINIEST
    x[1, ::3], x[1, 4] = 223 * TINIEST, -224 * TINIEST
    x[2, 1::2], x[2, 2] = -100 * TINIEST, 5 * TINIEST
    x[3, 0], x[3, 5] = 225 * TINIEST, -TINIEST
    x[4, :] = 200 * TINIEST
    x[5, 0], x[5, 3] = 448 * TINIEST, 224 * TINIEST
    x[6, :] = np.linspace(-1, 1, h)
    return x.astype(np.float32)


def check(x, codes, scale, group=None):
    """Codes and scales of rows of tiny_rows, by definition."""
    group = x.shape[1] if group is None else group
    scale = scale.reshape(x.shape[0], -1)
    for r in range(x.shape[0]):
        for g in range(x.shape[1] // group):
            v, c = x[r, g * group:(g + 1) * group].astype(np.float64), codes[r, g * group:(g + 1) * group]
            want = np.float32(np.abs(v).max() / 448)  # one rounding: the quotient is exact enough in 64 bits
            assert scale[r, g] == (want if want > 0 else 1), (r, g)
            assert not np.any(c & 0x7F == 0x7F), (r, g)
            if want == 0:
                assert np.all(c & 0x7F == 0), (r, g)
            assert np.all(c[v == 0] & 0x7F == 0), (r, g)


@pytest.mark.parametrize("group", [None, 8])
def test_oracle(group):
    x = tiny_rows(64)
    codes, scale = oracle.quantize_fp8_rows(x, "f32", group)
    check(x, codes, scale, group)


@pytest.mark.gpu
@pytest.mark.parametrize("h", [64, 1024, 4096, 20000])
@pytest.mark.parametrize("repeat", [1, 200])
def test_quantize_rows(hip_device, h, repeat):
    x = np.tile(tiny_rows(h), (repeat, 1))
    codes, scale = poisoned(x.shape, torch.uint8, hip_device), poisoned((x.shape[0],), torch.float32, hip_device)
    moe.moe_quantize_rows_fp8(torch.from_numpy(x).to(hip_device), codes, scale)
    torch.cuda.synchronize()
    check(x, to_np(codes), to_np(scale))


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 8, 64])
@pytest.mark.parametrize("repeat", [1, 30, 300])
def test_permute(hip_device, group, repeat):
    """One-launch, several waves per token, a wave per token."""
    x = np.tile(tiny_rows(256), (repeat, 1))
    n, h = x.shape
    groups = h // group if group else 1
    dev, i32 = hip_device, torch.int32
    ids = (torch.arange(n, dtype=i32, device=dev) % 5).view(n, 1).contiguous()
    codes, scale = poisoned((n, h), torch.uint8, dev), poisoned((n, groups), torch.float32, dev)
    off, perm, inv = poisoned((6,), torch.int64, dev), poisoned((n,), i32, dev), poisoned((n,), i32, dev)
    ws = poisoned((max(16, binding.moe_permute_workspace_size(n, 1, 5)),), torch.uint8, dev)
    binding.moe_permute_quant_fp8(torch.from_numpy(x).to(dev), ids, 5, codes, scale, off, perm, inv, ws,
                                  group_size=group)
    torch.cuda.synchronize()
    check(x[to_np(perm)], to_np(codes), to_np(scale), group or None)
