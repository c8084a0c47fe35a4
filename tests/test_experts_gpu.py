"""GPU parity of the expert layers (include/moe_experts.h) against 64-bit references.

The bounds are derived in tests/_experts.py.  Every output is poisoned before
the call, and rows behind the last expert's (the buffers hold a few more than
off[E]) must keep the poison; those rows hold NaN in the inputs.
"""

import numpy as np
import pytest
import torch

import _experts as X
from _parity import POISON, gpu_permute, gpu_unpermute, poisoned
import mixture_experts_token_amd as moe
from mixture_experts_token_amd import binding

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TAIL = 3  # rows behind the last expert's


def _say(msg):
    print("[case] " + msg, flush=True)


def _bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def assert_untouched(t, what):
    assert bool((t.contiguous().view(torch.uint8) == POISON).all()), what + " was written"


def randn(shape, seed, dev, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev)


def rows_of(counts, cols, seed, dev, scale=1.0):
    """[sum(counts) + TAIL, cols] with NaN in the rows behind the experts'."""
    t = randn((sum(counts) + TAIL, cols), seed, dev, scale)
    t[sum(counts):] = float("nan")
    return t


def offsets(counts, dev):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64, device=dev)


# (rows of each expert, n, k): one row; empty experts; sizes that fill no tile
# or k-step; whole tiles; decode sizes (about a row per expert) with k of
# every kind; experts longer than a tile
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0], 64, 64),
    ([0, 0], 72, 16),
    ([3, 0, 130, 1, 64], 264, 200),
    ([513, 0, 256], 512, 1024),
    ([65, 127, 129], 136, 72),
    ([1, 1, 1, 1, 1, 1, 1, 1], 520, 2048),
    ([1, 0, 2, 1, 0, 3, 1, 1], 96, 1000),
    ([2, 2, 0, 1], 256, 8200),
    ([17, 5, 9, 33], 1032, 448),
    ([300] + [0] * 30 + [5], 128, 128),
    ([1] * 1024, 40, 64),
    ([9, 1, 3, 8, 0, 4], 72, 1096),
    ([0, 5, 1], 136, 16392),
    ([2, 0, 1], 40, 33000),
    # one expert with most of the rows beside many with few (streamed and tiled in one call)
    ([1, 0, 2] * 15 + [190, 33, 32], 136, 1096),
    # experts on both sides of the weight gradient's row limit, rows of whole
    # lines and not, more columns than one of its items
    ([16, 17, 0, 2, 15, 8, 1, 4, 40], 72, 2176),
    ([16, 17, 0, 2, 15, 8, 1, 4, 40], 264, 2120),
    # enough work for the large tiles in the forward, the input's and the weight's gradient
    ([1500, 0, 700, 257, 1000, 3], 3864, 520),
    ([1500, 0, 700, 257, 1000, 3], 520, 3864),
    ([700, 0, 1, 410], 1800, 2000),
    ([128, 384, 385, 256, 0, 641], 2056, 1288),
    # 256 heavy large tiles and the remainders of two experts beside them (forward; input's gradient)
    ([1024, 1025, 1134, 1023], 3960, 1032),
    ([1024, 1025, 1134, 1023], 1032, 3960),
]
ACTS = ["silu", "gelu_tanh", "relu", "none"]


def _id(v):
    return "rows%d-%dx%d" % (sum(v[0]), v[1], v[2])


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("act", ACTS)
def test_gated_forward(hip_device, shape, act):
    counts, n, k = shape
    dev = hip_device
    _say("gated %s act=%s" % (_id(shape), act))
    m = sum(counts)
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w = randn((len(counts), 2 * n, k), 2, dev, k**-0.5)
    keep = poisoned((m + TAIL, 2 * n), BF16, dev)
    h, h2 = poisoned((m + TAIL, n), BF16, dev), poisoned((m + TAIL, n), BF16, dev)
    moe.moe_grouped_gated_gemm_bf16(x, w, off, h, gate_up=keep, activation=act)
    moe.moe_grouped_gated_gemm_bf16(x, w, off, h2, activation=act)
    torch.cuda.synchronize()
    X.check_gated(x, w, off, act, h, keep)
    assert torch.equal(_bits(h), _bits(h2))
    assert_untouched(h[m:], "h behind the last expert")
    assert_untouched(keep[m:], "gate_up behind the last expert")


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("act,bias,residual,keep", [("none", False, False, False), ("gelu_tanh", True, True, True),
                                                    ("silu", True, False, True), ("relu", False, True, False)])
def test_linear_forward(hip_device, shape, act, bias, residual, keep):
    counts, n, k = shape
    dev = hip_device
    _say("linear %s act=%s" % (_id(shape), act))
    m, e = sum(counts), len(counts)
    off, x = offsets(counts, dev), rows_of(counts, k, 3, dev)
    w = randn((e, n, k), 4, dev, k**-0.5)
    b = randn((e, n), 5, dev) if bias else None
    r = rows_of(counts, n, 6, dev) if residual else None
    pre = poisoned((m + TAIL, n), BF16, dev) if keep else None
    y = poisoned((m + TAIL, n), BF16, dev)
    moe.moe_grouped_linear_bf16(x, w, off, y, bias=b, residual=r, pre_activation=pre, activation=act)
    torch.cuda.synchronize()
    X.check_linear(x, w, b, r, off, act, y, pre)
    assert_untouched(y[m:], "y behind the last expert")
    if keep:
        assert_untouched(pre[m:], "pre_activation behind the last expert")


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward(hip_device, shape, act):
    counts, n, k = shape
    dev = hip_device
    _say("gated backward %s act=%s" % (_id(shape), act))
    m, e = sum(counts), len(counts)
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w = randn((e, 2 * n, k), 2, dev, k**-0.5)
    gate_up, d_h = rows_of(counts, 2 * n, 7, dev), rows_of(counts, n, 8, dev)
    d_gu, d_x = poisoned((m + TAIL, 2 * n), BF16, dev), poisoned((m + TAIL, k), BF16, dev)
    d_w = poisoned((e, 2 * n, k), BF16, dev)
    moe.moe_grouped_gated_gemm_backward_bf16(d_h, gate_up, x, w, off, d_gu, d_x=d_x, d_w=d_w, activation=act)
    torch.cuda.synchronize()
    X.check_gated_slopes(d_h, gate_up, off, act, d_gu)
    X.check_products(d_gu, x, w, off, d_x, d_w)
    for t, name in ((d_gu, "d_gate_up"), (d_x, "d_x")):
        assert_untouched(t[m:], name + " behind the last expert")


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_linear_backward(hip_device, shape, act):
    counts, n, k = shape
    dev = hip_device
    _say("linear backward %s act=%s" % (_id(shape), act))
    m, e = sum(counts), len(counts)
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w = randn((e, n, k), 2, dev, k**-0.5)
    d_y = rows_of(counts, n, 9, dev)
    pre = rows_of(counts, n, 10, dev) if act != "none" else None
    d_z = poisoned((m + TAIL, n), BF16, dev) if act != "none" else None
    d_x, d_w = poisoned((m + TAIL, k), BF16, dev), poisoned((e, n, k), BF16, dev)
    d_b = poisoned((e, n), BF16, dev)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=d_x, d_w=d_w, d_bias=d_b, pre_activation=pre,
                                         d_pre_activation=d_z, activation=act)
    torch.cuda.synchronize()
    if act != "none":
        X.check_slopes(d_y, pre, off, act, d_z)
        assert_untouched(d_z[m:], "d_pre_activation behind the last expert")
    X.check_products(d_y if act == "none" else d_z, x, w, off, d_x, d_w, d_b)
    assert_untouched(d_x[m:], "d_x behind the last expert")


def test_backward_outputs_one_at_a_time(hip_device):
    """Each output alone: the products' bits are those of the full call."""
    dev = hip_device
    counts, n, k = [70, 0, 200], 136, 264
    m, e = sum(counts), 3
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w, d_y = randn((e, n, k), 2, dev, k**-0.5), rows_of(counts, n, 3, dev)
    full = [poisoned((m + TAIL, k), BF16, dev), poisoned((e, n, k), BF16, dev), poisoned((e, n), BF16, dev)]
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=full[0], d_w=full[1], d_bias=full[2])
    for i, name in enumerate(("d_x", "d_w", "d_bias")):
        one = poisoned(tuple(full[i].shape), BF16, dev)
        moe.moe_grouped_linear_backward_bf16(d_y, None if name == "d_x" else x, w, off, **{name: one})
        torch.cuda.synchronize()
        if name == "d_bias":  # summed in another order than beside d_w
            X.check_products(d_y, x, w, off, None, None, one)
        else:
            assert torch.equal(_bits(one), _bits(full[i])), name


# Tile sizes of the input's and the weight's gradient: both small, large and
# small, small and large, both large; a second launch for the remainders where the
# input's gradient is the only one; an expert with few rows beside them
@pytest.mark.parametrize("shape", [([90, 0, 110], 136, 72), ([4104], 72, 2312), ([120] * 15 + [1], 520, 2312),
                                   ([700, 3, 1801, 2500], 2056, 2312), ([1024, 1025, 1134, 1023], 1032, 3960)], ids=_id)
def test_gradients_together_and_alone(hip_device, shape):
    """Both gradients in one call have the bits of each alone."""
    counts, n, k = shape
    dev = hip_device
    _say("gradients together and alone %s" % _id(shape))
    m, e = sum(counts), len(counts)
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w, d_y = randn((e, n, k), 2, dev, k**-0.5), rows_of(counts, n, 3, dev)
    both = [poisoned((m + TAIL, k), BF16, dev), poisoned((e, n, k), BF16, dev)]
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=both[0], d_w=both[1])
    torch.cuda.synchronize()
    X.check_products(d_y, x, w, off, both[0], both[1])
    assert_untouched(both[0][m:], "d_x behind the last expert")
    for name, whole in zip(("d_x", "d_w"), both):
        one = poisoned(tuple(whole.shape), BF16, dev)
        moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, **{name: one})
        torch.cuda.synchronize()
        assert torch.equal(_bits(one), _bits(whole)), name


def test_no_rows_at_all(hip_device):
    """max_rows of 0: the forward writes nothing, the weights' gradients are zeros."""
    dev = hip_device
    off = offsets([0, 0], dev)
    x, d_y = torch.empty(0, 64, dtype=BF16, device=dev), torch.empty(0, 48, dtype=BF16, device=dev)
    w = randn((2, 48, 64), 1, dev)
    moe.moe_grouped_linear_bf16(x, w, off, torch.empty_like(d_y))
    d_w, d_b = poisoned((2, 48, 64), BF16, dev), poisoned((2, 48), BF16, dev)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=torch.empty_like(x), d_w=d_w, d_bias=d_b)
    torch.cuda.synchronize()
    assert not d_w.any() and not d_b.any()


# the last: every difference is positive once it wraps around 2^64
BAD_OFFSETS = [[0, 5, 3, 9], [1, 3, 5, 9], [0, 3, 5, 400], [-1, -1, -1, -1], [0, 3, -2, 9], [0, 2**63 - 1, -2, 9]]


@pytest.mark.parametrize("off", BAD_OFFSETS, ids=str)
def test_bad_offsets_write_nothing(hip_device, off):
    dev = hip_device
    n, k, m, e = 136, 72, 9, 3
    _say("bad offsets %s" % off)
    o = torch.tensor(off, dtype=torch.int64, device=dev)
    x, w = randn((m, k), 1, dev), randn((e, n, k), 2, dev)
    wg, gu = randn((e, 2 * n, k), 3, dev), randn((m, 2 * n), 4, dev)
    d_y = randn((m, n), 5, dev)
    outs = {}

    def out(name, *shape):
        outs[name] = poisoned(shape, BF16, dev)
        return outs[name]

    moe.moe_grouped_linear_bf16(x, w, o, out("y", m, n), pre_activation=out("pre", m, n), activation="silu")
    moe.moe_grouped_gated_gemm_bf16(x, wg, o, out("h", m, n), gate_up=out("gate_up", m, 2 * n))
    moe.moe_grouped_gated_gemm_backward_bf16(d_y, gu, x, wg, o, out("d_gate_up", m, 2 * n), d_x=out("d_x", m, k),
                                             d_w=out("d_w", e, 2 * n, k))
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, o, d_x=out("d_x2", m, k), d_w=out("d_w2", e, n, k),
                                         d_bias=out("d_b", e, n), pre_activation=d_y.clone(),
                                         d_pre_activation=out("d_z", m, n), activation="relu")
    torch.cuda.synchronize()
    for name, t in outs.items():
        assert_untouched(t, name)


@pytest.mark.parametrize("act", ACTS)
def test_far_and_special_pre_activations(hip_device, act):
    """Slopes at 0, far out (where exp and cubes overflow), at infinities and NaN."""
    dev = hip_device
    vals = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 3, -3, 12, -12, 29, -29, 31, -31, 90, -90, 1e4, -1e4, 1e20, -1e20,
            3e38, -3e38, float("nan"), 1.0]
    z = torch.tensor([vals], dtype=BF16, device=dev)
    d_y = torch.full_like(z, 0.75)
    off = torch.tensor([0, 1], dtype=torch.int64, device=dev)
    n = z.shape[1]
    w, x = randn((1, n, 8), 1, dev), randn((1, 8), 2, dev)
    ref = torch.nan_to_num(X.f64(z), nan=0.0)
    far = ref.abs() > 40
    slope = X.act_slope(torch.where(far, torch.zeros_like(ref), ref), act)
    if act != "none":
        slope = torch.where(far, (ref > 0).double(), slope)
        d_z = poisoned((1, n), BF16, dev)
        moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, pre_activation=z, d_pre_activation=d_z, activation=act)
        torch.cuda.synchronize()
        want = 0.75 * slope
        nan = torch.isnan(X.f64(z)) & (act != "relu")  # relu: a NaN is not above 0, so its slope is 0
        want[nan] = float("nan")
        X.assert_within(d_z, want, X.HALF * want.abs().nan_to_num(0) + X.SLOPE, "slope")


def test_masked_rows_infinities_stay_in_their_rows(hip_device):
    """A row of infinities or NaN changes that row alone; an expert's NaN weights change its rows alone."""
    dev = hip_device
    counts, n, k = [40, 0, 70], 72, 136
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w = randn((3, 2 * n, k), 2, dev, k**-0.5)
    clean, dirty = poisoned((113, n), BF16, dev), poisoned((113, n), BF16, dev)
    moe.moe_grouped_gated_gemm_bf16(x, w, off, clean)
    x2, w2 = x.clone(), w.clone()
    x2[7] = float("inf")
    x2[50, 3] = float("nan")
    w2[1] = float("nan")  # the expert without rows
    moe.moe_grouped_gated_gemm_bf16(x2, w2, off, dirty)
    torch.cuda.synchronize()
    keep = [i for i in range(110) if i not in (7, 50)]
    assert torch.equal(_bits(clean[keep]), _bits(dirty[keep]))
    assert not torch.isfinite(dirty[50].float()).any()


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[-1]], ids=_id)
def test_repeated_calls_give_the_same_bits(hip_device, shape):
    """No sum depends on timing: three calls, the same bits."""
    counts, n, k = shape
    dev = hip_device
    m, e = sum(counts), len(counts)
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w, d_y = randn((e, n, k), 2, dev, k**-0.5), rows_of(counts, n, 3, dev)
    first = None
    for _ in range(3):
        outs = [poisoned((m + TAIL, n), BF16, dev), poisoned((m + TAIL, k), BF16, dev), poisoned((e, n, k), BF16, dev),
                poisoned((e, n), BF16, dev)]
        moe.moe_grouped_linear_bf16(x, w, off, outs[0])
        moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=outs[1], d_w=outs[2], d_bias=outs[3])
        torch.cuda.synchronize()
        bits = [_bits(t) for t in outs]
        first = first or bits
        assert all(torch.equal(a, b) for a, b in zip(first, bits))


def test_row_offsets_past_32_bits(hip_device):
    """600001 rows of 4096: elements pass 2^31 and bytes 2^32; a k-loop of 300000 rows."""
    dev = hip_device
    counts, n, k = [300000, 300001], 64, 4096
    m = sum(counts)
    _say("row offsets past 32 bits: %d rows of %d" % (m, k))
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(m, k, generator=g, device=dev, dtype=BF16)
    w, off = randn((2, n, k), 2, dev, k**-0.5), offsets(counts, dev)
    d_y = torch.randn(m, n, generator=g, device=dev, dtype=BF16)
    y, d_x = poisoned((m, n), BF16, dev), poisoned((m, k), BF16, dev)
    d_w, d_b = poisoned((2, n, k), BF16, dev), poisoned((2, n), BF16, dev)
    moe.moe_grouped_linear_bf16(x, w, off, y)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=d_x, d_w=d_w, d_bias=d_b)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, 255, 256, 299998, 299999, 300000, 300001, 524287, 524288, 599999, 600000], device=dev)
    part = torch.tensor([0, 6, 12])
    X.check_linear(x[pick], w, None, None, part, "none", y[pick], None)
    X.check_products(d_y[pick], None, w, part, d_x[pick], None)
    for e, lo, hi in X.segments(off.cpu()):
        ref, mag = torch.zeros(n, k, dtype=torch.float64, device=dev), torch.zeros(n, k, dtype=torch.float64, device=dev)
        ref_b, mag_b = 0.0, 0.0
        for at in range(lo, hi, 20000):
            rows = slice(at, min(at + 20000, hi))
            d, xs = d_y[rows].double().t().contiguous(), x[rows].double()
            ref += torch.mm(d, xs)
            mag += torch.mm(d.abs(), xs.abs())
            ref_b, mag_b = ref_b + d.sum(1), mag_b + d.abs().sum(1)
        t = X.accumulate(hi - lo)
        X.assert_within(d_w[e], ref.cpu(), X.HALF * ref.abs().cpu() + t * mag.cpu(), "d_w")
        X.assert_within(d_b[e], ref_b.cpu(), X.HALF * ref_b.abs().cpu() + t * mag_b.cpu(), "d_bias")


def test_unpermute_backward_past_32_bits(hip_device):
    dev = hip_device
    n, k, h = 150000, 2, 8192
    _say("unpermute backward past 32 bits: %d rows of %d" % (n * k, h))
    g = torch.Generator(device=dev).manual_seed(1)
    d_out = torch.randn(n, h, generator=g, device=dev, dtype=BF16)
    y = torch.randn(n * k, h, generator=g, device=dev, dtype=BF16)
    wts = torch.rand(n, k, generator=g, device=dev)
    inv = torch.randperm(n * k, generator=g, device=dev).int()
    d_y, d_w = poisoned((n * k, h), BF16, dev), poisoned((n, k), torch.float32, dev)
    moe.moe_unpermute_backward(d_out, y, wts, inv, d_expanded_output=d_y, d_topk_weights=d_w)
    torch.cuda.synchronize()
    for t in (0, 1, 77777, n - 2, n - 1):
        for i in range(k):
            j = int(inv[t * k + i])
            ref = X.f64(wts[t, i]) * X.f64(d_out[t])
            X.assert_within(d_y[j], ref, (X.HALF + 2.0**-24) * ref.abs(), "row %d" % j)
            prod = X.f64(d_out[t]) * X.f64(y[j])
            X.assert_within(d_w[t, i:i + 1], prod.sum()[None], X.accumulate(h) * prod.abs().sum()[None], "weight")


# ------------------------------------------------------------ unpermute backward

UNPERMUTE = [(1, 1, 8), (1, 8, 64), (5, 3, 72), (33, 2, 520), (16, 8, 1032), (200, 1, 256), (7, 4, 4104), (3, 11, 128)]


@pytest.mark.parametrize("shape", UNPERMUTE, ids=str)
@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["all", "local", "none"])
def test_unpermute_backward(hip_device, shape, dtype, kind):
    dev = hip_device
    n, k, h = shape
    _say("unpermute backward N=%d topk=%d H=%d %s %s" % (n, k, h, dtype, kind))
    rng = np.random.default_rng(n * 100 + k)
    here = rng.random(n * k) < {"all": 1.1, "local": 0.4, "none": -1.0}[kind]
    inv = np.full(n * k, -1, dtype=np.int32)
    inv[here] = rng.permutation(int(here.sum()))
    inv = torch.from_numpy(inv).to(dev)
    d_out, y = randn((n, h), 1, dev, dtype=dtype), randn((n * k, h), 2, dev, dtype=dtype)
    wts = torch.rand(n, k, generator=torch.Generator().manual_seed(3)).to(dev)
    d_y, d_w = poisoned((n * k, h), dtype, dev), poisoned((n, k), torch.float32, dev)
    moe.moe_unpermute_backward(d_out, y, wts, inv, d_expanded_output=d_y, d_topk_weights=d_w)
    torch.cuda.synchronize()
    rows, ref_w, mag = X.unpermute_backward(d_out, y, wts, inv.cpu())
    half = X.HALF if dtype == BF16 else 2.0**-24
    for j, ref in rows.items():  # one product in fp32, one rounding to the type
        X.assert_within(d_y[j], ref, (half + 2.0**-24) * ref.abs(), "row %d" % j)
    for j in set(range(n * k)) - set(rows):
        assert_untouched(d_y[j], "row %d" % j)
    X.assert_within(d_w, ref_w, X.accumulate(h) * mag, "d_topk_weights")
    for only in ("d_expanded_output", "d_topk_weights"):  # each alone gives the same bits
        full = d_y if only == "d_expanded_output" else d_w
        one = poisoned(tuple(full.shape), full.dtype, dev)
        moe.moe_unpermute_backward(d_out, None if only == "d_expanded_output" else y, wts, inv, **{only: one})
        torch.cuda.synchronize()
        assert torch.equal(_bits(one), _bits(full))


def test_unpermute_backward_bad_entries(hip_device):
    dev = hip_device
    n, k, h = 6, 2, 64
    inv = torch.tensor([0, 1, 12, 2, -2, 3, 2**31 - 1, 4, -(2**31), 5, -1, 6], dtype=torch.int32, device=dev)
    d_out, y = randn((n, h), 1, dev), randn((n * k, h), 2, dev)
    wts = torch.rand(n, k, generator=torch.Generator().manual_seed(3)).to(dev)
    d_y, d_w = poisoned((n * k, h), BF16, dev), poisoned((n, k), torch.float32, dev)
    moe.moe_unpermute_backward(d_out, y, wts, inv, d_expanded_output=d_y, d_topk_weights=d_w)
    torch.cuda.synchronize()
    rows, ref_w, mag = X.unpermute_backward(d_out, y, wts, inv.cpu())
    assert set(rows) == set(range(7))
    for j, ref in rows.items():
        X.assert_within(d_y[j], ref, (X.HALF + 2.0**-24) * ref.abs(), "row %d" % j)
    assert_untouched(d_y[7:], "rows that no slot names")
    X.assert_within(d_w, ref_w, X.accumulate(h) * mag, "d_topk_weights")
    assert torch.isnan(d_w.view(-1)[[2, 4, 6, 8]]).all() and float(d_w.view(-1)[10]) == 0.0


# ------------------------------------------------------------ a whole block

class Block:
    """Permute, gated layer, down layer, unpermute, and back, in buffers kept by the caller."""

    def __init__(self, dev, n, topk, e, hidden, width, seed=0):
        rng = np.random.default_rng(seed)
        self.e, self.n, self.topk = e, n, topk
        ids = np.argsort(rng.random((n, e)), axis=1)[:, :topk].astype(np.int32)
        self.ids = torch.from_numpy(ids).to(dev)
        self.wts = torch.softmax(randn((n, topk), seed + 1, dev, dtype=torch.float32), 1)
        self.x, self.d_out = randn((n, hidden), seed + 2, dev), randn((n, hidden), seed + 3, dev)
        self.w13 = randn((e, 2 * width, hidden), seed + 4, dev, hidden**-0.5)
        self.w2, self.b2 = randn((e, hidden, width), seed + 5, dev, width**-0.5), randn((e, hidden), seed + 6, dev)
        rows = n * topk
        self.idx = {
            "permuted_hidden_states": poisoned((rows, hidden), BF16, dev),
            "permuted_scale": None,
            "expert_first_token_offset": poisoned((e + 1,), torch.int64, dev),
            "permuted_idx": poisoned((rows,), torch.int32, dev),
            "inv_permuted_idx": poisoned((rows,), torch.int32, dev),
        }
        ws = binding.moe_permute_workspace_size(n, topk, e)
        self.ws = poisoned((max(ws, 16),), torch.uint8, dev)
        self.out = {name: poisoned(shape, BF16, dev) for name, shape in dict(
            h=(rows, width), gate_up=(rows, 2 * width), y=(rows, hidden), out=(n, hidden), d_y=(rows, hidden),
            d_h=(rows, width), d_w2=(e, hidden, width), d_b2=(e, hidden), d_gate_up=(rows, 2 * width),
            d_xp=(rows, hidden), d_w13=(e, 2 * width, hidden), d_x=(n, hidden)).items()}
        self.out["d_wts"] = poisoned((n, topk), torch.float32, dev)
        self.ones = torch.ones(n, topk, device=dev)

    def run(self, stream=None):
        o, idx = self.out, self.idx
        gpu_permute(self.x, self.ids, self.e, workspace=self.ws, stream=stream, outs=idx)
        xp, off, inv = idx["permuted_hidden_states"], idx["expert_first_token_offset"], idx["inv_permuted_idx"]
        moe.moe_grouped_gated_gemm_bf16(xp, self.w13, off, o["h"], gate_up=o["gate_up"], stream=stream)
        moe.moe_grouped_linear_bf16(o["h"], self.w2, off, o["y"], bias=self.b2, stream=stream)
        binding.moe_unpermute(o["y"], self.wts, inv, o["out"], stream=stream)
        moe.moe_unpermute_backward(self.d_out, o["y"], self.wts, inv, d_expanded_output=o["d_y"],
                                   d_topk_weights=o["d_wts"], stream=stream)
        moe.moe_grouped_linear_backward_bf16(o["d_y"], o["h"], self.w2, off, d_x=o["d_h"], d_w=o["d_w2"],
                                             d_bias=o["d_b2"], stream=stream)
        moe.moe_grouped_gated_gemm_backward_bf16(o["d_h"], o["gate_up"], xp, self.w13, off, o["d_gate_up"],
                                                 d_x=o["d_xp"], d_w=o["d_w13"], stream=stream)
        binding.moe_unpermute(o["d_xp"], self.ones, inv, o["d_x"], stream=stream)  # the permute's backward

    def check(self):
        """Every step against its 64-bit reference, from the inputs that the step had."""
        o, idx = self.out, self.idx
        xp, off, inv = idx["permuted_hidden_states"], idx["expert_first_token_offset"], idx["inv_permuted_idx"]
        X.check_gated(xp, self.w13, off, "silu", o["h"], o["gate_up"])
        X.check_linear(o["h"], self.w2, self.b2, None, off, "none", o["y"], None)
        rows, ref_w, mag = X.unpermute_backward(self.d_out, o["y"], self.wts, inv.cpu())
        ref = torch.stack([rows[j] for j in range(len(rows))])
        X.assert_within(o["d_y"], ref, (X.HALF + 2.0**-24) * ref.abs(), "d_y")
        X.assert_within(o["d_wts"], ref_w, X.accumulate(self.x.shape[1]) * mag, "d_topk_weights")
        X.check_products(o["d_y"], o["h"], self.w2, off, o["d_h"], o["d_w2"], o["d_b2"])
        X.check_gated_slopes(o["d_h"], o["gate_up"], off, "silu", o["d_gate_up"])
        X.check_products(o["d_gate_up"], xp, self.w13, off, o["d_xp"], o["d_w13"])
        d_xp = X.f64(o["d_xp"])[inv.long().cpu()].view(self.n, self.topk, -1)
        ref = d_xp.sum(1)
        tol = X.HALF * ref.abs() + X.accumulate(self.topk) * d_xp.abs().sum(1)
        X.assert_within(o["d_x"], ref, tol, "d_x")


@pytest.mark.parametrize("n,topk,e,hidden,width", [(1, 2, 4, 256, 136), (150, 3, 7, 264, 104), (40, 8, 64, 512, 256)])
def test_block_forward_and_backward(hip_device, n, topk, e, hidden, width):
    _say("block N=%d topk=%d E=%d H=%d n=%d" % (n, topk, e, hidden, width))
    b = Block(hip_device, n, topk, e, hidden, width)
    b.run()
    torch.cuda.synchronize()
    b.check()


def test_block_on_another_stream(hip_device):
    b = Block(hip_device, 60, 2, 5, 128, 72)
    s = torch.cuda.Stream(device=hip_device)
    s.wait_stream(torch.cuda.current_stream(hip_device))
    b.run(stream=s)
    s.synchronize()
    b.check()


def test_block_captured_and_replayed(hip_device):
    """A captured block, replayed on new inputs with eager work between, gives the eager results each time."""
    a, ref = Block(hip_device, 90, 2, 6, 136, 96), Block(hip_device, 90, 2, 6, 136, 96)
    s = torch.cuda.Stream(device=hip_device)
    s.wait_stream(torch.cuda.current_stream(hip_device))
    with torch.cuda.stream(s):
        a.run()
    torch.cuda.current_stream(hip_device).wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for i in range(3):
        for b in (a, ref):
            b.x.copy_(randn(tuple(b.x.shape), 50 + i, hip_device))
            b.ids.copy_(torch.roll(b.ids, 1, 0))
            for t in b.out.values():
                t.view(torch.uint8).fill_(POISON)
        ref.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, t in a.out.items():
            assert torch.equal(_bits(t), _bits(ref.out[name])), "%s at replay %d" % (name, i)
    a.check()


def test_two_streams_at_once(hip_device):
    """Two blocks in flight on two streams (no shared state in the library)."""
    blocks = [Block(hip_device, 120, 2, 8, 256, 128, seed=s) for s in (0, 100)]
    streams = [torch.cuda.Stream(device=hip_device) for _ in blocks]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(hip_device))
    for _ in range(3):
        for b, s in zip(blocks, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b in blocks:
        b.check()
