"""GPU parity of the 8-bit expert path (include/moe_experts_8bit.h) against 64-bit references.

The bounds are derived in tests/_experts_8bit.py; codes, scales and indices are
compared for equality.  Every output is poisoned before the call, and rows
behind the last expert's (the buffers hold a few more than off[E]) must keep
the poison; what those rows hold in the inputs would be seen in the results.
"""

import numpy as np
import pytest
import torch

import oracle
import _experts as X
import _experts_8bit as E8
from _parity import POISON, poisoned, to_np
import mixture_experts_token_amd as moe
from mixture_experts_token_amd import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CODE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
KINDS = ["int8", "fp8"]
TAIL = 3  # rows behind the last expert's
LAYER = {("gated", "int8"): moe.moe_grouped_gated_gemm_int8, ("gated", "fp8"): moe.moe_grouped_gated_gemm_fp8,
         ("linear", "int8"): moe.moe_grouped_linear_int8, ("linear", "fp8"): moe.moe_grouped_linear_fp8}
QUANTIZE = {"int8": moe.moe_quantize_rows_int8, "fp8": moe.moe_quantize_rows_fp8}


def _say(msg):
    print("[case] " + msg, flush=True)


def _bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def assert_untouched(t, what):
    assert bool((t.contiguous().view(torch.uint8) == POISON).all()), what + " was written"


def offsets(counts, dev):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64, device=dev)


def rand_codes(shape, kind, seed, dev):
    """Codes of every finite value (int8 with -128 too, fp8 without NaN)."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    if kind == "int8":
        return torch.randint(-128, 128, shape, generator=g, dtype=torch.int32).to(torch.int8).to(dev)
    return (torch.randn(shape, generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn).to(dev)


def rand_scale(shape, seed, dev, top):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return ((torch.rand(shape, generator=g) + 0.5) * top).to(dev)


def row_codes(counts, k, kind, seed, dev):
    """Codes and scales of sum(counts) + TAIL rows; the rows behind the experts' have NaN scales (and fp8 NaN codes)."""
    m = sum(counts)
    x, s = rand_codes((m + TAIL, k), kind, seed, dev), rand_scale((m + TAIL,), seed + 1, dev, 0.01)
    s[m:] = float("nan")
    if kind == "fp8":
        x.view(torch.uint8)[m:] = 0x7F
    return x, s


def randn(shape, seed, dev, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev)


# (rows of each expert, n, k): one row; empty experts; sizes that fill no tile or
# k-step; whole tiles; decode sizes with k of every kind; experts longer than a
# tile; experts on both sides of the limits of the forms for few rows
SHAPES = [
    ([1], 8, 16),
    ([0, 1, 0], 64, 64),
    ([0, 0], 72, 16),
    ([3, 0, 130, 1, 64], 264, 208),
    ([513, 0, 256], 512, 1024),
    ([65, 127, 129], 136, 80),
    ([1, 1, 1, 1, 1, 1, 1, 1], 520, 2048),
    ([1, 0, 2, 1, 0, 3, 1, 1], 96, 1008),
    ([2, 2, 0, 1], 256, 8208),
    ([17, 5, 9, 33], 1032, 448),
    ([16, 15, 32, 31, 0, 33, 1], 200, 4112),
    ([300] + [0] * 30 + [5], 128, 128),
    ([1] * 1024, 40, 64),
    ([9, 1, 3, 8, 0, 4], 72, 1104),
    ([0, 5, 1], 136, 16400),
    ([2, 0, 1], 40, 33040),
    ([1, 0, 2] * 15 + [190, 33, 32], 136, 1104),
    ([1500, 0, 700, 257, 1000, 3], 3864, 528),
    ([700, 0, 1, 410], 1800, 2000),
    ([1024, 1025, 1134, 1023], 3960, 1040),
    # more experts than lanes look at once, in tiles; rows per expert at which the
    # streamed rows per pass change, with experts of more passes than are streamed
    ([13 + e % 3 for e in range(1024)], 24, 48),
    ([2, 1, 2, 30, 0, 2, 3, 1, 0, 1], 72, 784),
    ([3, 9, 16, 17, 0, 1, 70, 4], 264, 2064),
    ([1, 2, 0, 1, 0, 0, 17, 0, 1, 0, 1, 0] * 2, 40, 1296),
]
ACTS = ["silu", "gelu_tanh", "relu", "none"]


def _id(v):
    return "rows%d-%dx%d" % (sum(v[0]), v[1], v[2])


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("kind,act", [("int8", "silu"), ("fp8", "silu"), ("int8", "gelu_tanh"), ("fp8", "relu"),
                                      ("int8", "none")])
def test_gated(hip_device, shape, kind, act):
    counts, n, k = shape
    dev, m, e = hip_device, sum(shape[0]), len(shape[0])
    _say("gated %s %s act=%s" % (kind, _id(shape), act))
    off = offsets(counts, dev)
    x, xs = row_codes(counts, k, kind, 1, dev)
    w, ws = rand_codes((e, 2 * n, k), kind, 3, dev), rand_scale((e, 2 * n), 4, dev, 0.02 * k**-0.5)
    h = poisoned((m + TAIL, n), BF16, dev)
    LAYER["gated", kind](x, xs, w, ws, off, h, activation=act)
    torch.cuda.synchronize()
    E8.check_gated(x, xs, w, ws, off, kind, act, h)
    assert_untouched(h[m:], "h behind the last expert")


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
@pytest.mark.parametrize("kind,act,bias,residual", [("int8", "none", False, False), ("fp8", "none", False, False),
                                                    ("int8", "gelu_tanh", True, True), ("fp8", "silu", True, False),
                                                    ("int8", "relu", False, True), ("fp8", "gelu_tanh", True, True)])
def test_linear(hip_device, shape, kind, act, bias, residual):
    counts, n, k = shape
    dev, m, e = hip_device, sum(shape[0]), len(shape[0])
    _say("linear %s %s act=%s" % (kind, _id(shape), act))
    off = offsets(counts, dev)
    x, xs = row_codes(counts, k, kind, 5, dev)
    w, ws = rand_codes((e, n, k), kind, 7, dev), rand_scale((e, n), 8, dev, 0.02 * k**-0.5)
    b = randn((e, n), 9, dev) if bias else None
    r = randn((m + TAIL, n), 10, dev) if residual else None
    y = poisoned((m + TAIL, n), BF16, dev)
    LAYER["linear", kind](x, xs, w, ws, off, y, bias=b, residual=r, activation=act)
    torch.cuda.synchronize()
    E8.check_linear(x, xs, w, ws, b, r, off, kind, act, y)
    assert_untouched(y[m:], "y behind the last expert")


@pytest.mark.parametrize("shape", SHAPES, ids=_id)
def test_fp8_sums_of_small_whole_numbers_are_exact(hip_device, shape):
    """Codes of whole numbers up to 8: products of at most 64, of which nothing is cut
    (2^(6 - 13) is below one), and sums below 2^24."""
    counts, n, k = shape
    dev, m, e = hip_device, sum(shape[0]), len(shape[0])
    _say("fp8 exact %s" % _id(shape))
    g = torch.Generator(device="cpu").manual_seed(11)
    off = offsets(counts, dev)

    def whole(*size):
        return torch.randint(-8, 9, size, generator=g).float().to(torch.float8_e4m3fn)

    x, w = whole(m + TAIL, k), whole(e, n, k)
    xs = 2.0 ** torch.randint(-3, 3, (m + TAIL,), generator=g)
    ws = 2.0 ** torch.randint(-3, 3, (e, n), generator=g)
    y = poisoned((m + TAIL, n), BF16, dev)
    moe.moe_grouped_linear_fp8(x.to(dev), xs.to(dev), w.to(dev), ws.to(dev), off, y)
    torch.cuda.synchronize()
    want = torch.zeros(m, n, dtype=torch.float64)
    for i, lo, hi in X.segments(off):
        want[lo:hi] = (x[lo:hi].double() @ w[i].double().t()) * xs[lo:hi, None] * ws[i]
    assert torch.equal(y[:m].cpu(), want.float().to(BF16))
    assert_untouched(y[m:], "y behind the last expert")


@pytest.mark.parametrize("counts", [[1, 0, 2], [40, 3, 0], [300, 500, 0]], ids=str)
def test_int8_sums_are_exact(hip_device, counts):
    """Sums that pass 2^29 on the way and end at a small number: with scales of one
    that number, which a bf16 holds."""
    dev, n, k = hip_device, 72, 131056  # the longest int8 row
    m, e = sum(counts), len(counts)
    off = offsets(counts, dev)
    x = torch.full((m + TAIL, k), 127, dtype=torch.int8)
    x[:, k // 2:] = -127
    w = torch.full((e, n, k), 100, dtype=torch.int8)
    a, d = torch.arange(m + TAIL) % 2, torch.arange(n) % 3 - 1
    x[:, k - 1] += a.to(torch.int8)               # adds 100 a
    w[:, :, k - 2] += d.to(torch.int8)            # takes off 127 d
    y = poisoned((m + TAIL, n), BF16, dev)
    moe.moe_grouped_linear_int8(x.to(dev), torch.ones(m + TAIL, device=dev), w.to(dev),
                                torch.ones(e, n, device=dev), off, y)
    torch.cuda.synchronize()
    assert torch.equal(y[:m].cpu().float(), (100.0 * a[:m, None] - 127.0 * d))
    assert_untouched(y[m:], "y behind the last expert")


@pytest.mark.parametrize("counts", [[1], [20], [200, 90]], ids=str)
def test_int8_extremes_fit_32_bits(hip_device, counts):
    """The longest row, every code -128: the sum is 2^14 k, below 2^31."""
    dev, n, k = hip_device, 8, 131056
    m, e = sum(counts), len(counts)
    off = offsets(counts, dev)
    x, w = torch.full((m, k), -128, dtype=torch.int8, device=dev), torch.full((e, n, k), -128, dtype=torch.int8, device=dev)
    y = poisoned((m, n), BF16, dev)
    moe.moe_grouped_linear_int8(x, torch.ones(m, device=dev), w, torch.full((e, n), 2.0**-14, device=dev), off, y)
    torch.cuda.synchronize()
    assert bool((y == torch.tensor(float(k)).to(BF16).to(dev)).all())


@pytest.mark.parametrize("counts", [[3, 0, 1], [40, 0, 30], [300, 200, 1]], ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_special_rows_and_channels_stay_their_own(hip_device, counts, kind):
    """NaN and infinite scales and fp8 NaN codes show in their row or channel alone."""
    dev, n, k = hip_device, 136, 272
    m, e = sum(counts), len(counts)
    off = offsets(counts, dev)
    x, xs = row_codes(counts, k, kind, 1, dev)
    w, ws = rand_codes((e, n, k), kind, 3, dev), rand_scale((e, n), 4, dev, 1e-3)
    y0, y1 = poisoned((m + TAIL, n), BF16, dev), poisoned((m + TAIL, n), BF16, dev)
    call = LAYER["linear", kind]
    call(x, xs, w, ws, off, y0)
    xs[1] = float("nan")
    x.view(torch.uint8)[2] = 0
    xs[2] = float("inf")
    ws[:, 5] = float("nan")
    if kind == "fp8":
        w.view(torch.uint8)[:, 7, k - 1] = 0x7F
    call(x, xs, w, ws, off, y1)
    torch.cuda.synchronize()
    same = torch.ones(m, n, dtype=torch.bool)
    same[1:3] = False
    same[:, 5] = False
    if kind == "fp8":
        same[:, 7] = False
    nan = torch.isnan(y1[:m].cpu().float())
    assert bool(nan[~same].all()) and not bool(nan[same].any())  # row 2 is 0 times infinity
    assert torch.equal(y1[:m].cpu()[same], y0[:m].cpu()[same])


BAD = [[1, 2, 3, 4], [0, 5, 4, 6], [-1, -1, -1, -1], [0, 2, 4, 1 << 40], [0, 1, 2, 9], [0, -(1 << 63), 2, 4],
       [0, (1 << 63) - 1, 3, 4]]


@pytest.mark.parametrize("off", BAD, ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_bad_offsets_write_nothing(hip_device, kind, off):
    dev, rows = hip_device, 8
    off = torch.tensor(off, dtype=torch.int64, device=dev)
    x, xs = rand_codes((rows, 64), kind, 1, dev), rand_scale((rows,), 2, dev, 1.0)
    w, ws = rand_codes((3, 64, 64), kind, 3, dev), rand_scale((3, 64), 4, dev, 1.0)
    h, y = poisoned((rows, 32), BF16, dev), poisoned((rows, 64), BF16, dev)
    codes, scale = poisoned((rows, 64), torch.uint8, dev), poisoned((rows,), F32, dev)
    LAYER["gated", kind](x, xs, w, ws, off, h)
    LAYER["linear", kind](x, xs, w, ws, off, y)
    QUANTIZE[kind](randn((rows, 64), 5, dev), codes.view(CODE[kind]), scale, expert_first_token_offset=off)
    torch.cuda.synchronize()
    for t in (h, y, codes, scale):
        assert_untouched(t, "an output")


def special_rows(x, top):
    """Rows that the quantisers have to get right, written over the first ones of x where they fit."""
    n = x.shape[1]
    ramp = torch.arange(n, dtype=torch.float64)
    ties = (ramp.remainder(2 * top) - top + 0.5).clamp(-top, top)  # a half beside every whole number
    ties[0] = top
    rows = [torch.zeros(n, dtype=torch.float64), ties, ties * 2.0**-40, ties * 2.0**90, -ties * 2.0**-126,
            ties * 2.0**-132, ties / 3, torch.full((n,), float("nan"), dtype=torch.float64)]
    one_nan, one_inf, big = torch.ones(n, dtype=torch.float64), torch.ones(n, dtype=torch.float64), ties.clone()
    one_nan[n // 2], one_inf[n - 1] = float("nan"), -float("inf")
    big[0] = 3.3e38
    for i, r in enumerate(rows + [one_nan, one_inf, big]):
        if i < x.shape[0]:
            x[i] = r.to(x.dtype)
    return x


# lengths held by a wave, by a workgroup of 4, 8 and 16 waves, and by none
LENGTHS = [(1, 8, BF16), (5, 4, F32), (7, 64, BF16), (40, 520, BF16), (1, 7168, BF16), (1500, 520, BF16),
           (1030, 2048, BF16), (1025, 1020, F32), (300, 2056, BF16), (33, 8192, BF16), (20, 8200, BF16),
           (13, 14336, BF16), (12, 8196, F32), (11, 16392, BF16), (11, 32768, BF16), (12, 32776, BF16),
           (11, 100004, F32), (600, 16384, F32)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n,dtype", LENGTHS)
@pytest.mark.parametrize("grouped", [False, True])
def test_quantize_rows(hip_device, kind, rows, n, dtype, grouped):
    dev = hip_device
    _say("quantize %s rows=%d n=%d %s grouped=%s" % (kind, rows, n, dtype, grouped))
    g = torch.Generator(device="cpu").manual_seed(rows + n)
    mag = torch.exp(torch.randn((rows + TAIL, 1), generator=g) * 3)
    x = special_rows((torch.randn((rows + TAIL, n), generator=g) * mag).to(dtype), 127 if kind == "int8" else 448)
    x = x.to(dev)
    total = rows + TAIL
    codes, scale = poisoned((total, n), torch.uint8, dev), poisoned((total, 1), F32, dev)
    off, m = None, total
    if grouped:
        m = rows
        cut = sorted(torch.randint(0, rows + 1, (4,), generator=g).tolist())
        off = torch.tensor([0] + cut + [rows], dtype=torch.int64, device=dev)
    QUANTIZE[kind](x, codes.view(CODE[kind]), scale, expert_first_token_offset=off)
    torch.cuda.synchronize()
    want, want_scale = E8.codes_of(x[:m].cpu(), kind)
    got, want = codes[:m].cpu(), want.view(torch.uint8)
    bad = torch.nonzero(got != want)
    assert not len(bad), (len(bad), bad[0].tolist(), float(x[tuple(bad[0].tolist())]))
    gs = scale[:m, 0].cpu()
    assert torch.equal(torch.isnan(gs), torch.isnan(want_scale))
    assert torch.equal(gs[~torch.isnan(gs)], want_scale[~torch.isnan(gs)])
    if grouped:
        assert_untouched(codes[m:], "codes behind the last expert")
        assert_untouched(scale[m:], "scale behind the last expert")


def test_quantize_every_bf16(hip_device):
    """Every finite bf16 against many scales: a row holds 4096 values of one magnitude range and its largest."""
    dev = hip_device
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    allv = torch.cat([bits, bits | 0x8000]).to(torch.int16).view(BF16)
    order = torch.sort(allv.float().abs(), stable=True).indices
    v = allv[order]
    v = torch.cat([v, v[-(-v.numel() % 1024):]]) if v.numel() % 1024 else v
    x = v.view(-1, 1024).contiguous()
    wide = torch.cat([x, x.roll(1, 0) * 1.0], dim=1)[1:].contiguous()  # two neighbouring ranges
    for t in (x, wide):
        codes, scale = poisoned(tuple(t.shape), torch.int8, dev), poisoned((t.shape[0],), F32, dev)
        moe.moe_quantize_rows_int8(t.to(dev), codes, scale)
        want, want_scale = E8.int8_codes(t)
        assert torch.equal(codes.cpu(), want) and torch.equal(scale.cpu(), want_scale)


# (tokens, topk, experts, hidden, type, id type, local experts or None): the permute's wave, fused, coarse and
# staged schedules, each with and without a map
PERMUTES = [
    (1, 8, 256, 7168, BF16, torch.int32, None),
    (1, 1, 1, 8, BF16, torch.int64, None),
    (13, 3, 13, 424, F32, torch.int32, None),
    (100, 2, 8, 4096, BF16, torch.int64, 3),
    (1111, 3, 13, 424, F32, torch.int32, 6),
    (1500, 8, 128, 2048, BF16, torch.int32, None),
    (3000, 8, 64, 520, BF16, torch.int32, 16),
    (9000, 4, 256, 136, BF16, torch.int64, None),
    (70, 4, 16, 8192, BF16, torch.int32, None),
    (60000, 8, 256, 72, BF16, torch.int32, None),
]


@pytest.mark.parametrize("n,k,e,h,dtype,idt,local", PERMUTES)
def test_permute_quant_int8(hip_device, n, k, e, h, dtype, idt, local):
    dev = hip_device
    _say("permute %d %d %d %d" % (n, k, e, h))
    g = torch.Generator(device="cpu").manual_seed(n + h)
    x = special_rows((torch.randn((n, h), generator=g) * torch.exp(torch.randn((n, 1), generator=g) * 3)).to(dtype), 127)
    ids = torch.randint(0, e, (n, k), generator=g).to(idt)
    emap = None
    if local is not None:
        emap = np.full(e, -1, np.int32)
        emap[np.random.default_rng(n).permutation(e)[:local]] = np.arange(local)
    rows, buckets = n * k, e if local is None else local
    outs = {"codes": poisoned((rows, h), torch.int8, dev), "scale": poisoned((rows,), F32, dev),
            "off": poisoned((buckets + 1,), torch.int64, dev), "perm": poisoned((rows,), torch.int32, dev),
            "inv": poisoned((rows,), torch.int32, dev)}
    ws = (binding.moe_permute_workspace_size(n, k, e) if local is None
          else binding.moe_permute_local_workspace_size(n, k, e, local))
    moe.moe_permute_quant_int8(x.to(dev), ids.to(dev), e, outs["codes"], outs["scale"], outs["off"], outs["perm"],
                               outs["inv"], poisoned((max(ws, 16),), torch.uint8, dev),
                               expert_map=None if emap is None else torch.from_numpy(emap).to(dev),
                               num_local_experts=local or 0)
    torch.cuda.synchronize()
    empty = np.zeros((n, 0), np.float32)
    ref = oracle.permute(empty, to_np(ids), e) if local is None else oracle.permute_local(empty, to_np(ids), e, emap,
                                                                                           local)
    for key, name in (("off", "expert_first_token_offset"), ("inv", "inv_permuted_idx")):
        np.testing.assert_array_equal(to_np(outs[key]), ref[name])
    m = int(ref["expert_first_token_offset"][-1])
    perm = outs["perm"][:m].cpu()
    np.testing.assert_array_equal(perm.numpy(), ref["permuted_idx"][:m])
    codes, scale = E8.int8_codes(x)
    token = torch.div(perm.long(), k, rounding_mode="floor")
    assert torch.equal(outs["codes"][:m].cpu(), codes[token])
    got, want = outs["scale"][:m].cpu(), scale[token]
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])
    for key in ("codes", "scale", "perm"):
        assert_untouched(outs[key][m:], key + " behind the local rows")


@pytest.mark.parametrize("n", [5, 400])
def test_permute_bad_id_and_no_tokens(hip_device, n):
    dev, e, k, h = hip_device, 8, 2, 64
    ids = torch.zeros(n, k, dtype=torch.int32, device=dev)
    ids[n - 1, 1] = e
    codes, scale = poisoned((n * k, h), torch.int8, dev), poisoned((n * k,), F32, dev)
    off, perm, inv = (poisoned((s,), t, dev) for s, t in ((e + 1, torch.int64), (n * k, torch.int32),
                                                         (n * k, torch.int32)))
    moe.moe_permute_quant_int8(randn((n, h), 1, dev), ids, e, codes, scale, off, perm, inv)
    torch.cuda.synchronize()
    assert bool((off == -1).all())
    for t in (codes, scale, perm, inv):
        assert_untouched(t, "an output of a rejected id")
    moe.moe_permute_quant_int8(randn((0, h), 1, dev), ids[:0], e, codes[:0], scale[:0], off, perm[:0], inv[:0])
    torch.cuda.synchronize()
    assert bool((off == 0).all())


@pytest.mark.parametrize("kind", KINDS)
def test_no_rows_and_no_live_rows(hip_device, kind):
    dev = hip_device
    w, ws = rand_codes((3, 32, 64), kind, 1, dev), torch.ones(3, 32, device=dev)
    off = torch.zeros(4, dtype=torch.int64, device=dev)
    for rows in (0, 7, 700):
        x, xs = rand_codes((rows, 64), kind, 2, dev), torch.ones(rows, device=dev)
        h, y = poisoned((rows, 16), BF16, dev), poisoned((rows, 32), BF16, dev)
        codes, scale = poisoned((rows, 64), torch.uint8, dev), poisoned((rows,), F32, dev)
        LAYER["gated", kind](x, xs, w, ws, off, h)
        LAYER["linear", kind](x, xs, w, ws, off, y)
        QUANTIZE[kind](randn((rows, 64), 3, dev), codes.view(CODE[kind]), scale, expert_first_token_offset=off)
        torch.cuda.synchronize()
        for t in (h, y, codes, scale):
            assert_untouched(t, "an output without rows")


@pytest.mark.parametrize("shape", [([2, 1, 0, 1], 264, 2064), ([20, 33, 1, 9], 264, 2064), ([600, 0, 301], 520, 528)],
                         ids=_id)
@pytest.mark.parametrize("kind", KINDS)
def test_repeated_calls_give_the_same_bits(hip_device, shape, kind):
    counts, n, k = shape
    dev, m, e = hip_device, sum(shape[0]), len(shape[0])
    off = offsets(counts, dev)
    x, xs = row_codes(counts, k, kind, 1, dev)
    w, ws = rand_codes((e, 2 * n, k), kind, 3, dev), rand_scale((e, 2 * n), 4, dev, 1e-3)
    first = None
    for _ in range(20):
        h = poisoned((m + TAIL, n), BF16, dev)
        LAYER["gated", kind](x, xs, w, ws, off, h)
        torch.cuda.synchronize()
        first = _bits(h) if first is None else first
        assert torch.equal(_bits(h), first)


@pytest.mark.parametrize("kind", KINDS)
def test_row_offsets_past_32_bits(hip_device, kind):
    """Rows, codes and outputs whose byte offsets pass 2^32, and weights whose do."""
    dev, n, k, rows = hip_device, 24, 8192, 540000
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((rows, k), dtype=torch.uint8, device=dev)
    for i in range(0, rows, 60000):
        piece = x[i:i + 60000]
        piece.copy_(torch.randint(0, 0x70, piece.shape, generator=g, device=dev, dtype=torch.uint8))
    x = x.view(CODE[kind])
    xs = torch.full((rows,), 2.0**-10, device=dev)
    w, ws = rand_codes((2, n, k), kind, 3, dev), rand_scale((2, n), 4, dev, 1e-4)
    y = poisoned((rows, n), BF16, dev)
    last = rows - 5
    off = torch.tensor([0, 300000, last], dtype=torch.int64, device=dev)
    LAYER["linear", kind](x, xs, w, ws, off, y)
    torch.cuda.synchronize()
    for lo, hi, e in ((0, 40, 0), (299980, 300000, 0), (300000, 300020, 1), (last - 300, last, 1)):
        E8.check_linear(x[lo:hi], xs[lo:hi], w[e:e + 1], ws[e:e + 1], None, None, [0, hi - lo], kind, "none", y[lo:hi])
    assert_untouched(y[last:], "y behind the last expert")
    v = torch.empty((rows, k), dtype=BF16, device=dev)
    for i in range(0, rows, 60000):
        piece = v[i:i + 60000]
        piece.copy_(torch.randn(piece.shape, generator=g, device=dev))
    codes, scale = x.view(torch.uint8), xs
    codes[last:].fill_(POISON)
    QUANTIZE[kind](v, codes.view(CODE[kind]), scale, expert_first_token_offset=off)
    torch.cuda.synchronize()
    for lo, hi in ((0, 40), (299990, 300010), (last - 300, last)):
        want, want_scale = E8.codes_of(v[lo:hi].cpu(), kind)
        assert torch.equal(codes[lo:hi].cpu(), want.view(torch.uint8)) and torch.equal(scale[lo:hi].cpu(), want_scale)
    assert_untouched(codes[last:], "codes behind the last expert")


@pytest.mark.parametrize("counts", [[1], [10, 0, 3], [40, 60], [300]], ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_longest_rows(hip_device, kind, counts):
    """Codes of one against codes of one and of nought: the sum is the number of ones, which fp32 holds."""
    dev, n, k = hip_device, 40, 2**20 if kind == "fp8" else 131056
    m, e = sum(counts), len(counts)
    off = offsets(counts, dev)
    one = torch.ones(1).to(CODE[kind]).view(torch.uint8).item()
    x = torch.full((m, k), one, dtype=torch.uint8, device=dev).view(CODE[kind])
    w = torch.zeros((e, n, k), dtype=torch.uint8, device=dev)
    for c in range(n):
        w[:, c, : k - 16 * c].fill_(one)
        w[:, c, k - 1].fill_(one)
    y = poisoned((m, n), BF16, dev)
    LAYER["linear", kind](x, torch.full((m,), 0.5, device=dev), w.view(CODE[kind]), torch.ones(e, n, device=dev), off, y)
    torch.cuda.synchronize()
    want = torch.tensor([k if c == 0 else k - 16 * c + 1 for c in range(n)], dtype=torch.float64) * 0.5
    assert torch.equal(y.cpu(), want.float().to(BF16).expand(m, n))


@pytest.mark.parametrize("counts", [[1, 0], [9, 2], [50, 90]], ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_most_columns(hip_device, kind, counts):
    dev, n, k = hip_device, 2**20, 16
    m, e = sum(counts), len(counts)
    off = offsets(counts, dev)
    x, xs = row_codes(counts, k, kind, 1, dev)
    w, ws = rand_codes((e, 2 * n, k), kind, 3, dev), rand_scale((e, 2 * n), 4, dev, 1e-3)
    h = poisoned((m + TAIL, n), BF16, dev)
    LAYER["gated", kind](x, xs, w, ws, off, h)
    torch.cuda.synchronize()
    cols = torch.cat([torch.arange(0, 300), torch.arange(n // 2 - 150, n // 2 + 150), torch.arange(n - 300, n)]).to(dev)
    both = torch.cat([cols, cols + n])
    E8.check_gated(x, xs, w.view(torch.uint8)[:, both].view(CODE[kind]), ws[:, both], off, kind, "silu", h[:, cols])
    assert_untouched(h[m:], "h behind the last expert")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,max_rows", [([1, 0, 2], 4000), ([1, 0, 2], 30), ([40, 0, 3], 900), ([300, 5, 0], 5000),
                                             ([130, 0, 257], 387)], ids=str)
def test_buffers_larger_than_the_rows(hip_device, kind, counts, max_rows):
    """The choice of kernels goes by the buffers' rows, the work by the offsets."""
    dev, n, k = hip_device, 200, 528
    m, e = sum(counts), len(counts)
    off = offsets(counts, dev)
    x, xs = row_codes(counts + [max_rows - m], k, kind, 1, dev)
    xs[m:] = float("nan")
    w, ws = rand_codes((e, n, k), kind, 3, dev), rand_scale((e, n), 4, dev, 1e-3)
    b, r = randn((e, n), 5, dev), randn((max_rows + TAIL, n), 6, dev)
    y = poisoned((max_rows + TAIL, n), BF16, dev)
    LAYER["linear", kind](x, xs, w, ws, off, y, bias=b, residual=r, activation="silu")
    h = poisoned((max_rows + TAIL, n // 2 // 8 * 8), BF16, dev)
    wg, wgs = w[:, :2 * h.shape[1]].contiguous(), ws[:, :2 * h.shape[1]].contiguous()
    LAYER["gated", kind](x, xs, wg, wgs, off, h, activation="relu")
    torch.cuda.synchronize()
    E8.check_linear(x, xs, w, ws, b, r, off, kind, "silu", y)
    E8.check_gated(x, xs, wg, wgs, off, kind, "relu", h)
    assert_untouched(y[m:], "y behind the last expert")
    assert_untouched(h[m:], "h behind the last expert")


@pytest.mark.parametrize("counts", [[0, 1, 1], [0, 90, 200]], ids=str)
def test_weight_offsets_past_32_bits(hip_device, counts):
    dev, n, k = hip_device, 20000, 65536
    g = torch.Generator(device=dev).manual_seed(3)
    w = torch.empty((3, 2 * n, k), dtype=torch.int8, device=dev)
    for i in range(3):
        for j in range(0, 2 * n, 10000):
            piece = w[i, j:j + 10000]
            piece.copy_(torch.randint(-127, 128, piece.shape, generator=g, device=dev, dtype=torch.int8))
    m = sum(counts)
    off = offsets(counts, dev)
    x, xs = row_codes(counts, k, "int8", 1, dev)
    ws = rand_scale((3, 2 * n), 4, dev, 1e-4)
    h = poisoned((m + TAIL, n), BF16, dev)
    moe.moe_grouped_gated_gemm_int8(x, xs, w, ws, off, h)
    torch.cuda.synchronize()
    cols = torch.cat([torch.arange(0, 20), torch.arange(n - 20, n)]).to(dev)
    both = torch.cat([cols, cols + n])
    E8.check_gated(x, xs, w[:, both].cpu(), ws[:, both].cpu(), off, "int8", "silu", h[:, cols])


class Block:
    """A gated feed-forward block in 8 bits from tokens to tokens, in buffers of its own."""

    def __init__(self, dev, n, topk, e, hidden, width, kind, seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.kind, self.e, self.topk = kind, e, topk
        self.x = torch.randn((n, hidden), generator=g).to(BF16).to(dev)
        self.ids = torch.rand((n, e), generator=g).argsort(dim=1)[:, :topk].to(torch.int32).contiguous().to(dev)
        self.wts = torch.softmax(torch.randn((n, topk), generator=g), dim=1).to(dev)
        self.w13 = (torch.randn((e, 2 * width, hidden), generator=g) * hidden**-0.5).to(BF16).to(dev)
        self.w2 = (torch.randn((e, hidden, width), generator=g) * width**-0.5).to(BF16).to(dev)
        rows, code = n * topk, CODE[kind]

        def new(*shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.q13, self.s13 = new(e, 2 * width, hidden, dtype=code), new(e, 2 * width, dtype=F32)
        self.q2, self.s2 = new(e, hidden, width, dtype=code), new(e, hidden, dtype=F32)
        for w, q, s in ((self.w13, self.q13, self.s13), (self.w2, self.q2, self.s2)):
            QUANTIZE[kind](w.view(-1, w.shape[2]), q.view(-1, w.shape[2]), s.view(-1))  # weights, once
        self.xq, self.xs = new(rows, hidden, dtype=code), new(rows, dtype=F32)
        self.off = new(e + 1, dtype=torch.int64)
        self.perm, self.inv = new(rows, dtype=torch.int32), new(rows, dtype=torch.int32)
        self.ws = new(max(16, binding.moe_permute_workspace_size(n, topk, e)), dtype=torch.uint8)
        self.h, self.hq, self.hs = new(rows, width, dtype=BF16), new(rows, width, dtype=code), new(rows, dtype=F32)
        self.y, self.out = new(rows, hidden, dtype=BF16), new(n, hidden, dtype=BF16)

    def run(self, stream=None):
        permute = moe.moe_permute_quant_int8 if self.kind == "int8" else moe.moe_permute_quant_fp8
        permute(self.x, self.ids, self.e, self.xq, self.xs, self.off, self.perm, self.inv, self.ws, stream=stream)
        LAYER["gated", self.kind](self.xq, self.xs, self.q13, self.s13, self.off, self.h, stream=stream)
        QUANTIZE[self.kind](self.h, self.hq, self.hs, expert_first_token_offset=self.off, stream=stream)
        LAYER["linear", self.kind](self.hq, self.hs, self.q2, self.s2, self.off, self.y, stream=stream)
        moe.moe_unpermute(self.y, self.wts, self.inv, self.out, stream=stream)

    def outputs(self):
        return [self.xq, self.xs, self.off, self.h, self.hq, self.hs, self.y, self.out]

    def check(self):
        """Every step from what the step before wrote, then the whole against the unquantised block."""
        token = torch.div(self.perm.long(), self.topk, rounding_mode="floor")
        codes, scale = E8.codes_of(self.x[token].cpu(), self.kind)
        assert torch.equal(_bits(self.xq), codes.view(torch.uint8)) and torch.equal(self.xs.cpu(), scale)
        E8.check_gated(self.xq, self.xs, self.q13, self.s13, self.off, self.kind, "silu", self.h)
        codes, scale = E8.codes_of(self.h.cpu(), self.kind)
        assert torch.equal(_bits(self.hq), codes.view(torch.uint8)) and torch.equal(self.hs.cpu(), scale)
        E8.check_linear(self.hq, self.hs, self.q2, self.s2, None, None, self.off, self.kind, "none", self.y)
        z, _ = X.grouped(X.f64(self.x)[token.cpu()], X.f64(self.w13), self.off)
        width = self.h.shape[1]
        h = X.act_value(z[:, :width], "silu") * z[:, width:]
        y, _ = X.grouped(h, X.f64(self.w2), self.off)
        ref = (y[self.inv.long().cpu()].view(*self.wts.shape, -1) * X.f64(self.wts)[..., None]).sum(1)
        # codes are within half a step of their values, 1/254 of the row's largest (int8) or 2^-4 of
        # the value (fp8), evenly: a third of its square in the mean.  A row's largest is taken as ten
        # times its root mean square at most, and the result has six such errors: the tokens' and the
        # first weights' in both projections, those of h and of the second weights.
        off = float((X.f64(self.out) - ref).norm() / ref.norm())
        assert off < 6 * (10 / 254 if self.kind == "int8" else 2.0**-4) / 3**0.5, off


BLOCKS = [(1, 8, 32, 512, 256), (4, 2, 8, 1024, 512), (33, 3, 13, 432, 208), (300, 4, 16, 256, 512)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,topk,e,hidden,width", BLOCKS)
def test_block(hip_device, kind, n, topk, e, hidden, width):
    b = Block(hip_device, n, topk, e, hidden, width, kind)
    b.run()
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("kind", KINDS)
def test_block_on_another_stream(hip_device, kind):
    b = Block(hip_device, 33, 3, 13, 432, 208, kind)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b.run(stream=s)
    s.synchronize()
    b.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [2, 300])
def test_block_captured_and_replayed(hip_device, kind, n):
    """A graph of the whole block on new inputs each time, with eager work between the replays."""
    b = Block(hip_device, n, 4, 16, 256, 512, kind)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for i in range(4):
        other = Block(hip_device, n, 4, 16, 256, 512, kind, seed=i + 1)
        other.run()
        for name in ("x", "ids", "wts", "q13", "s13", "q2", "s2"):
            getattr(b, name).copy_(getattr(other, name))
        for t in b.outputs():
            t.view(torch.uint8).fill_(POISON)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(b.outputs(), other.outputs()):
            assert torch.equal(_bits(got), _bits(want)), i


def test_two_streams_at_once(hip_device):
    blocks = [Block(hip_device, 300, 4, 16, 256, 512, kind, seed=i) for i, kind in enumerate(KINDS)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(blocks, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b in blocks:
        b.check()
