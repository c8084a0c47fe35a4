"""GPU parity of the forms and calls of the expert layers beside tests/test_experts_gpu.py: every activation in
the backward, buffers far larger than the rows in them (the state of an expert-parallel rank, where
max_rows is N * topk and a fraction of it is local), and a rank's whole block.

References and bounds as there.
"""

import numpy as np
import pytest
import torch

import _experts as X
import workloads as W
from _parity import gpu_permute_local, poisoned
from mixture_experts_token_amd import binding
import mixture_experts_token_amd as moe
from test_experts_gpu import BF16, SHAPES, _id, _say, assert_untouched, offsets, randn, rows_of

pytestmark = pytest.mark.gpu

# one row; ragged; few rows (streamed, and the weight gradient of few rows); large tiles
SOME = [SHAPES[0], SHAPES[3], SHAPES[7], SHAPES[16], SHAPES[20]]


def buffer_rows(counts, capacity, cols, seed, dev):
    """[capacity, cols]: the experts' rows, then NaN."""
    t = torch.full((capacity, cols), float("nan"), dtype=BF16, device=dev)
    t[:sum(counts)] = randn((sum(counts), cols), seed, dev)
    return t


@pytest.mark.parametrize("shape", SOME, ids=_id)
@pytest.mark.parametrize("act", ["relu", "none"])
def test_gated_backward(hip_device, shape, act):
    counts, n, k = shape
    dev, m, e = hip_device, sum(counts), len(counts)
    _say("gated backward %s act=%s" % (_id(shape), act))
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w = randn((e, 2 * n, k), 2, dev, k**-0.5)
    gate_up, d_h = rows_of(counts, 2 * n, 7, dev), rows_of(counts, n, 8, dev)
    d_gu, d_x = poisoned(tuple(gate_up.shape), BF16, dev), poisoned(tuple(x.shape), BF16, dev)
    d_w = poisoned((e, 2 * n, k), BF16, dev)
    moe.moe_grouped_gated_gemm_backward_bf16(d_h, gate_up, x, w, off, d_gu, d_x=d_x, d_w=d_w, activation=act)
    torch.cuda.synchronize()
    X.check_gated_slopes(d_h, gate_up, off, act, d_gu)
    X.check_products(d_gu, x, w, off, d_x, d_w)
    assert_untouched(d_gu[m:], "d_gate_up behind the last expert")
    assert_untouched(d_x[m:], "d_x behind the last expert")


@pytest.mark.parametrize("shape", SOME, ids=_id)
def test_linear_backward_gelu(hip_device, shape):
    counts, n, k = shape
    dev, m, e = hip_device, sum(counts), len(counts)
    _say("linear backward %s act=gelu_tanh" % _id(shape))
    off, x = offsets(counts, dev), rows_of(counts, k, 1, dev)
    w = randn((e, n, k), 2, dev, k**-0.5)
    d_y, pre = rows_of(counts, n, 9, dev), rows_of(counts, n, 10, dev)
    d_z, d_x = poisoned(tuple(pre.shape), BF16, dev), poisoned(tuple(x.shape), BF16, dev)
    d_w, d_b = poisoned((e, n, k), BF16, dev), poisoned((e, n), BF16, dev)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=d_x, d_w=d_w, d_bias=d_b, pre_activation=pre,
                                         d_pre_activation=d_z, activation="gelu_tanh")
    torch.cuda.synchronize()
    X.check_slopes(d_y, pre, off, "gelu_tanh", d_z)
    X.check_products(d_z, x, w, off, d_x, d_w, d_b)
    assert_untouched(d_z[m:], "d_pre_activation behind the last expert")
    assert_untouched(d_x[m:], "d_x behind the last expert")


# (rows of each expert, rows of the buffers, n, k): the variants are chosen by the buffers' rows
CAPACITY = [
    ([1, 0, 2, 1], 64, 136, 1096),
    ([5, 0, 3, 9, 0, 0, 1, 2], 4096, 264, 520),
    ([0] * 8, 4096, 264, 520),
    ([300, 0, 17, 128, 100], 8192, 2056, 1288),        # large tiles, remainders perhaps apart
    ([1024, 1025, 1134, 1023], 8192, 3960, 1032),      # and apart in earnest
    ([1] + [0] * 62 + [70], 128, 520, 4104),           # a row or two per expert at most, all of them one expert's
    ([0, 33, 0, 0, 31, 0, 0, 0] * 4, 8192, 128, 2312),
]


@pytest.mark.parametrize("case", CAPACITY, ids=lambda c: "%dof%d-%dx%d" % (sum(c[0]), c[1], c[2], c[3]))
def test_buffers_larger_than_the_rows(hip_device, case):
    counts, capacity, n, k = case
    dev, m, e = hip_device, sum(counts), len(counts)
    _say("%d rows in buffers of %d, %d x %d" % (m, capacity, n, k))
    off, x = offsets(counts, dev), buffer_rows(counts, capacity, k, 1, dev)
    w, wg = randn((e, n, k), 2, dev, k**-0.5), randn((e, 2 * n, k), 3, dev, k**-0.5)
    b, res = randn((e, n), 4, dev), buffer_rows(counts, capacity, n, 5, dev)
    d_y, gate_up = buffer_rows(counts, capacity, n, 6, dev), buffer_rows(counts, capacity, 2 * n, 7, dev)
    rows = {}

    def out(name, cols):
        rows[name] = poisoned((capacity, cols), BF16, dev)
        return rows[name]

    d_w, d_wg, d_b = (poisoned(s, BF16, dev) for s in ((e, n, k), (e, 2 * n, k), (e, n)))
    moe.moe_grouped_gated_gemm_bf16(x, wg, off, out("h", n), gate_up=out("keep", 2 * n))
    moe.moe_grouped_linear_bf16(x, w, off, out("y", n), bias=b, residual=res, pre_activation=out("pre", n),
                                activation="silu")
    moe.moe_grouped_gated_gemm_backward_bf16(d_y, gate_up, x, wg, off, out("d_gate_up", 2 * n),
                                             d_x=out("d_xg", k), d_w=d_wg)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=out("d_x", k), d_w=d_w, d_bias=d_b)
    moe.moe_grouped_linear_backward_bf16(d_y, x, w, off, d_x=out("d_x alone", k))
    torch.cuda.synchronize()
    X.check_gated(x[:m], wg, off, "silu", rows["h"], rows["keep"])
    X.check_linear(x[:m], w, b, res, off, "silu", rows["y"], rows["pre"])
    X.check_gated_slopes(d_y, gate_up, off, "silu", rows["d_gate_up"])
    X.check_products(rows["d_gate_up"], x[:m], wg, off, rows["d_xg"], d_wg)
    X.check_products(d_y, x[:m], w, off, rows["d_x"], d_w, d_b)
    X.check_products(d_y, x[:m], w, off, rows["d_x alone"], None)
    for name, t in rows.items():
        assert_untouched(t[m:], name + " behind the last expert")


def test_layers_on_scratch_buffers(hip_device):
    """MoEPermuteScratch made for more tokens than a call has: its views go to the layers as they are."""
    dev, n, topk, e, hidden, width = hip_device, 21, 2, 5, 136, 72
    scratch = moe.MoEPermuteScratch(64, topk, e, dev, hidden_size=hidden, hidden_dtype=BF16)
    x, wts = randn((n, hidden), 1, dev), torch.full((n, topk), 0.5, device=dev)
    ids = torch.stack([torch.arange(n) % e, (torch.arange(n) + 2) % e], 1).int().to(dev)
    res = scratch.permute(x, ids)
    xp, off, inv = res["permuted_hidden_states"], res["expert_first_token_offset"], res["inv_permuted_idx"]
    w13, w2 = randn((e, 2 * width, hidden), 2, dev, hidden**-0.5), randn((e, hidden, width), 3, dev, width**-0.5)
    rows = n * topk
    h, y, out = poisoned((rows, width), BF16, dev), poisoned((rows, hidden), BF16, dev), poisoned((n, hidden), BF16, dev)
    moe.moe_grouped_gated_gemm_bf16(xp, w13, off, h)
    moe.moe_grouped_linear_bf16(h, w2, off, y)
    moe.moe_unpermute(y, wts, inv, out)
    d_y, d_w2 = poisoned((rows, hidden), BF16, dev), poisoned((e, hidden, width), BF16, dev)
    moe.moe_unpermute_backward(out, y, wts, inv, d_expanded_output=d_y)
    moe.moe_grouped_linear_backward_bf16(d_y, h, w2, off, d_w=d_w2)
    torch.cuda.synchronize()
    X.check_gated(xp, w13, off, "silu", h, None)
    X.check_linear(h, w2, None, None, off, "none", y, None)
    X.check_products(d_y, h, w2, off, None, d_w2)
    slots = X.f64(y)[inv.long().cpu()].view(n, topk, hidden)
    ref = 0.5 * slots.sum(1)
    X.assert_within(out, ref, X.HALF * ref.abs() + X.accumulate(topk) * slots.abs().sum(1), "out")


def test_empty_batches(hip_device):
    """Tensors of no rows have no address; every call takes them."""
    dev, n, k = hip_device, 48, 64
    off = offsets([0, 0], dev)
    w, wg = randn((2, n, k), 1, dev), randn((2, 2 * n, k), 2, dev)

    def rows(cols, dtype=BF16):
        return torch.empty(0, cols, dtype=dtype, device=dev)

    moe.moe_grouped_gated_gemm_bf16(rows(k), wg, off, rows(n), gate_up=rows(2 * n))
    moe.moe_grouped_linear_bf16(rows(k), w, off, rows(n), residual=rows(n), pre_activation=rows(n), activation="silu")
    moe.moe_grouped_linear_backward_bf16(rows(n), None, w, off, d_x=rows(k))
    moe.moe_grouped_gated_gemm_backward_bf16(rows(n), rows(2 * n), None, wg, off, rows(2 * n), d_x=rows(k))
    d_wg, d_b = poisoned((2, 2 * n, k), BF16, dev), poisoned((2, n), BF16, dev)
    moe.moe_grouped_gated_gemm_backward_bf16(rows(n), rows(2 * n), rows(k), wg, off, rows(2 * n), d_x=rows(k), d_w=d_wg)
    moe.moe_grouped_linear_backward_bf16(rows(n), None, w, off, d_bias=d_b, pre_activation=rows(n),
                                         d_pre_activation=rows(n), activation="silu")
    moe.moe_unpermute_backward(rows(k), rows(k), rows(2, torch.float32),
                               torch.empty(0, dtype=torch.int32, device=dev), d_expanded_output=rows(k),
                               d_topk_weights=rows(2, torch.float32))
    torch.cuda.synchronize()
    assert not d_wg.any() and not d_b.any()


@pytest.mark.parametrize("rank", [0, 3])
def test_block_of_one_rank(hip_device, rank):
    """moe_permute_local, both layers, moe_unpermute_local and back, as one of four expert-parallel ranks."""
    dev, n, topk, experts, hidden, width = hip_device, 130, 4, 16, 264, 104
    _say("block of rank %d of 4" % rank)
    rng = np.random.default_rng(rank)
    ids = torch.from_numpy(np.argsort(rng.random((n, experts)), axis=1)[:, :topk].astype(np.int32)).to(dev)
    emap, e = W.expert_map_for(experts, 4, rank, "contiguous")
    x, d_out = randn((n, hidden), 1, dev), randn((n, hidden), 2, dev)
    wts = torch.softmax(randn((n, topk), 3, dev, dtype=torch.float32), 1)
    w13, w2 = randn((e, 2 * width, hidden), 4, dev, hidden**-0.5), randn((e, hidden, width), 5, dev, width**-0.5)
    idx = gpu_permute_local(x, ids, experts, emap, e)
    xp, off, inv = idx["permuted_hidden_states"], idx["expert_first_token_offset"], idx["inv_permuted_idx"]
    rows = n * topk
    t = {name: poisoned(s, BF16, dev) for name, s in dict(
        h=(rows, width), gate_up=(rows, 2 * width), y=(rows, hidden), out=(n, hidden), d_y=(rows, hidden),
        d_h=(rows, width), d_w2=(e, hidden, width), d_gate_up=(rows, 2 * width), d_xp=(rows, hidden),
        d_w13=(e, 2 * width, hidden), d_x=(n, hidden)).items()}
    d_wts = poisoned((n, topk), torch.float32, dev)
    moe.moe_grouped_gated_gemm_bf16(xp, w13, off, t["h"], gate_up=t["gate_up"])
    moe.moe_grouped_linear_bf16(t["h"], w2, off, t["y"])
    binding.moe_unpermute_local(t["y"], wts, inv, t["out"])
    moe.moe_unpermute_backward(d_out, t["y"], wts, inv, d_expanded_output=t["d_y"], d_topk_weights=d_wts)
    moe.moe_grouped_linear_backward_bf16(t["d_y"], t["h"], w2, off, d_x=t["d_h"], d_w=t["d_w2"])
    moe.moe_grouped_gated_gemm_backward_bf16(t["d_h"], t["gate_up"], xp, w13, off, t["d_gate_up"], d_x=t["d_xp"],
                                             d_w=t["d_w13"])
    binding.moe_unpermute_local(t["d_xp"], torch.ones_like(wts), inv, t["d_x"])
    torch.cuda.synchronize()
    live = int(off[-1])
    assert 0 < live < rows // 2
    X.check_gated(xp[:live], w13, off, "silu", t["h"], t["gate_up"])
    X.check_linear(t["h"][:live], w2, None, None, off, "none", t["y"], None)
    ref_rows, ref_w, mag = X.unpermute_backward(d_out, t["y"], wts, inv.cpu())
    assert sorted(ref_rows) == list(range(live))
    ref = torch.stack([ref_rows[j] for j in range(live)])
    X.assert_within(t["d_y"][:live], ref, (X.HALF + 2.0**-24) * ref.abs(), "d_y")
    X.assert_within(d_wts, ref_w, X.accumulate(hidden) * mag, "d_topk_weights")
    X.check_products(t["d_y"], t["h"][:live], w2, off, t["d_h"], t["d_w2"])
    X.check_gated_slopes(t["d_h"], t["gate_up"], off, "silu", t["d_gate_up"])
    X.check_products(t["d_gate_up"], xp[:live], w13, off, t["d_xp"], t["d_w13"])
    for name in ("h", "gate_up", "y", "d_y", "d_h", "d_gate_up", "d_xp"):
        assert_untouched(t[name][live:], name + " behind the last local row")
    here = inv.cpu() >= 0
    slots = torch.where(here, inv.cpu(), torch.zeros_like(inv.cpu())).long()
    for got, per, weight in (("out", "y", X.f64(wts).view(-1)), ("d_x", "d_xp", torch.ones(rows, dtype=torch.float64))):
        each = X.f64(t[per])[slots] * weight[:, None]
        each[~here] = 0.0
        each = each.view(n, topk, hidden)
        ref = each.sum(1)
        X.assert_within(t[got], ref, X.HALF * ref.abs() + X.accumulate(topk) * each.abs().sum(1), got)
