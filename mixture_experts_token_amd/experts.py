"""Python binding of the expert layers of libmoe_permute.so (argument marshalling only).

The entry points carry the C names of ``include/moe_experts.h``:
``moe_grouped_gated_gemm_bf16`` and ``moe_grouped_linear_bf16`` run between the
permute and the unpermute, the ``*_backward*`` entry points are their
gradients and the unpermute's.  As in ``binding``, tensors become raw device
pointers, outputs are written in place into the caller's buffers, the work
goes to ``stream`` (default: torch's current stream on the tensors' device),
and a non-OK status raises ``MoEError``.
"""

from __future__ import annotations

import ctypes

from . import binding
from .binding import MOE_OK, MoEError, _dtype_code, _require_gpu

MOE_ACT_NONE = 0
MOE_ACT_RELU = 1
MOE_ACT_SILU = 2
MOE_ACT_GELU_TANH = 3

ACTIVATIONS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU, "gelu_tanh": MOE_ACT_GELU_TANH}

_lib = None


def _load() -> ctypes.CDLL:
    """The library with the expert layers' signatures set."""
    global _lib
    lib = binding.load_library()
    if _lib is not lib:
        p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        _set_signatures(lib, {
            "moe_grouped_gated_gemm_bf16": [p, p, p, i32, i64, i64, i64, i32, p, p, p],
            "moe_grouped_gated_gemm_backward_bf16": [p, p, p, p, p, i32, i64, i64, i64, i32, p, p, p, p],
            "moe_grouped_linear_bf16": [p, p, p, p, p, i32, i64, i64, i64, i32, p, p, p],
            "moe_grouped_linear_backward_bf16": [p, p, p, p, p, i32, i64, i64, i64, i32, p, p, p, p, p],
            "moe_unpermute_backward": [p, p, i32, p, p, i64, i64, i32, p, p, p],
        })
        _lib = lib
    return lib


def _set_signatures(lib, signatures) -> None:
    for name, argtypes in signatures.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = argtypes, ctypes.c_int


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(sorted(ACTIVATIONS)), name))
    return ACTIVATIONS[name]


def _matrix(t, name: str, dims: int):
    if t is None or t.dim() != dims:
        raise ValueError("%s must be a tensor of %d dimensions" % (name, dims))
    return t


def _buffer(t, name: str, dtypes, shape, device, optional: bool = False):
    """Raw device address of a contiguous buffer of exactly this shape (None stays None where it may).

    One pass over a buffer instead of a check and a conversion: at single
    tokens the call is as short as its kernel.
    """
    if t is None:
        if optional:
            return None
        raise ValueError("%s is required" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got shape %s" % (name, list(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.device != device:
        raise TypeError("%s is on %s, expected %s (every buffer of the call on one GPU)" % (name, t.device, device))
    return t.data_ptr()


def _call(name: str, device, stream, args, load=_load) -> None:
    """Calls the entry point on the tensors' device, whichever device is current."""
    import torch

    _require_gpu(device)
    if stream is not None and stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    handle = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)
    if torch._C._cuda_getDevice() == device.index:
        status = getattr(load(), name)(*args, handle)
    else:
        with torch.cuda.device(device):
            status = getattr(load(), name)(*args, handle)
    if status != MOE_OK:
        raise MoEError(status, name)


def _bf16():
    import torch

    return (torch.bfloat16,)


def _offsets(off, experts: int, device):
    import torch

    return _buffer(off, "expert_first_token_offset", (torch.int64,), (experts + 1,), device)


def _gate_up_width(w):
    experts, m, k = _matrix(w, "w", 3).shape
    if m % 2:
        raise ValueError("w must be [E, 2 n, k]: the gate rows, then the up rows; got %d rows" % m)
    return experts, m // 2, k


def moe_grouped_gated_gemm_bf16(x, w, expert_first_token_offset, h, gate_up=None, activation: str = "silu",
                                stream=None) -> None:
    """h[j] = act(x[j] @ w[e, :n]^T) * (x[j] @ w[e, n:]^T) for the permuted rows j of expert e.

    ``x`` bfloat16 [max_rows, k]; ``w`` bfloat16 [E, 2n, k], the gate rows then
    the up rows; offsets int64 [E + 1] on the device; ``h`` bfloat16
    [max_rows, n]; ``gate_up`` bfloat16 [max_rows, 2n] or None receives both
    projections, which the backward takes.
    """
    act = _activation(activation)
    experts, n, k = _gate_up_width(w)
    rows = _matrix(x, "x", 2).shape[0]
    dev, bf16 = x.device, _bf16()
    args = (_buffer(x, "x", bf16, (rows, k), dev), _buffer(w, "w", bf16, (experts, 2 * n, k), dev),
            _offsets(expert_first_token_offset, experts, dev), experts, rows, n, k, act,
            _buffer(gate_up, "gate_up", bf16, (rows, 2 * n), dev, optional=True), _buffer(h, "h", bf16, (rows, n), dev))
    _call("moe_grouped_gated_gemm_bf16", dev, stream, args)


def moe_grouped_gated_gemm_backward_bf16(d_h, gate_up, x, w, expert_first_token_offset, d_gate_up, d_x=None, d_w=None,
                                         activation: str = "silu", stream=None) -> None:
    """Backward of moe_grouped_gated_gemm_bf16 from the kept ``gate_up``.

    Writes ``d_gate_up`` [max_rows, 2n] and, where given, ``d_x`` [max_rows, k]
    and ``d_w`` [E, 2n, k] (zeros for experts without rows).
    """
    act = _activation(activation)
    experts, n, k = _gate_up_width(w)
    rows = _matrix(d_h, "d_h", 2).shape[0]
    dev, bf16 = d_h.device, _bf16()
    args = (_buffer(d_h, "d_h", bf16, (rows, n), dev), _buffer(gate_up, "gate_up", bf16, (rows, 2 * n), dev),
            _buffer(x, "x", bf16, (rows, k), dev, optional=d_w is None),
            _buffer(w, "w", bf16, (experts, 2 * n, k), dev), _offsets(expert_first_token_offset, experts, dev),
            experts, rows, n, k, act, _buffer(d_gate_up, "d_gate_up", bf16, (rows, 2 * n), dev),
            _buffer(d_x, "d_x", bf16, (rows, k), dev, optional=True),
            _buffer(d_w, "d_w", bf16, (experts, 2 * n, k), dev, optional=True))
    _call("moe_grouped_gated_gemm_backward_bf16", dev, stream, args)


def moe_grouped_linear_bf16(x, w, expert_first_token_offset, y, bias=None, residual=None, pre_activation=None,
                            activation: str = "none", stream=None) -> None:
    """y[j] = act(x[j] @ w[e]^T + bias[e]) + residual[j] for the permuted rows j of expert e.

    ``x`` bfloat16 [max_rows, k]; ``w`` bfloat16 [E, n, k]; ``bias`` [E, n];
    ``residual`` and ``y`` [max_rows, n]; ``pre_activation`` [max_rows, n] or
    None receives the argument of the activation, which the backward takes.
    """
    act = _activation(activation)
    experts, n, k = _matrix(w, "w", 3).shape
    rows = _matrix(x, "x", 2).shape[0]
    dev, bf16 = x.device, _bf16()
    args = (_buffer(x, "x", bf16, (rows, k), dev), _buffer(w, "w", bf16, (experts, n, k), dev),
            _buffer(bias, "bias", bf16, (experts, n), dev, optional=True),
            _buffer(residual, "residual", bf16, (rows, n), dev, optional=True),
            _offsets(expert_first_token_offset, experts, dev), experts, rows, n, k, act,
            _buffer(pre_activation, "pre_activation", bf16, (rows, n), dev, optional=True),
            _buffer(y, "y", bf16, (rows, n), dev))
    _call("moe_grouped_linear_bf16", dev, stream, args)


def moe_grouped_linear_backward_bf16(d_y, x, w, expert_first_token_offset, d_x=None, d_w=None, d_bias=None,
                                     pre_activation=None, d_pre_activation=None, activation: str = "none",
                                     stream=None) -> None:
    """Backward of moe_grouped_linear_bf16 (the residual's gradient is ``d_y``).

    Writes what is given of ``d_x`` [max_rows, k], ``d_w`` [E, n, k] and
    ``d_bias`` [E, n] (zeros for experts without rows).  With an activation,
    ``pre_activation`` is the tensor the forward wrote and
    ``d_pre_activation`` [max_rows, n] receives its gradient; without one
    both are None.
    """
    act = _activation(activation)
    experts, n, k = _matrix(w, "w", 3).shape
    rows = _matrix(d_y, "d_y", 2).shape[0]
    dev, bf16, plain = d_y.device, _bf16(), act == MOE_ACT_NONE
    if plain and (pre_activation is not None or d_pre_activation is not None):
        raise ValueError("pre_activation and d_pre_activation go with an activation")
    args = (_buffer(d_y, "d_y", bf16, (rows, n), dev),
            _buffer(pre_activation, "pre_activation", bf16, (rows, n), dev, optional=plain),
            _buffer(x, "x", bf16, (rows, k), dev, optional=d_w is None), _buffer(w, "w", bf16, (experts, n, k), dev),
            _offsets(expert_first_token_offset, experts, dev), experts, rows, n, k, act,
            _buffer(d_pre_activation, "d_pre_activation", bf16, (rows, n), dev, optional=plain),
            _buffer(d_x, "d_x", bf16, (rows, k), dev, optional=True),
            _buffer(d_w, "d_w", bf16, (experts, n, k), dev, optional=True),
            _buffer(d_bias, "d_bias", bf16, (experts, n), dev, optional=True))
    _call("moe_grouped_linear_backward_bf16", dev, stream, args)


def moe_unpermute_backward(d_output, expanded_output, topk_weights, inv_permuted_idx, d_expanded_output=None,
                           d_topk_weights=None, stream=None) -> None:
    """Backward of moe_unpermute / moe_unpermute_local (see the C header).

    ``d_output`` [N, H] float32 or bfloat16; ``expanded_output`` and
    ``d_expanded_output`` [N*topk, H] of the same type; ``topk_weights`` and
    ``d_topk_weights`` float32 [N, topk]; ``inv_permuted_idx`` int32 [N*topk].
    ``expanded_output`` is only needed for ``d_topk_weights``.
    """
    import torch

    n, topk = _matrix(topk_weights, "topk_weights", 2).shape
    h = _matrix(d_output, "d_output", 2).shape[1]
    dev = d_output.device
    if d_output.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("d_output must be float32 or bfloat16, got %s" % d_output.dtype)
    same, f32, slots = (d_output.dtype,), (torch.float32,), n * topk
    args = (_buffer(d_output, "d_output", same, (n, h), dev),
            _buffer(expanded_output, "expanded_output", same, (slots, h), dev, optional=d_topk_weights is None),
            _dtype_code(d_output), _buffer(topk_weights, "topk_weights", f32, (n, topk), dev),
            _buffer(inv_permuted_idx, "inv_permuted_idx", (torch.int32,), (slots,), dev), n, h, topk,
            _buffer(d_expanded_output, "d_expanded_output", same, (slots, h), dev, optional=True),
            _buffer(d_topk_weights, "d_topk_weights", f32, (n, topk), dev, optional=True))
    _call("moe_unpermute_backward", dev, stream, args)
