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

import contextlib
import ctypes

from . import binding
from .binding import MOE_OK, MoEError, _check, _dtype_code, _ptr, _require_gpu, _stream

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
        lib.moe_grouped_gated_gemm_bf16.argtypes = [p, p, p, i32, i64, i64, i64, i32, p, p, p]
        lib.moe_grouped_gated_gemm_backward_bf16.argtypes = [p, p, p, p, p, i32, i64, i64, i64, i32, p, p, p, p]
        lib.moe_grouped_linear_bf16.argtypes = [p, p, p, p, p, i32, i64, i64, i64, i32, p, p, p]
        lib.moe_grouped_linear_backward_bf16.argtypes = [p, p, p, p, p, i32, i64, i64, i64, i32, p, p, p, p, p]
        lib.moe_unpermute_backward.argtypes = [p, p, i32, p, p, i64, i64, i32, p, p, p]
        for fn in (lib.moe_grouped_gated_gemm_bf16, lib.moe_grouped_gated_gemm_backward_bf16,
                   lib.moe_grouped_linear_bf16, lib.moe_grouped_linear_backward_bf16, lib.moe_unpermute_backward):
            fn.restype = ctypes.c_int
        _lib = lib
    return lib


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(sorted(ACTIVATIONS)), name))
    return ACTIVATIONS[name]


def _matrix(t, name: str, dims: int):
    if t is None or t.dim() != dims:
        raise ValueError("%s must be a tensor of %d dimensions" % (name, dims))
    return t


def _shaped(t, name: str, shape, device, optional: bool = False) -> None:
    """A bf16 buffer of exactly this shape."""
    import torch

    numel = 1
    for s in shape:
        numel *= s
    _check(t, name, (torch.bfloat16,), numel, device, optional=optional)
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s, got shape %s" % (name, list(shape), tuple(t.shape)))


def _call(name: str, device, stream, tensor, args) -> None:
    """Calls the entry point on the tensors' device, whichever device is current."""
    import torch

    if stream is not None and stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    other = torch.cuda.current_device() != device.index
    with torch.cuda.device(device) if other else contextlib.nullcontext():
        status = getattr(_load(), name)(*args, _stream(stream, tensor))
    if status != MOE_OK:
        raise MoEError(status, name)


def _offsets(off, experts: int, device) -> None:
    import torch

    _check(off, "expert_first_token_offset", (torch.int64,), experts + 1, device)


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
    dev = x.device
    _shaped(x, "x", (rows, k), dev)
    _shaped(w, "w", (experts, 2 * n, k), dev)
    _shaped(h, "h", (rows, n), dev)
    _shaped(gate_up, "gate_up", (rows, 2 * n), dev, optional=True)
    _offsets(expert_first_token_offset, experts, dev)
    _require_gpu(dev)
    _call("moe_grouped_gated_gemm_bf16", dev, stream, x,
          (_ptr(x), _ptr(w), _ptr(expert_first_token_offset), experts, rows, n, k, act, _ptr(gate_up), _ptr(h)))


def moe_grouped_gated_gemm_backward_bf16(d_h, gate_up, x, w, expert_first_token_offset, d_gate_up, d_x=None, d_w=None,
                                         activation: str = "silu", stream=None) -> None:
    """Backward of moe_grouped_gated_gemm_bf16 from the kept ``gate_up``.

    Writes ``d_gate_up`` [max_rows, 2n] and, where given, ``d_x`` [max_rows, k]
    and ``d_w`` [E, 2n, k] (zeros for experts without rows).
    """
    act = _activation(activation)
    experts, n, k = _gate_up_width(w)
    rows = _matrix(d_h, "d_h", 2).shape[0]
    dev = d_h.device
    _shaped(d_h, "d_h", (rows, n), dev)
    _shaped(gate_up, "gate_up", (rows, 2 * n), dev)
    _shaped(x, "x", (rows, k), dev, optional=d_w is None)
    _shaped(w, "w", (experts, 2 * n, k), dev)
    _shaped(d_gate_up, "d_gate_up", (rows, 2 * n), dev)
    _shaped(d_x, "d_x", (rows, k), dev, optional=True)
    _shaped(d_w, "d_w", (experts, 2 * n, k), dev, optional=True)
    _offsets(expert_first_token_offset, experts, dev)
    _require_gpu(dev)
    _call("moe_grouped_gated_gemm_backward_bf16", dev, stream, d_h,
          (_ptr(d_h), _ptr(gate_up), _ptr(x), _ptr(w), _ptr(expert_first_token_offset), experts, rows, n, k, act,
           _ptr(d_gate_up), _ptr(d_x), _ptr(d_w)))


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
    dev = x.device
    _shaped(x, "x", (rows, k), dev)
    _shaped(w, "w", (experts, n, k), dev)
    _shaped(y, "y", (rows, n), dev)
    _shaped(bias, "bias", (experts, n), dev, optional=True)
    _shaped(residual, "residual", (rows, n), dev, optional=True)
    _shaped(pre_activation, "pre_activation", (rows, n), dev, optional=True)
    _offsets(expert_first_token_offset, experts, dev)
    _require_gpu(dev)
    _call("moe_grouped_linear_bf16", dev, stream, x,
          (_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(expert_first_token_offset), experts, rows, n, k, act,
           _ptr(pre_activation), _ptr(y)))


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
    dev = d_y.device
    if act == MOE_ACT_NONE and (pre_activation is not None or d_pre_activation is not None):
        raise ValueError("pre_activation and d_pre_activation go with an activation")
    _shaped(d_y, "d_y", (rows, n), dev)
    _shaped(x, "x", (rows, k), dev, optional=d_w is None)
    _shaped(w, "w", (experts, n, k), dev)
    _shaped(d_x, "d_x", (rows, k), dev, optional=True)
    _shaped(d_w, "d_w", (experts, n, k), dev, optional=True)
    _shaped(d_bias, "d_bias", (experts, n), dev, optional=True)
    _shaped(pre_activation, "pre_activation", (rows, n), dev, optional=act == MOE_ACT_NONE)
    _shaped(d_pre_activation, "d_pre_activation", (rows, n), dev, optional=act == MOE_ACT_NONE)
    _offsets(expert_first_token_offset, experts, dev)
    _require_gpu(dev)
    _call("moe_grouped_linear_backward_bf16", dev, stream, d_y,
          (_ptr(d_y), _ptr(pre_activation), _ptr(x), _ptr(w), _ptr(expert_first_token_offset), experts, rows, n, k,
           act, _ptr(d_pre_activation), _ptr(d_x), _ptr(d_w), _ptr(d_bias)))


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
    same = (d_output.dtype,)
    _check(d_output, "d_output", same, n * h, dev)
    _check(expanded_output, "expanded_output", same, n * topk * h, dev, optional=d_topk_weights is None)
    _check(topk_weights, "topk_weights", (torch.float32,), n * topk, dev)
    _check(inv_permuted_idx, "inv_permuted_idx", (torch.int32,), n * topk, dev)
    _check(d_expanded_output, "d_expanded_output", same, n * topk * h, dev, optional=True)
    _check(d_topk_weights, "d_topk_weights", (torch.float32,), n * topk, dev, optional=True)
    _require_gpu(dev)
    _call("moe_unpermute_backward", dev, stream, d_output,
          (_ptr(d_output), _ptr(expanded_output), _dtype_code(d_output), _ptr(topk_weights), _ptr(inv_permuted_idx),
           n, h, topk, _ptr(d_expanded_output), _ptr(d_topk_weights)))
