"""Python binding of the 8-bit expert path of libmoe_permute.so (argument marshalling only).

The entry points carry the C names of ``include/moe_experts_8bit.h``: the
permute that quantises to int8, the row quantisers between an expert's two
layers, and the layers on int8 or fp8 E4M3FN codes with a scale for each row
and output channel.  As in ``experts``, tensors become raw device pointers,
outputs are written in place into the caller's buffers, the work goes to
``stream`` (default: torch's current stream on the tensors' device), and a
non-OK status raises ``MoEError``.

int8 codes are ``torch.int8``, fp8 codes ``torch.float8_e4m3fn`` or
``torch.uint8``; a scale may be [rows] or [rows, 1].
"""

from __future__ import annotations

import ctypes

from . import binding
from .binding import MOE_DTYPE_INT32, MOE_DTYPE_INT64, _dtype_code
from .experts import _activation, _bf16, _buffer, _call, _matrix, _offsets, _set_signatures

_lib = None


def _load() -> ctypes.CDLL:
    """The library with the 8-bit path's signatures set."""
    global _lib
    lib = binding.load_library()
    if _lib is not lib:
        p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        quantize = [p, i32, p, i32, i64, i64, p, p, p]
        gated = [p, p, p, p, p, i32, i64, i64, i64, i32, p, p]
        linear = [p, p, p, p, p, p, p, i32, i64, i64, i64, i32, p, p]
        _set_signatures(lib, {
            "moe_permute_quant_int8": [p, i32, p, i32, i64, i64, i32, i32, p, i32, p, p, p, p, p, p, sz, p],
            "moe_quantize_rows_int8": quantize, "moe_quantize_rows_fp8": quantize,
            "moe_grouped_gated_gemm_int8": gated, "moe_grouped_gated_gemm_fp8": gated,
            "moe_grouped_linear_int8": linear, "moe_grouped_linear_fp8": linear,
        })
        _lib = lib
    return lib


_TYPES = None


def _types():
    """(int8 codes, fp8 codes, quantisers' inputs, scales)"""
    global _TYPES
    if _TYPES is None:
        import torch

        _TYPES = ((torch.int8,), (torch.float8_e4m3fn, torch.uint8), (torch.bfloat16, torch.float32),
                  (torch.float32,))
    return _TYPES


def _row_scale(t, name: str, rows: int, device):
    shape = (rows, 1) if t is not None and t.dim() == 2 else (rows,)
    return _buffer(t, name, _types()[3], shape, device)


def moe_permute_quant_int8(hidden_states, topk_ids, num_experts: int, permuted_codes, permuted_scale,
                           expert_first_token_offset, permuted_idx, inv_permuted_idx, workspace=None,
                           expert_map=None, num_local_experts: int = 0, stream=None) -> None:
    """moe_permute_quant_fp8 with int8 codes and a scale for each token.

    ``hidden_states`` bfloat16 or float32 [N, H]; ``topk_ids`` int32 or int64
    [N, topk]; ``permuted_codes`` int8 [N*topk, H]; ``permuted_scale`` float32
    [N*topk]; with ``expert_map`` (int32 [num_experts]) the local-expert
    permute over ``num_local_experts``.
    """
    import torch

    int8, _, inputs, _ = _types()
    num_experts = int(num_experts)
    n, topk = _matrix(topk_ids, "topk_ids", 2).shape
    h = _matrix(hidden_states, "hidden_states", 2).shape[1]
    dev, rows, i32 = topk_ids.device, n * topk, (torch.int32,)
    if expert_map is None:
        num_local_experts = 0
    buckets = int(num_local_experts) if expert_map is not None else num_experts
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.device != dev:
            raise TypeError("workspace is on %s, expected %s" % (workspace.device, dev))
    args = (_buffer(hidden_states, "hidden_states", inputs, (n, h), dev), _dtype_code(hidden_states),
            _buffer(topk_ids, "topk_ids", (torch.int32, torch.int64), (n, topk), dev),
            MOE_DTYPE_INT64 if topk_ids.dtype == torch.int64 else MOE_DTYPE_INT32, n, h, topk, num_experts,
            _buffer(expert_map, "expert_map", i32, (num_experts,), dev, optional=True), int(num_local_experts),
            _buffer(permuted_codes, "permuted_codes", int8, (rows, h), dev),
            _row_scale(permuted_scale, "permuted_scale", rows, dev),
            _offsets(expert_first_token_offset, buckets, dev),
            _buffer(permuted_idx, "permuted_idx", i32, (rows,), dev),
            _buffer(inv_permuted_idx, "inv_permuted_idx", i32, (rows,), dev),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size())
    _call("moe_permute_quant_int8", dev, stream, args, _load)


def _quantize_rows(name: str, code_types, x, codes, scale, off, stream) -> None:
    rows, n = _matrix(x, "x", 2).shape
    dev = x.device
    experts, offsets = 0, None
    if off is not None:
        experts = off.numel() - 1
        offsets = _offsets(off, experts, dev)
    args = (_buffer(x, "x", _types()[2], (rows, n), dev), _dtype_code(x), offsets, experts, rows, n,
            _buffer(codes, "codes", code_types, (rows, n), dev), _row_scale(scale, "scale", rows, dev))
    _call(name, dev, stream, args, _load)


def moe_quantize_rows_int8(x, codes, scale, expert_first_token_offset=None, stream=None) -> None:
    """int8 codes and a scale for each row of ``x`` (bfloat16 or float32 [max_rows, n]).

    ``codes`` int8 [max_rows, n]; ``scale`` float32 [max_rows].  With the
    offsets (int64 [E + 1]) only the experts' rows are read and written.
    """
    _quantize_rows("moe_quantize_rows_int8", _types()[0], x, codes, scale, expert_first_token_offset, stream)


def moe_quantize_rows_fp8(x, codes, scale, expert_first_token_offset=None, stream=None) -> None:
    """moe_quantize_rows_int8 with fp8 E4M3FN codes."""
    _quantize_rows("moe_quantize_rows_fp8", _types()[1], x, codes, scale, expert_first_token_offset, stream)


def _gated(name: str, codes, x, x_scale, w, w_scale, off, h, activation, stream) -> None:
    act = _activation(activation)
    experts, m, k = _matrix(w, "w", 3).shape
    if m % 2:
        raise ValueError("w must be [E, 2 n, k]: the gate rows, then the up rows; got %d rows" % m)
    rows = _matrix(x, "x", 2).shape[0]
    dev, n = x.device, m // 2
    args = (_buffer(x, "x", codes, (rows, k), dev), _row_scale(x_scale, "x_scale", rows, dev),
            _buffer(w, "w", codes, (experts, m, k), dev), _buffer(w_scale, "w_scale", _types()[3], (experts, m), dev),
            _offsets(off, experts, dev), experts, rows, n, k, act, _buffer(h, "h", _bf16(), (rows, n), dev))
    _call(name, dev, stream, args, _load)


def moe_grouped_gated_gemm_int8(x, x_scale, w, w_scale, expert_first_token_offset, h, activation: str = "silu",
                                stream=None) -> None:
    """h[j] = act(g[j]) * u[j] for the permuted rows j of expert e, g and u the two
    projections x[j] @ w[e]^T of codes, times w_scale[e] and x_scale[j].

    ``x`` int8 [max_rows, k]; ``x_scale`` float32 [max_rows]; ``w`` int8
    [E, 2n, k], the gate rows then the up rows; ``w_scale`` float32 [E, 2n];
    offsets int64 [E + 1]; ``h`` bfloat16 [max_rows, n].
    """
    _gated("moe_grouped_gated_gemm_int8", _types()[0], x, x_scale, w, w_scale, expert_first_token_offset, h,
           activation, stream)


def moe_grouped_gated_gemm_fp8(x, x_scale, w, w_scale, expert_first_token_offset, h, activation: str = "silu",
                               stream=None) -> None:
    """moe_grouped_gated_gemm_int8 on fp8 E4M3FN codes."""
    _gated("moe_grouped_gated_gemm_fp8", _types()[1], x, x_scale, w, w_scale, expert_first_token_offset, h,
           activation, stream)


def _linear(name: str, codes, x, x_scale, w, w_scale, off, y, bias, residual, activation, stream) -> None:
    act = _activation(activation)
    experts, n, k = _matrix(w, "w", 3).shape
    rows = _matrix(x, "x", 2).shape[0]
    dev, bf16 = x.device, _bf16()
    args = (_buffer(x, "x", codes, (rows, k), dev), _row_scale(x_scale, "x_scale", rows, dev),
            _buffer(w, "w", codes, (experts, n, k), dev), _buffer(w_scale, "w_scale", _types()[3], (experts, n), dev),
            _buffer(bias, "bias", bf16, (experts, n), dev, optional=True),
            _buffer(residual, "residual", bf16, (rows, n), dev, optional=True),
            _offsets(off, experts, dev), experts, rows, n, k, act, _buffer(y, "y", bf16, (rows, n), dev))
    _call(name, dev, stream, args, _load)


def moe_grouped_linear_int8(x, x_scale, w, w_scale, expert_first_token_offset, y, bias=None, residual=None,
                            activation: str = "none", stream=None) -> None:
    """y[j] = act((x[j] @ w[e]^T) * w_scale[e] * x_scale[j] + bias[e]) + residual[j].

    ``x`` int8 [max_rows, k]; ``x_scale`` float32 [max_rows]; ``w`` int8
    [E, n, k]; ``w_scale`` float32 [E, n]; ``bias`` bfloat16 [E, n];
    ``residual`` and ``y`` bfloat16 [max_rows, n].
    """
    _linear("moe_grouped_linear_int8", _types()[0], x, x_scale, w, w_scale, expert_first_token_offset, y, bias,
            residual, activation, stream)


def moe_grouped_linear_fp8(x, x_scale, w, w_scale, expert_first_token_offset, y, bias=None, residual=None,
                           activation: str = "none", stream=None) -> None:
    """moe_grouped_linear_int8 on fp8 E4M3FN codes."""
    _linear("moe_grouped_linear_fp8", _types()[1], x, x_scale, w, w_scale, expert_first_token_offset, y, bias,
            residual, activation, stream)
