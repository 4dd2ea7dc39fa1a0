"""Operators around the MoE block that need no handle (``include/beam_ops.h``).

``rms_norm``      residual addition and RMSNorm, out in 16 / 32 bits and / or MXFP8;
``mx_quantize``   rows to NVFP4, MXFP4 or MXFP8 (``mx_dequantize`` reads them back,
                  ``mx_tensor_scale`` finds an NVFP4 tensor scale, ``mx_tile_scales``
                  lays a checkpoint's scales out for the product);
``mx_matmul``     the product of two microscaled operands on the block-scaled tensor cores;
``route_scores``  experts and weights from logits, softmax or sigmoid scores.

Argument marshalling only, as in ``binding``: the work is the library's CUDA
kernels; PyTorch supplies device memory and streams.  The checks of tensors
and the outputs are made in ``csrc/ops_binding.cpp``, since they run beside
kernels of a few microseconds.  Every call runs on the device of its tensors,
on ``stream`` or that device's current stream.  Where ``stream`` is another
one than the current stream, the caller orders the two for the inputs; outputs
are made on ``stream`` and both are marked as used there.

For inference: there is no backward pass.  Inputs may require a gradient (a
layer's parameters do), results never do and nothing is recorded, also where
gradients are enabled.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple, Optional, Tuple

import torch

from .binding import BEAM_ERR_INVALID_ARG, BeamMoEError, library
from .build import OPS_BINDING

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
FORMATS = {"nvfp4": 0, "mxfp4": 1, "mxfp8": 2}
LAYOUTS = {"rows": 0, "tiled": 1}
SCORES = {"sigmoid": 0, "softmax": 1}
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


class MxTensor(NamedTuple):
    """A microscaled operand of `rows` x `K` elements.

    codes         uint8 [rows, K / 2] (E2M1 pairs, the first in the low nibble) or [rows, K] (E4M3)
    scales        uint8, [rows, K / block] ("rows") or flat, as beam_ops.h lays it out ("tiled")
    tensor_scale  fp32 [1] (NVFP4) or None
    """
    codes: torch.Tensor
    scales: torch.Tensor
    format: str
    layout: str
    rows: int
    K: int
    tensor_scale: Optional[torch.Tensor] = None


class NormResult(NamedTuple):
    out: Optional[torch.Tensor]
    residual: Optional[torch.Tensor]
    quantized: Optional[MxTensor]


def _key(table, value, name):
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name}: expected one of {list(table)}, got {value!r}")
    return code


_binding = None


def _native():
    """The compiled binding, given the library's functions once (raises if either has not been built)."""
    global _binding
    if _binding is None:
        lib = library()
        if not os.path.exists(OPS_BINDING):
            raise RuntimeError(f"{OPS_BINDING} is missing: build it with "
                               "`python -m group_limited_routing_sigmoid_b200.build`")
        spec = importlib.util.spec_from_file_location(__package__ + "._ops_binding", OPS_BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(BeamMoEError, NormResult, MxTensor, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.beam_rms_norm, lib.beam_mx_tensor_scale, lib.beam_mx_quantize, lib.beam_mx_quantize_nvfp4, lib.beam_mx_dequantize,
            lib.beam_mx_tile_scales, lib.beam_mx_matmul, lib.beam_route_scores, lib.beam_ops_error)))
        _binding = module
    return _binding


def _elsewhere(stream, f, *args):
    """f(*args) on `stream` of the first argument's device, all tensors marked as used there."""
    first = args[0].codes if isinstance(args[0], MxTensor) else args[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        return f(*args)                # which refuses it
    device = first.device
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    with torch.cuda.device(device):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle == torch.cuda.current_stream(device).cuda_stream:
            return f(*args)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(handle, device=device)
        with torch.cuda.stream(stream):
            result = f(*args)
        _used(stream, *args, result)
        return result


def _used(stream, *values):
    for v in values:
        if isinstance(v, torch.Tensor) and v.is_cuda:
            v.record_stream(stream)
        elif isinstance(v, tuple):
            _used(stream, *v)


def ops_status(device=None, stream=None) -> int:
    """Wait for `stream`, then read and clear the device's status word.

    0, or BEAM_ERR_TIMEOUT when a bounded wait inside mx_matmul ran out since
    the last call.  mx_matmul does not look at the word itself (that would wait
    for the GPU): the result of that product, and of every later one on the
    device until this call, is not valid and raises nothing, so a program looks
    here where it synchronises anyway, before it uses what it computed."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        return library().beam_ops_status(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


# --- microscaled operands ------------------------------------------------------

def scale_bytes(format: str, rows: int, K: int, layout: str) -> int:
    """Bytes of the scales of a [rows, K] operand (beam_mx_scale_bytes)."""
    block = BLOCK.get(format)
    if block is None or layout not in LAYOUTS:
        raise ValueError(f"format {format!r}, layout {layout!r}: expected one of {list(FORMATS)}, {list(LAYOUTS)}")
    if rows < 0 or K <= 0 or K % block:
        raise BeamMoEError(BEAM_ERR_INVALID_ARG,
                           f"{format}: K must be a positive multiple of {block} and rows >= 0, got {rows} x {K}")
    n = K // block
    return rows * n if layout == "rows" else (rows + 127) // 128 * ((n + 3) // 4) * 512


def _operand(q, name: str):
    """Fields of an operand: codes, scales, tensor scale, codes of its format and layout, rows, K."""
    if not isinstance(q, MxTensor):
        raise TypeError(f"{name}: expected an MxTensor, got {type(q)}")
    codes, scales, format, layout, rows, K, tensor_scale = q
    return codes, scales, tensor_scale, _key(FORMATS, format, name), _key(LAYOUTS, layout, name), rows, K


def _given(q, name: str, format: str, layout: str, x):
    """Codes and scales of an operand to write into: of this format and layout and x's shape."""
    codes, scales, _, _, _, rows, K = _operand(q, name)
    if codes is None or scales is None:
        raise TypeError(f"{name}: an operand to write into has codes and scales")
    if (q.format, q.layout, rows, K) != (format, layout, *x.shape):
        raise ValueError(f"{name}: {q.format} {q.layout} {rows} x {K}, not {format} {layout} {tuple(x.shape)}")
    return codes, scales


def mx_tensor_scale(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The NVFP4 scale of x [rows, K]: the least power of two g with amax <= 6 * 448 * g (fp32 [1]).

    With elements above 1.4e37 it is above 2^112, under which mx_quantize gives
    NaN; mx_quantize finding the scale itself stops at 2^112."""
    f = (_binding or _native()).tensor_scale
    return f(x, out) if stream is None else _elsewhere(stream, f, x, out)


def mx_quantize(x: torch.Tensor, format: str, layout: str = "rows", tensor_scale: Optional[torch.Tensor] = None,
                out: Optional[MxTensor] = None, stream=None) -> MxTensor:
    """x [rows, K] (bf16, fp16 or fp32, rows may be strided) to a microscaled operand.

    NVFP4 without a `tensor_scale` (fp32 [1]) finds one first (mx_tensor_scale,
    2^112 at most: one more pass over x).  layout "rows" is what BeamMoE.nvfp4 and checkpoints
    take, "tiled" what mx_matmul takes.  `out`: an operand of the same shape to
    write into (its tensor_scale is not)."""
    f, lay = _key(FORMATS, format, "format"), _key(LAYOUTS, layout, "layout")
    codes, scales = (None, None) if out is None else _given(out, "out", format, layout, x)
    if f != 0 and tensor_scale is not None:
        raise ValueError(f"{format} has no tensor scale")
    q = (_binding or _native()).quantize
    if stream is None:
        return q(x, f, lay, tensor_scale, codes, scales, format, layout)
    return _elsewhere(stream, q, x, f, lay, tensor_scale, codes, scales, format, layout)


def mx_dequantize(q: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of a microscaled operand, [rows, K]."""
    d = _key(DTYPES, dtype, "dtype")
    f = (_binding or _native()).dequantize
    return f(q, d, out) if stream is None else _elsewhere(stream, f, q, d, out)


def mx_tile_scales(q: MxTensor, stream=None) -> MxTensor:
    """The same operand with its scales in the "tiled" layout (once, for a checkpoint's weights)."""
    _, scales, _, format, _, rows, K = _operand(q, "q")
    if q.layout == "tiled":
        return q
    f = (_binding or _native()).tile_scales
    tiled = f(scales, format, rows, K) if stream is None else _elsewhere(stream, f, scales, format, rows, K)
    return q._replace(scales=tiled, layout="tiled")


def mx_matmul(a: MxTensor, w: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """a [T, K] . w [N, K]^T -> [T, N]: NVFP4 x NVFP4, MXFP4 x MXFP4, MXFP8 x MXFP4 or MXFP8 x MXFP8, scales tiled.

    Its waits on the GPU are bounded; whether one ran out, ops_status tells."""
    d = _key(DTYPES, dtype, "dtype")
    f = (_binding or _native()).matmul
    return f(a, w, d, out) if stream is None else _elsewhere(stream, f, a, w, d, out)


# --- norm and routing ----------------------------------------------------------

def rms_norm(x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None, alpha: float = 1.0,
             beta: float = 1.0, eps: float = 1e-6, dtype=torch.bfloat16, quantize: Optional[str] = None,
             layout: str = "tiled", out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
             want_out: bool = True, quantized: Optional[MxTensor] = None, stream=None) -> NormResult:
    """s = alpha residual + beta x; y = s / sqrt(mean(s^2) + eps) gamma; FP32 inside.

    x [T, H] bf16, fp16 or fp32; residual [T, H] fp32 or x's type, or None;
    gamma fp32 [H].  Returns y in `dtype` (None without want_out), the new
    residual s (None without residual; residual_out may be residual itself,
    to update it in place) and, with quantize="mxfp8", y as an MXFP8 operand.
    `out`, `residual_out`, `quantized`: buffers to write into."""
    codes = scales = None
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without residual")
    if not want_out and out is not None:
        raise ValueError("out given, but want_out is false")
    if quantize is not None and quantize != "mxfp8":
        raise ValueError(f"quantize: expected None or 'mxfp8', got {quantize!r}")
    if quantized is not None:
        if quantize is None:
            raise ValueError("quantized given, but quantize is None")
        codes, scales = _given(quantized, "quantized", quantize, layout, x)
    f = (_binding or _native()).rms_norm
    d, lay = _key(DTYPES, dtype, "dtype"), _key(LAYOUTS, layout, "layout")
    want_out = bool(want_out)
    if stream is None:
        return f(x, gamma, residual, alpha, beta, eps, d, quantize, lay, layout, out, residual_out, want_out, codes, scales)
    return _elsewhere(stream, f, x, gamma, residual, alpha, beta, eps, d, quantize, lay, layout, out, residual_out, want_out,
                      codes, scales)


def route_scores(logits: torch.Tensor, top_k: int, score: str = "sigmoid", bias: Optional[torch.Tensor] = None,
                 n_group: int = 1, topk_group: int = 1, group_top: int = 2, renormalize: bool = True,
                 scale: float = 1.0, idx: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Experts (int32 [T, top_k]) and weights (fp32 [T, top_k]) from router logits fp32 [T, E].

    Scores are sigmoid(logit) or the row's softmax; `bias` (fp32 [E]) steers
    the choice only; with topk_group < n_group the groups are ranked by the
    sum of their `group_top` best keys first.  A logit of -inf masks an
    expert; slots with no expert left get index -1, weight 0.  Near ties are
    decided in 64 bits, by the handle's router (BeamMoE.route_logits) in FP32:
    use that one beside a handle's own routing."""
    s = _key(SCORES, score, "score")
    f = (_binding or _native()).route_scores
    if stream is None:
        return f(logits, top_k, s, bias, n_group, topk_group, group_top, renormalize, scale, idx, w)
    return _elsewhere(stream, f, logits, top_k, s, bias, n_group, topk_group, group_top, renormalize, scale, idx, w)
