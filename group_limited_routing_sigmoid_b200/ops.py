"""Operators around the MoE block that need no handle (``include/beam_ops.h``).

``rms_norm``      residual addition and RMSNorm, out in 16 / 32 bits and / or MXFP8;
``mx_quantize``   rows to NVFP4, MXFP4 or MXFP8 (``mx_dequantize`` reads them back,
                  ``mx_tensor_scale`` finds an NVFP4 tensor scale, ``mx_tile_scales``
                  lays a checkpoint's scales out for the product);
``mx_matmul``     the product of two microscaled operands on the block-scaled tensor cores;
``route_scores``  experts and weights from logits, softmax or sigmoid scores.

Argument marshalling only, as in ``binding``: the work is the library's CUDA
kernels; PyTorch supplies device memory and streams.  Every call runs on the
device of its tensors, on ``stream`` or that device's current stream.  Where
``stream`` is another one than the current stream, the caller orders the two
for the inputs; outputs are made on ``stream`` and both are marked as used
there.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from .binding import BEAM_ERR_INVALID_ARG, BEAM_OK, BeamMoEError, library

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


def _check(rc: int):
    if rc != BEAM_OK:
        raise BeamMoEError(rc, library().beam_ops_error().decode())


# The checks below run on every call, beside kernels of a few microseconds:
# they read each property of a tensor once and take the common case first.

def _bad_device(t, name: str, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor, got {t.device if isinstance(t, torch.Tensor) else type(t)}")
    raise ValueError(f"{name}: on {t.device}, the others on {device}")


def _rows(t, name: str, device=None):
    """A matrix of a supported type on `device` (any CUDA device when None)
    whose rows are contiguous -> (rows, columns, row stride, type code)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (device is not None and t.device != device):
        _bad_device(t, name, device)
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected one of {list(DTYPES)}, got {t.dtype}")
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        if t.is_contiguous():
            return rows, cols, cols, code
        if cols <= 1 or t.stride(1) == 1:
            ld = t.stride(0)
            if rows <= 1:
                return rows, cols, cols, code
            if ld >= cols:
                return rows, cols, ld, code
            raise TypeError(f"{name}: rows overlap (stride {ld} for {cols} elements)")
    raise TypeError(f"{name}: expected a matrix with contiguous rows, got shape {tuple(shape)}, strides {t.stride()}")


def _flat(t, name: str, dtype, n: int, device):
    """A contiguous tensor of n elements of `dtype` on `device` -> its address."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        _bad_device(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise TypeError(f"{name}: expected {n} contiguous elements, got shape {tuple(t.shape)} "
                        f"(contiguous={t.is_contiguous()})")
    return t.data_ptr()


def _out(t, name: str, rows: int, cols: int, dtype, device) -> int:
    """An output matrix the caller gave -> its row stride."""
    r, c, ld, _ = _rows(t, name, device)
    if r != rows or c != cols or t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype} {(rows, cols)}, got {t.dtype} {tuple(t.shape)}")
    return ld


# The current stream's handle without a Stream object around it, where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, stream, body, *args):
    """body(stream handle, *args) on `device` and `stream` (None: the device's
    current stream).  body returns (result, tensors it uses): those are made
    on that stream and, where it is another one than the current stream,
    marked as used there."""
    if stream is None and device.index == torch.cuda.current_device():
        return body(_raw_stream(device.index), *args)[0]
    with torch.cuda.device(device):
        current = _raw_stream(device.index)
        if stream is None:
            return body(current, *args)[0]
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle == current:
            return body(current, *args)[0]
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(handle, device=device)
        if stream.device != device:
            raise ValueError(f"stream on {stream.device}, tensors on {device}")
        with torch.cuda.stream(stream):
            result, tensors = body(handle, *args)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return result


def ops_status(device=None, stream=None) -> int:
    """Wait for `stream`, then read and clear the device's status word."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return _on(device, stream, lambda handle: (library().beam_ops_status(handle), ()))


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


def _new_mx(format: str, layout: str, rows: int, K: int, device) -> MxTensor:
    n = scale_bytes(format, rows, K, layout)
    codes = torch.empty((rows, K if format == "mxfp8" else K // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((rows, K // BLOCK[format]) if layout == "rows" else n, dtype=torch.uint8, device=device)
    return MxTensor(codes, scales, format, layout, rows, K)


def _mx(q: MxTensor, name: str, device=None):
    """Types, sizes and device of an operand's tensors -> (device, addresses of codes, scales, tensor scale)."""
    if not isinstance(q, MxTensor):
        raise TypeError(f"{name}: expected an MxTensor, got {type(q)}")
    codes, scales, fmt, layout, rows, K, ts = q
    n = scale_bytes(fmt, rows, K, layout)
    if device is None:
        if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
            _bad_device(codes, name + ".codes", device)
        device = codes.device
    return (device, _flat(codes, name, torch.uint8, rows * (K if fmt == "mxfp8" else K // 2), device),
            _flat(scales, name, torch.uint8, n, device),
            None if ts is None else _flat(ts, name, torch.float32, 1, device))


def _given_mx(q: MxTensor, name: str, format: str, layout: str, rows: int, K: int, device):
    """An operand to write into: of this format, layout and shape -> addresses of codes, scales."""
    _, codes, scales, _ = _mx(q, name, device)
    if (q.format, q.layout, q.rows, q.K) != (format, layout, rows, K):
        raise ValueError(f"{name}: {q.format} {q.layout} {q.rows} x {q.K}, not {format} {layout} {rows} x {K}")
    return codes, scales


def _tensor_scale(handle, x, shape, out):
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    rows, K, ld, code = shape
    _check(library().beam_mx_tensor_scale(handle, x.data_ptr(), code, rows, K, ld,
                                          _flat(out, "out", torch.float32, 1, x.device)))
    return out, (x, out)


def mx_tensor_scale(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The NVFP4 scale of x [rows, K]: the least power of two g with amax <= 6 * 448 * g (fp32 [1])."""
    return _on(x.device, stream, _tensor_scale, x, _rows(x, "x"), out)


def _quantize(handle, x, shape, format, f, layout, lay, tensor_scale, out):
    rows, K, ld, code = shape
    device = x.device
    if out is None:
        out = _new_mx(format, layout, rows, K, device)
        codes, scales = out.codes.data_ptr(), out.scales.data_ptr()
    else:
        codes, scales = _given_mx(out, "out", format, layout, rows, K, device)
    ts = None
    if f == 0:
        if tensor_scale is None:
            tensor_scale, _ = _tensor_scale(handle, x, shape, None)
        ts = _flat(tensor_scale, "tensor_scale", torch.float32, 1, device)
    elif tensor_scale is not None:
        raise ValueError(f"{format} has no tensor scale")
    _check(library().beam_mx_quantize(handle, x.data_ptr(), code, rows, K, ld, f, lay, ts, codes, scales))
    out = MxTensor(out.codes, out.scales, format, layout, rows, K, tensor_scale)
    return out, (x, tensor_scale, out.codes, out.scales)


def mx_quantize(x: torch.Tensor, format: str, layout: str = "rows", tensor_scale: Optional[torch.Tensor] = None,
                out: Optional[MxTensor] = None, stream=None) -> MxTensor:
    """x [rows, K] (bf16, fp16 or fp32, rows may be strided) to a microscaled operand.

    NVFP4 without a `tensor_scale` (fp32 [1]) finds one first (mx_tensor_scale:
    one more pass over x).  layout "rows" is what BeamMoE.nvfp4 and checkpoints
    take, "tiled" what mx_matmul takes.  `out`: an operand of the same shape to
    write into (its tensor_scale is not)."""
    return _on(x.device, stream, _quantize, x, _rows(x, "x"), format, _key(FORMATS, format, "format"), layout,
               _key(LAYOUTS, layout, "layout"), tensor_scale, out)


def _dequantize(handle, q, device, codes, scales, ts, dtype, d, out):
    if out is None:
        out = torch.empty((q.rows, q.K), dtype=dtype, device=device)
        ld = q.K
    else:
        ld = _out(out, "out", q.rows, q.K, dtype, device)
    _check(library().beam_mx_dequantize(handle, codes, scales, ts, FORMATS[q.format], LAYOUTS[q.layout], q.rows, q.K,
                                        out.data_ptr(), d, ld))
    return out, (q.codes, q.scales, q.tensor_scale, out)


def mx_dequantize(q: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of a microscaled operand, [rows, K]."""
    device, codes, scales, ts = _mx(q, "q")
    return _on(device, stream, _dequantize, q, device, codes, scales, ts, dtype, _key(DTYPES, dtype, "dtype"), out)


def _tile(handle, q, device, scales):
    tiled = torch.empty(scale_bytes(q.format, q.rows, q.K, "tiled"), dtype=torch.uint8, device=device)
    _check(library().beam_mx_tile_scales(handle, FORMATS[q.format], scales, q.rows, q.K, tiled.data_ptr()))
    return q._replace(scales=tiled, layout="tiled"), (q.scales, tiled)


def mx_tile_scales(q: MxTensor, stream=None) -> MxTensor:
    """The same operand with its scales in the "tiled" layout (once, for a checkpoint's weights)."""
    device, _, scales, _ = _mx(q, "q")
    return q if q.layout == "tiled" else _on(device, stream, _tile, q, device, scales)


def _matmul(handle, a, w, device, pa, pw, dtype, d, out):
    T, N = a.rows, w.rows
    if out is None:
        out = torch.empty((T, N), dtype=dtype, device=device)
        ld = N
    else:
        ld = _out(out, "out", T, N, dtype, device)
    _check(library().beam_mx_matmul(handle, FORMATS[a.format], pa[1], pa[2], pa[3], FORMATS[w.format], pw[1], pw[2],
                                    pw[3], T, N, a.K, out.data_ptr(), d, ld))
    return out, (a.codes, a.scales, a.tensor_scale, w.codes, w.scales, w.tensor_scale, out)


def mx_matmul(a: MxTensor, w: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """a [T, K] . w [N, K]^T -> [T, N]: NVFP4 x NVFP4, MXFP4 x MXFP4, MXFP8 x MXFP4 or MXFP8 x MXFP8, scales tiled."""
    pa = _mx(a, "a")
    device = pa[0]
    pw = _mx(w, "w", device)
    if a.layout != "tiled" or w.layout != "tiled":
        raise ValueError("mx_matmul takes scales in the tiled layout (mx_tile_scales)")
    if a.K != w.K:
        raise ValueError(f"a has {a.K} columns, w {w.K}")
    return _on(device, stream, _matmul, a, w, device, pa, pw, dtype, _key(DTYPES, dtype, "dtype"), out)


# --- norm and routing ----------------------------------------------------------

def _norm(handle, x, shape, gamma, residual, alpha, beta, eps, dtype, quantize, layout, out, residual_out, want_out,
          quantized):
    T, H, ldx, code = shape
    device = x.device
    d, lay = _key(DTYPES, dtype, "dtype"), _key(LAYOUTS, layout, "layout")
    pr = pro = po = codes = scales = None
    ldr = ldro = ldo = rd = 0
    if residual is not None:
        rt, rh, ldr, rd = _rows(residual, "residual", device)
        if rt != T or rh != H or (rd != 2 and rd != code):
            raise TypeError(f"residual: expected fp32 or {x.dtype} {(T, H)}, got {residual.dtype} {tuple(residual.shape)}")
        if residual_out is None:
            residual_out = torch.empty((T, H), dtype=residual.dtype, device=device)
            ldro = H
        else:
            ldro = _out(residual_out, "residual_out", T, H, residual.dtype, device)
        pr, pro = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    if want_out:
        if out is None:
            out = torch.empty((T, H), dtype=dtype, device=device)
            ldo = H
        else:
            ldo = _out(out, "out", T, H, dtype, device)
        po = out.data_ptr()
    elif out is not None:
        raise ValueError("out given, but want_out is false")
    if quantize is not None:
        if quantize != "mxfp8":
            raise ValueError(f"quantize: expected None or 'mxfp8', got {quantize!r}")
        if quantized is None:
            quantized = _new_mx(quantize, layout, T, H, device)
            codes, scales = quantized.codes.data_ptr(), quantized.scales.data_ptr()
        else:
            codes, scales = _given_mx(quantized, "quantized", quantize, layout, T, H, device)
    elif quantized is not None:
        raise ValueError("quantized given, but quantize is None")
    _check(library().beam_rms_norm(handle, x.data_ptr(), code, ldx, pr, rd, ldr, pro, ldro, alpha, beta,
                                   _flat(gamma, "gamma", torch.float32, H, device), eps, T, H, po, d, ldo, codes, scales,
                                   lay))
    return NormResult(out, residual_out, quantized), (
        x, gamma, residual, residual_out, out, *(() if quantized is None else quantized[:2]))


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
    shape = _rows(x, "x")
    return _on(x.device, stream, _norm, x, shape, gamma, residual, alpha, beta, eps, dtype, quantize, layout, out,
               residual_out, want_out, quantized)


def _route(handle, logits, shape, top_k, s, bias, n_group, topk_group, group_top, renormalize, scale, idx, w):
    T, E, ld, code = shape
    device = logits.device
    if code != 2:
        raise TypeError(f"logits: expected torch.float32, got {logits.dtype}")
    k = top_k if top_k > 0 else 0      # refused below
    if idx is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=device)
        pi = idx.data_ptr()
    else:
        pi = _flat(idx, "idx", torch.int32, T * k, device)
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=device)
        pw = w.data_ptr()
    else:
        pw = _flat(w, "w", torch.float32, T * k, device)
    _check(library().beam_route_scores(handle, logits.data_ptr(), T, E, ld, s,
                                       None if bias is None else _flat(bias, "bias", torch.float32, E, device), n_group,
                                       topk_group, group_top, top_k, 1 if renormalize else 0, scale, pi, pw))
    return (idx, w), (logits, bias, idx, w)


def route_scores(logits: torch.Tensor, top_k: int, score: str = "sigmoid", bias: Optional[torch.Tensor] = None,
                 n_group: int = 1, topk_group: int = 1, group_top: int = 2, renormalize: bool = True,
                 scale: float = 1.0, idx: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Experts (int32 [T, top_k]) and weights (fp32 [T, top_k]) from router logits fp32 [T, E].

    Scores are sigmoid(logit) or the row's softmax; `bias` (fp32 [E]) steers
    the choice only; with topk_group < n_group the groups are ranked by the
    sum of their `group_top` best keys first.  A logit of -inf masks an
    expert; slots with no expert left get index -1, weight 0."""
    shape = _rows(logits, "logits")
    return _on(logits.device, stream, _route, logits, shape, top_k, _key(SCORES, score, "score"), bias, n_group,
               topk_group, group_top, renormalize, scale, idx, w)
