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

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from .binding import BEAM_OK, BeamMoEError, library

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
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"{name}: expected one of {list(table)}, got {value!r}") from None


def _check(rc: int):
    if rc != BEAM_OK:
        raise BeamMoEError(rc, library().beam_ops_error().decode())


def _cuda(t, name: str, dtype=None, device=None):
    """`t` is a CUDA tensor (of `dtype`, on `device`)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor, got {t.device if isinstance(t, torch.Tensor) else type(t)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the others on {device}")
    return t


def _rows(t, name: str, device=None):
    """A 2-D matrix of a supported type whose rows are contiguous -> row stride."""
    _cuda(t, name, device=device)
    if t.dtype not in DTYPES:
        raise TypeError(f"{name}: expected one of {list(DTYPES)}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise TypeError(f"{name}: expected a matrix with contiguous rows, got shape {tuple(t.shape)}, "
                        f"strides {t.stride()}")
    if t.shape[0] <= 1:
        return t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise TypeError(f"{name}: rows overlap (stride {t.stride(0)} for {t.shape[1]} elements)")
    return t.stride(0)


def _flat(t, name: str, dtype, n: int, device):
    """A contiguous tensor of n elements."""
    _cuda(t, name, dtype, device)
    if not t.is_contiguous() or t.numel() != n:
        raise TypeError(f"{name}: expected {n} contiguous elements, got shape {tuple(t.shape)} "
                        f"(contiguous={t.is_contiguous()})")
    return t


def _out(t, name: str, shape, dtype, device):
    """An output matrix the caller gave -> row stride."""
    ld = _rows(t, name, device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return ld


def _p(t):
    return None if t is None else t.data_ptr()


class _On:
    """The device and stream a call runs on: `stream` or the device's current
    stream; tensors are made there and, on another stream than the current
    one, marked as used there."""

    __slots__ = ("handle", "device", "contexts", "stream")

    def __init__(self, device, stream):
        self.device, self.contexts, self.stream = device, (), None
        if device.index != torch.cuda.current_device():
            self.contexts = (torch.cuda.device(device),)
        current = torch.cuda.current_stream(device)
        if stream is None:
            self.handle = current.cuda_stream
            return
        self.handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if self.handle != current.cuda_stream:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(self.handle, device=device)
            if stream.device != device:
                raise ValueError(f"stream on {stream.device}, tensors on {device}")
            self.stream = stream
            self.contexts += (torch.cuda.stream(stream),)

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)

    def used(self, *tensors):
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)


def ops_status(device=None, stream=None) -> int:
    """Wait for `stream`, then read and clear the device's status word."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _On(device, stream) as on:
        return library().beam_ops_status(on.handle)


# --- microscaled operands ------------------------------------------------------

def scale_bytes(format: str, rows: int, K: int, layout: str) -> int:
    n = library().beam_mx_scale_bytes(_key(FORMATS, format, "format"), rows, K, _key(LAYOUTS, layout, "layout"))
    if n < 0:
        raise BeamMoEError(int(n), library().beam_ops_error().decode())
    return n


def _new_mx(format: str, layout: str, rows: int, K: int, device) -> MxTensor:
    n = scale_bytes(format, rows, K, layout)
    codes = torch.empty(rows, K if format == "mxfp8" else K // 2, dtype=torch.uint8, device=device)
    scales = torch.empty((rows, K // BLOCK[format]) if layout == "rows" else n, dtype=torch.uint8, device=device)
    return MxTensor(codes, scales, format, layout, rows, K)


def _mx(q: MxTensor, name: str, device=None):
    """Types, sizes and device of an operand's tensors."""
    if not isinstance(q, MxTensor):
        raise TypeError(f"{name}: expected an MxTensor, got {type(q)}")
    _key(FORMATS, q.format, name + ".format")
    device = _cuda(q.codes, name + ".codes").device if device is None else device
    _flat(q.codes, name + ".codes", torch.uint8, q.rows * (q.K if q.format == "mxfp8" else q.K // 2), device)
    _flat(q.scales, name + ".scales", torch.uint8, scale_bytes(q.format, q.rows, q.K, q.layout), device)
    if q.tensor_scale is not None:
        _flat(q.tensor_scale, name + ".tensor_scale", torch.float32, 1, device)
    return device


def mx_tensor_scale(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The NVFP4 scale of x [rows, K]: the least power of two g with amax <= 6 * 448 * g (fp32 [1])."""
    ld = _rows(x, "x")
    if x.shape[1] < 1:
        raise ValueError("x: rows of no elements")
    with _On(x.device, stream) as on:
        if out is None:
            out = torch.empty(1, dtype=torch.float32, device=x.device)
        _flat(out, "out", torch.float32, 1, x.device)
        _check(library().beam_mx_tensor_scale(on.handle, _p(x), DTYPES[x.dtype], x.shape[0], x.shape[1], ld, _p(out)))
        on.used(x, out)
    return out


def mx_quantize(x: torch.Tensor, format: str, layout: str = "rows", tensor_scale: Optional[torch.Tensor] = None,
                out: Optional[MxTensor] = None, stream=None) -> MxTensor:
    """x [rows, K] (bf16, fp16 or fp32, rows may be strided) to a microscaled operand.

    NVFP4 without a `tensor_scale` (fp32 [1]) finds one first (mx_tensor_scale:
    one more pass over x).  layout "rows" is what BeamMoE.nvfp4 and checkpoints
    take, "tiled" what mx_matmul takes.  `out`: an operand of the same shape to
    write into (its tensor_scale is not)."""
    ld = _rows(x, "x")
    rows, K = x.shape
    f, l = _key(FORMATS, format, "format"), _key(LAYOUTS, layout, "layout")
    with _On(x.device, stream) as on:
        if out is None:
            out = _new_mx(format, layout, rows, K, x.device)
        else:
            _mx(out, "out", x.device)
            if (out.format, out.layout, out.rows, out.K) != (format, layout, rows, K):
                raise ValueError(f"out: {out.format} {out.layout} {out.rows} x {out.K}, "
                                 f"not {format} {layout} {rows} x {K}")
        if format == "nvfp4":
            if tensor_scale is None:
                tensor_scale = mx_tensor_scale(x)
            _flat(tensor_scale, "tensor_scale", torch.float32, 1, x.device)
        elif tensor_scale is not None:
            raise ValueError(f"{format} has no tensor scale")
        _check(library().beam_mx_quantize(on.handle, _p(x), DTYPES[x.dtype], rows, K, ld, f, l, _p(tensor_scale),
                                          _p(out.codes), _p(out.scales)))
        on.used(x, tensor_scale, out.codes, out.scales)
    return out._replace(tensor_scale=tensor_scale)


def mx_dequantize(q: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of a microscaled operand, [rows, K]."""
    device = _mx(q, "q")
    d = _key(DTYPES, dtype, "dtype")
    with _On(device, stream) as on:
        if out is None:
            out = torch.empty(q.rows, q.K, dtype=dtype, device=device)
        ld = _out(out, "out", (q.rows, q.K), dtype, device)
        _check(library().beam_mx_dequantize(on.handle, _p(q.codes), _p(q.scales), _p(q.tensor_scale),
                                            FORMATS[q.format], LAYOUTS[q.layout], q.rows, q.K, _p(out), d, ld))
        on.used(q.codes, q.scales, q.tensor_scale, out)
    return out


def mx_tile_scales(q: MxTensor, stream=None) -> MxTensor:
    """The same operand with its scales in the "tiled" layout (once, for a checkpoint's weights)."""
    device = _mx(q, "q")
    if q.layout == "tiled":
        return q
    with _On(device, stream) as on:
        tiled = torch.empty(scale_bytes(q.format, q.rows, q.K, "tiled"), dtype=torch.uint8, device=device)
        _check(library().beam_mx_tile_scales(on.handle, FORMATS[q.format], _p(q.scales), q.rows, q.K, _p(tiled)))
        on.used(q.scales, tiled)
    return q._replace(scales=tiled, layout="tiled")


def mx_matmul(a: MxTensor, w: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """a [T, K] . w [N, K]^T -> [T, N]: NVFP4 x NVFP4, MXFP4 x MXFP4, MXFP8 x MXFP4 or MXFP8 x MXFP8, scales tiled."""
    device = _mx(a, "a")
    _mx(w, "w", device)
    d = _key(DTYPES, dtype, "dtype")
    if a.layout != "tiled" or w.layout != "tiled":
        raise ValueError("mx_matmul takes scales in the tiled layout (mx_tile_scales)")
    if a.K != w.K:
        raise ValueError(f"a has {a.K} columns, w {w.K}")
    with _On(device, stream) as on:
        if out is None:
            out = torch.empty(a.rows, w.rows, dtype=dtype, device=device)
        ld = _out(out, "out", (a.rows, w.rows), dtype, device)
        _check(library().beam_mx_matmul(on.handle, FORMATS[a.format], _p(a.codes), _p(a.scales), _p(a.tensor_scale),
                                        FORMATS[w.format], _p(w.codes), _p(w.scales), _p(w.tensor_scale),
                                        a.rows, w.rows, a.K, _p(out), d, ld))
        on.used(a.codes, a.scales, a.tensor_scale, w.codes, w.scales, w.tensor_scale, out)
    return out


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
    ldx = _rows(x, "x")
    T, H = x.shape
    device = x.device
    _flat(gamma, "gamma", torch.float32, H, device)
    d = _key(DTYPES, dtype, "dtype")
    lay = _key(LAYOUTS, layout, "layout")
    if quantize not in (None, "mxfp8"):
        raise ValueError(f"quantize: expected None or 'mxfp8', got {quantize!r}")
    ldr = ldro = ldo = 0
    if residual is not None:
        ldr = _rows(residual, "residual", device)
        if tuple(residual.shape) != (T, H) or residual.dtype not in (torch.float32, x.dtype):
            raise TypeError(f"residual: expected fp32 or {x.dtype} {(T, H)}, got {residual.dtype} {tuple(residual.shape)}")
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    if out is not None and not want_out:
        raise ValueError("out given, but want_out is false")
    if quantized is not None and quantize is None:
        raise ValueError("quantized given, but quantize is None")
    with _On(device, stream) as on:
        if residual is not None:
            if residual_out is None:
                residual_out = torch.empty(T, H, dtype=residual.dtype, device=device)
            ldro = _out(residual_out, "residual_out", (T, H), residual.dtype, device)
        if want_out:
            if out is None:
                out = torch.empty(T, H, dtype=dtype, device=device)
            ldo = _out(out, "out", (T, H), dtype, device)
        if quantize is not None:
            if quantized is None:
                quantized = _new_mx(quantize, layout, T, H, device)
            else:
                _mx(quantized, "quantized", device)
                if (quantized.format, quantized.layout, quantized.rows, quantized.K) != (quantize, layout, T, H):
                    raise ValueError(f"quantized: {quantized.format} {quantized.layout} {quantized.rows} x "
                                     f"{quantized.K}, not {quantize} {layout} {T} x {H}")
        codes, scales = (None, None) if quantized is None else (quantized.codes, quantized.scales)
        _check(library().beam_rms_norm(
            on.handle, _p(x), DTYPES[x.dtype], ldx, _p(residual), 0 if residual is None else DTYPES[residual.dtype],
            ldr, _p(residual_out), ldro, alpha, beta, _p(gamma), eps, T, H, _p(out), d, ldo, _p(codes), _p(scales), lay))
        on.used(x, gamma, residual, residual_out, out, codes, scales)
    return NormResult(out, residual_out, quantized)


def route_scores(logits: torch.Tensor, top_k: int, score: str = "sigmoid", bias: Optional[torch.Tensor] = None,
                 n_group: int = 1, topk_group: int = 1, group_top: int = 2, renormalize: bool = True,
                 scale: float = 1.0, idx: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Experts (int32 [T, top_k]) and weights (fp32 [T, top_k]) from router logits fp32 [T, E].

    Scores are sigmoid(logit) or the row's softmax; `bias` (fp32 [E]) steers
    the choice only; with topk_group < n_group the groups are ranked by the
    sum of their `group_top` best keys first.  A logit of -inf masks an
    expert; slots with no expert left get index -1, weight 0."""
    _cuda(logits, "logits", torch.float32)
    ld = _rows(logits, "logits")
    T, E = logits.shape
    device = logits.device
    s = _key(SCORES, score, "score")
    if bias is not None:
        _flat(bias, "bias", torch.float32, E, device)
    with _On(device, stream) as on:
        if idx is None:
            idx = torch.empty(T, max(top_k, 0), dtype=torch.int32, device=device)
        if w is None:
            w = torch.empty(T, max(top_k, 0), dtype=torch.float32, device=device)
        _flat(idx, "idx", torch.int32, T * top_k, device)
        _flat(w, "w", torch.float32, T * top_k, device)
        _check(library().beam_route_scores(on.handle, _p(logits), T, E, ld, s, _p(bias), n_group, topk_group,
                                           group_top, top_k, int(bool(renormalize)), scale, _p(idx), _p(w)))
        on.used(logits, bias, idx, w)
    return idx, w
