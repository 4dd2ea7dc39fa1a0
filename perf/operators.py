"""Measured cases of the handle-free operators around the MoE block.

Four operators, each with its plain form in elementary torch operations:

norm      the residual's addition and the root-mean-square norm in front of a
          block, with the normalised rows in 16 or 32 bits and / or as MXFP8
          (E4M3 elements, one power-of-two scale per 32 elements);
quantize  rows of 16- or 32-bit values to NVFP4, MXFP4 or MXFP8, read back as
          the values they stand for (the codes are 4 or 8 bits); NVFP4 has one
          scale per tensor besides, a power of two, found in the pass or given;
product   out = a . w^T of two microscaled operands: NVFP4 x NVFP4,
          MXFP4 x MXFP4, MXFP8 x MXFP4 and MXFP8 x MXFP8;
route     experts and weights from router logits: softmax or sigmoid scores, a
          bias that steers the choice, groups, top-k, renormalised weights,
          experts masked by a logit of -inf.

Scales come in two layouts.  "rows": uint8 [rows, K / block].  "tiled": the
512-byte tiles that the tensor cores take, [ceil(rows / 128)]
[ceil(K / block / 4)][32][4][4]: byte (row % 32, row / 32 % 4, scale % 4) of
the tile of rows and scales that holds (row, scale); bytes of rows and scales
past the end are zero.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


def listed():
    return [
        # one decoding step of 64 sequences: the stream's update and the bf16
        # rows that the router and the experts read
        dict(name="norm decode 64", op="norm", T=64, H=5120, x="bf16", res="f32", out="bf16",
             q=False, layout="rows"),
        # a prompt batch in front of a microscaled dense layer: bf16 rows for
        # the router and MXFP8 rows, tiled, for the product
        dict(name="norm prefill 8192 mxfp8", op="norm", T=8192, H=5120, x="bf16", res="f32",
             out="bf16", q=True, layout="tiled"),
        # an odd hidden size and a ragged batch, no residual
        dict(name="norm odd 1000x2563", op="norm", T=1000, H=2563, x="f16", res="none", out="f16",
             q=False, layout="rows"),
        # a dense layer's weights on their way into a 4-bit checkpoint; the
        # per-tensor scale is found in the same pass
        dict(name="quantize weights nvfp4", op="quantize", rows=20480, K=5120, dtype="bf16",
             fmt="nvfp4", layout="rows", dynamic=True),
        # a decoding step's activations in front of a 4-bit product
        dict(name="quantize tokens mxfp4", op="quantize", rows=64, K=5120, dtype="bf16",
             fmt="mxfp4", layout="tiled", dynamic=False),
        # FP32 rows of a ragged prompt to 8 bits
        dict(name="quantize ragged mxfp8", op="quantize", rows=1021, K=2592, dtype="f32",
             fmt="mxfp8", layout="tiled", dynamic=False),
        # a dense layer's up projection at a decoding step: 4-bit weights,
        # 8-bit activations
        dict(name="product decode w4a8", op="product", T=64, N=20480, K=5120, a="mxfp8",
             w="mxfp4", out="bf16"),
        # its down projection for one sequence, all in 4 bits
        dict(name="product single nvfp4", op="product", T=1, N=5120, K=20480, a="nvfp4",
             w="nvfp4", out="bf16"),
        # the up projection of a prompt batch
        dict(name="product prefill nvfp4", op="product", T=8192, N=20480, K=5120, a="nvfp4",
             w="nvfp4", out="bf16"),
        # a ragged batch against an odd number of weight rows
        dict(name="product ragged mxfp4", op="product", T=1021, N=5123, K=2560, a="mxfp4",
             w="mxfp4", out="f16"),
        # the Beam router at a long prompt: 256 experts in 8 groups
        dict(name="route sigmoid groups 32768", op="route", T=32768, E=256, k=8, score="sigmoid",
             bias=True, groups=8, keep=4, gtop=2, renorm=True, coarse=False, masked=False),
        # a small softmax router at a decoding step, with padded rows and
        # masked experts, on logits that left a 16-bit product (they tie)
        dict(name="route softmax 64", op="route", T=64, E=60, k=4, score="softmax", bias=False,
             groups=1, keep=1, gtop=1, renorm=False, coarse=True, masked=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "product", "product", "route"))
    if op == "norm":
        q = rng.random() < 0.5
        H = _log(rng, 64, 8192)
        if q:
            H = max(32, H // 32 * 32)
        elif rng.random() < 0.5:
            H = max(8, H // 8 * 8)
        T = _log(rng, 1, min(8192, 8192 * 5120 // H))
        x = rng.choice(("bf16", "f16", "f32"))
        res = rng.choice(("none", "f32") if x == "f32" else ("none", "f32", x))
        return dict(op=op, T=T, H=H, x=x, res=res, out=rng.choice(("bf16", "f16", "f32")), q=q,
                    layout=rng.choice(("rows", "tiled")))
    if op == "quantize":
        fmt = rng.choice(("nvfp4", "mxfp4", "mxfp8"))
        K = max(1, _log(rng, 64, 20480) // BLOCK[fmt]) * BLOCK[fmt]
        rows = _log(rng, 1, min(20480, 20480 * 5120 // K))
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(("bf16", "f16", "f32")) if rows * K < 1 << 25 else "bf16",
                    fmt=fmt, layout=rng.choice(("rows", "tiled")),
                    dynamic=fmt == "nvfp4" and rng.random() < 0.5)
    if op == "product":
        a, w = rng.choice((("nvfp4", "nvfp4"), ("mxfp4", "mxfp4"), ("mxfp8", "mxfp4"),
                           ("mxfp8", "mxfp8")))
        step = 128 if a == "mxfp8" else 64
        K = max(1, _log(rng, 64, 20480) // step) * step
        N = _log(rng, 1, min(20480, 20480 * 5120 // K // (2 if w == "mxfp8" else 1)))
        T = _log(rng, 1, 8192 // (2 if a == "mxfp8" else 1))
        return dict(op=op, T=T, N=N, K=K, a=a, w=w, out=rng.choice(("bf16", "f16")))
    groups = rng.choice((1, 1, 2, 4, 8))
    E = groups * _log(rng, 4, 512 // groups)
    keep = rng.randint(1, groups)
    k = min(rng.choice((1, 2, 4, 6, 8, 8, 12)), E // groups * keep)
    return dict(op=op, T=_log(rng, 1, min(32768, 32768 * 256 // E)), E=E, k=k, score=rng.choice(("sigmoid", "softmax")),
                bias=rng.random() < 0.5, groups=groups, keep=keep, gtop=rng.choice((1, 2)),
                renorm=rng.random() < 0.5, coarse=rng.random() < 0.5, masked=rng.random() < 0.3)


# --- the formats in plain torch ----------------------------------------------

def _e2m1(v):
    """Nearest value of {0, .5, 1, 1.5, 2, 3, 4, 6} with v's sign, ties to the even code."""
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return torch.copysign(torch.round(a / step) * step, v)


def _e4m3(v):
    """Nearest E4M3 value (largest 448), ties to even; works in v's own type."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)                                     # a = m 2^e, m in [0.5, 1)
    e = torch.clamp(e - 4, min=-9).to(torch.int32)           # 4 significant bits, 2^-9 the least
    one = torch.ones_like(a)
    return torch.copysign(torch.ldexp(torch.round(torch.ldexp(a, -e)), e) * one, v)


def _blocks(x, b):
    return x.reshape(x.shape[0], -1, b)


def _pow2_exponent(amax, fmt):
    """Least k with amax <= (largest element) 2^k, in [-127, 127]."""
    m, e = torch.frexp(amax)
    top, shift = (0.875, 9) if fmt == "mxfp8" else (0.75, 3)
    k = torch.where(m <= top, e - shift, e - shift + 1)
    return torch.where(amax > 0, k, -127).clamp(-127, 127).to(torch.int32)


def _tensor_scale(x):
    """The least power of two g with amax <= 6 x 448 g, the amax taken as 2^-100 at least."""
    amax = torch.clamp(x.abs().amax(), min=2.0 ** -100)
    m, e = torch.frexp(amax)                                  # 2688 = 0.65625 x 2^12
    return torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.65625, e - 12, e - 11))


def _quantize(x, fmt, g=None):
    """x [rows, K] -> (elements [rows, K], scales [rows, K / block]) as values, in x's type."""
    b = _blocks(x, BLOCK[fmt])
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        s = _e4m3(amax / (6.0 * g))
        d = (s * g).unsqueeze(-1)
        v = torch.where(d > 0, b / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(b))
        return _e2m1(v).reshape(x.shape), s
    k = _pow2_exponent(amax, fmt)
    v = torch.ldexp(b, -k.unsqueeze(-1))
    q = _e4m3(v) if fmt == "mxfp8" else _e2m1(v)
    return q.reshape(x.shape), torch.ldexp(torch.ones_like(amax), k)


def _tile(s):
    """[rows, scales] in the tiled order, zeros past the ends (any type)."""
    r, n = s.shape
    p = torch.zeros((r + 127) // 128 * 128, (n + 3) // 4 * 4, dtype=s.dtype, device=s.device)
    p[:r, :n] = s
    return p.reshape(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(t, r, n):
    rb, nb = (r + 127) // 128, (n + 3) // 4
    return t.reshape(rb, nb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, nb * 4)[:r, :n]


def _scale_bytes(s, fmt):
    """Scale values to bytes: E4M3 for NVFP4, biased exponents for the others."""
    if fmt == "nvfp4":
        return s.to(torch.float8_e4m3fn).view(torch.uint8)
    _, e = torch.frexp(s)
    return (e + 126).to(torch.uint8)


def _scale_values(b, fmt, dtype):
    if fmt == "nvfp4":
        return b.view(torch.float8_e4m3fn).to(torch.float32).to(dtype)
    return torch.ldexp(torch.ones(b.shape, dtype=dtype, device=b.device), b.to(torch.int32) - 127)


def _codes(q, fmt):
    """Element values to codes: E4M3 bytes, or two E2M1 codes a byte, the first in the low nibble."""
    if fmt == "mxfp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8)
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=q.device)
    c = torch.bucketize(q.abs().float(), grid).to(torch.uint8) + torch.signbit(q).to(torch.uint8) * 8
    return c[:, 0::2] + c[:, 1::2] * 16


def _elements(c, fmt, dtype):
    if fmt == "mxfp8":
        return c.view(torch.float8_e4m3fn).to(torch.float32).to(dtype)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device=c.device)
    grid = torch.cat([grid, -grid])
    return torch.stack([grid[(c & 15).int()], grid[(c >> 4).int()]], -1).reshape(c.shape[0], -1)


def _dequantize(q, s, fmt):
    return (_blocks(q, BLOCK[fmt]) * s.unsqueeze(-1)).reshape(q.shape)


# --- inputs ------------------------------------------------------------------

def _rows(gen, rows, K, dtype):
    """Values as activations and weights have them: normal, some columns ten times as large."""
    x = torch.randn(rows, K, generator=gen, device="cuda")
    big = torch.rand(K, generator=gen, device="cuda") < 0.01
    return (x * (1 + 9 * big)).to(dtype)


def _operand(gen, rows, K, fmt):
    """A quantised operand as a program keeps it: codes, tiled scales, tensor scale."""
    x = _rows(gen, rows, K, torch.float32) * 0.2
    g = _tensor_scale(x) if fmt == "nvfp4" else None
    q, s = _quantize(x, fmt, g)
    return dict(fmt=fmt, rows=rows, K=K, codes=_codes(q, fmt), scales=_tile(_scale_bytes(s, fmt)),
                tensor_scale=None if g is None else g.reshape(1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    op = c["op"]
    if op == "norm":
        T, H = c["T"], c["H"]
        c["xv"] = _rows(gen, T, H, DT[c["x"]])
        c["gamma"] = 1 + 0.02 * torch.randn(H, generator=gen, device="cuda")
        c["alpha"], c["beta"] = (math.sqrt(19 / 20), math.sqrt(1 / 20))
        if c["res"] != "none":
            c["rv"] = torch.randn(T, H, generator=gen, device="cuda").to(DT[c["res"]])
    elif op == "quantize":
        c["xv"] = _rows(gen, c["rows"], c["K"], DT[c["dtype"]])
        # a scale found beforehand on other data of the kind
        c["ts"] = torch.full((1,), 2.0 ** -5, device="cuda") if c["fmt"] == "nvfp4" and not c["dynamic"] else None
    elif op == "product":
        c["av"] = _operand(gen, c["T"], c["K"], c["a"])
        c["wv"] = _operand(gen, c["N"], c["K"], c["w"])
    else:
        T, E = c["T"], c["E"]
        l = torch.randn(T, E, generator=gen, device="cuda") * (1.0 if c["score"] == "sigmoid" else 2.0)
        if c["coarse"]:
            l = l.to(torch.bfloat16).float()
        if c["masked"]:
            l[:, torch.rand(E, generator=gen, device="cuda") < 0.05] = -math.inf
            l[torch.rand(T, generator=gen, device="cuda") < 0.1] = -math.inf
        c["lv"] = l.contiguous()
        c["bv"] = (torch.rand(E, generator=gen, device="cuda") * 0.2 - 0.1) * (1.0 if c["score"] == "sigmoid" else 0.1) if c["bias"] else None
    return c


# --- the plain forms, in the precision of `dt` -------------------------------

def _norm(c, dt):
    s = c["xv"].to(dt)
    if c["res"] != "none":
        s = c["alpha"] * c["rv"].to(dt) + c["beta"] * s
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * c["gamma"].to(dt)
    out = {"out": y}
    if c["res"] != "none":
        out["residual"] = s
    if c["q"]:
        q, sc = _quantize(y, "mxfp8")
        if c["layout"] == "tiled":  # a padding byte of zero stands for 2^-127
            pad = _tile(torch.ones_like(sc, dtype=torch.uint8))
            sc = torch.where(pad > 0, _tile(sc), 2.0 ** -127)
        out["elements"], out["scales"] = q, sc
    return out


def _norm_types(c, out):
    r = {"out": out["out"].to(DT[c["out"]])}
    if "residual" in out:
        r["residual"] = out["residual"].to(DT[c["res"]])
    if c["q"]:
        r["elements"] = out["elements"].to(torch.float8_e4m3fn)
        r["scales"] = _scale_bytes(out["scales"], "mxfp8").view(torch.float8_e8m0fnu)
    return r


def _quantize_op(c, dt):
    x = c["xv"].to(dt)
    g = None
    if c["fmt"] == "nvfp4":
        g = _tensor_scale(x) if c["dynamic"] else c["ts"][0].to(dt)
    q, s = _quantize(x, c["fmt"], g)
    v = _dequantize(q, s, c["fmt"])
    return (v, None) if g is None else (v * g, g.reshape(1))


def _values(o, dt):
    s = _untile(o["scales"], o["rows"], o["K"] // BLOCK[o["fmt"]])
    return _dequantize(_elements(o["codes"], o["fmt"], dt), _scale_values(s, o["fmt"], dt), o["fmt"])


def _product(c, dt):
    y = _values(c["av"], dt) @ _values(c["wv"], dt).t()
    for o in (c["av"], c["wv"]):
        if o["tensor_scale"] is not None:
            y = y * o["tensor_scale"].to(dt)
    return y


def _route(c):
    """Scores and choices in 64 bits: close scores decide which expert comes first."""
    l = c["lv"].double()
    T, E = l.shape
    ok = l > -math.inf
    if c["score"] == "sigmoid":
        p = torch.where(ok, 1 / (1 + torch.exp(-l)), 0.0)
    else:
        m = l.amax(-1, keepdim=True).clamp(min=-1e300)
        p = torch.where(ok, torch.exp(l - m), 0.0)
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    key = p if c["bv"] is None else p + c["bv"].double()
    key = torch.where(ok, key, -math.inf)
    G = c["groups"]
    if G > 1 and c["keep"] < G:
        per = key.reshape(T, G, E // G)
        best = per.sort(dim=-1, descending=True, stable=True).values[..., :c["gtop"]]
        score = torch.where(best > -math.inf, best, 0.0).sum(-1)
        score = torch.where(best[..., 0] > -math.inf, score, -math.inf)
        kept = score.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = torch.where(keep.unsqueeze(-1), per, -math.inf).reshape(T, E)
    best = key.sort(dim=-1, descending=True, stable=True)
    idx, key = best.indices[:, :c["k"]], best.values[:, :c["k"]]
    w = torch.where(key > -math.inf, p.gather(1, idx), 0.0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return torch.where(key > -math.inf, idx, -1).to(torch.int32), w


def run(state):
    c = state
    if own:
        return _run_own(c)
    if c["op"] == "norm":
        return _norm_types(c, _norm(c, torch.float32))
    if c["op"] == "quantize":
        v, g = _quantize_op(c, torch.float32)
        return {"values": v.to(torch.bfloat16)} if g is None else {"values": v.to(torch.bfloat16), "tensor_scale": g}
    if c["op"] == "product":
        return {"out": _product(c, torch.float32).to(DT[c["out"]])}
    idx, w = _route(c)
    return {"idx": idx, "w": w.float()}


def _run_own(c):
    from group_limited_routing_sigmoid_b200 import ops

    if c["op"] == "norm":
        # without a residual the rows are normalised as they are, unscaled
        r = ops.rms_norm(c["xv"], c["gamma"], residual=c.get("rv"), alpha=c["alpha"], beta=c["beta"] if "rv" in c else 1.0,
                         eps=1e-6, dtype=DT[c["out"]], quantize="mxfp8" if c["q"] else None, layout=c["layout"])
        out = {"out": r.out}
        if r.residual is not None:
            out["residual"] = r.residual
        if r.quantized is not None:
            out["elements"] = r.quantized.codes.view(torch.float8_e4m3fn)
            out["scales"] = r.quantized.scales.view(torch.float8_e8m0fnu)
        return out
    if c["op"] == "quantize":
        q = ops.mx_quantize(c["xv"], c["fmt"], layout=c["layout"], tensor_scale=c["ts"])
        out = {"values": ops.mx_dequantize(q, torch.bfloat16)}
        if q.tensor_scale is not None:
            out["tensor_scale"] = q.tensor_scale
        return out
    if c["op"] == "product":
        a, w = (ops.MxTensor(o["codes"], o["scales"], o["fmt"], "tiled", o["rows"], o["K"], o["tensor_scale"])
                for o in (c["av"], c["wv"]))
        return {"out": ops.mx_matmul(a, w, DT[c["out"]])}
    idx, w = ops.route_scores(c["lv"], c["k"], score=c["score"], bias=c["bv"], n_group=c["groups"],
                              topk_group=c["keep"], group_top=c["gtop"], renormalize=c["renorm"])
    return {"idx": idx, "w": w}


def work(case):
    c = case
    size = lambda t: {"bf16": 2, "f16": 2, "f32": 4, "none": 0}[t]  # noqa: E731
    packed = lambda fmt: {"nvfp4": 0.5 + 1 / 16, "mxfp4": 0.5 + 1 / 32, "mxfp8": 1 + 1 / 32}[fmt]  # noqa: E731
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        b = n * (size(c["x"]) + 2 * size(c["res"]) + size(c["out"]) + (packed("mxfp8") if c["q"] else 0))
        return {"bytes": b + 4 * c["H"], "flops": 8 * n}
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        # the rows in, the codes out and in again, the values out
        return {"bytes": n * (size(c["dtype"]) + 2 * packed(c["fmt"]) + 2), "flops": 6 * n}
    if c["op"] == "product":
        return {"bytes": c["T"] * c["K"] * packed(c["a"]) + c["N"] * c["K"] * packed(c["w"]) + 2 * c["T"] * c["N"],
                "flops": 2 * c["T"] * c["N"] * c["K"]}
    return {"bytes": c["T"] * (4 * c["E"] + 8 * c["k"]) + 4 * c["E"] * c["bias"], "flops": 8 * c["T"] * c["E"]}


# --- 64 bits, from the definitions -------------------------------------------

def _nearest(v, grid):
    """The value of the sorted `grid` next to |v|, with v's sign; ties to the even index."""
    a = v.abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    take = torch.where(up == down, torch.where(hi % 2 == 0, hi, lo), torch.where(up < down, hi, lo))
    return torch.where(v < 0, -grid[take], grid[take])


def _grid(fmt):
    if fmt == "e2m1":
        v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:  # E4M3: codes 0 to 126 in order
        v = [(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_quantize(x, fmt, g):
    n = BLOCK[fmt]
    b = x.reshape(-1, n)
    amax = b.abs().max(dim=1, keepdim=True).values
    if fmt == "nvfp4":
        s = _nearest(amax / 6 / g, _grid("e4m3"))
        q = _nearest(torch.where(s > 0, b / (s * g).clamp(min=1e-300), 0.0), _grid("e2m1"))
    else:
        top = 448.0 if fmt == "mxfp8" else 6.0
        s = torch.exp2(torch.ceil(torch.log2((amax / top).clamp(min=2.0 ** -127))))
        s = torch.where(amax > top * s, 2 * s, torch.where((2 * amax <= top * s) & (s > 2.0 ** -127), s / 2, s))
        q = _nearest(b / s, _grid("e4m3" if fmt == "mxfp8" else "e2m1"))
    return q.reshape(x.shape), s.reshape(x.shape[0], -1)


def _exact_values(o):
    """What an operand's bytes stand for, row by row and scale by scale."""
    r = torch.arange(o["rows"], device="cuda").unsqueeze(1)
    n = o["K"] // BLOCK[o["fmt"]]
    j = torch.arange(n, device="cuda").unsqueeze(0)
    at = ((r // 128) * ((n + 3) // 4) + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4
    s = o["scales"][at].double()
    sign = lambda c, bit: 1.0 - 2.0 * (c >= bit).double()  # noqa: E731
    if o["fmt"] == "nvfp4":
        s = _grid("e4m3")[s.long()]
    else:
        s = torch.exp2(s - 127)
    if o["fmt"] == "mxfp8":
        v = _grid("e4m3")[(o["codes"] % 128).long()] * sign(o["codes"], 128)
    else:
        c = torch.empty(o["rows"], o["K"], dtype=torch.uint8, device="cuda")
        c[:, 0::2], c[:, 1::2] = o["codes"] % 16, o["codes"] // 16
        v = _grid("e2m1")[(c % 8).long()] * sign(c, 8)
    v = v * s.repeat_interleave(BLOCK[o["fmt"]], dim=1)
    return v if o["tensor_scale"] is None else v * o["tensor_scale"].double()


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm":
        s = c["xv"].double()
        if c["res"] != "none":
            s = s * c["beta"] + c["rv"].double() * c["alpha"]
        y = s / torch.sqrt(torch.square(s).sum(1, keepdim=True) / c["H"] + 1e-6) * c["gamma"].double()
        out = {"out": y}
        if c["res"] != "none":
            out["residual"] = s
        if c["q"]:
            out["elements"], sc = _exact_quantize(y, "mxfp8", None)
            if c["layout"] == "tiled":
                r, n = sc.shape
                t = torch.full(((r + 127) // 128 * ((n + 3) // 4) * 512,), 2.0 ** -127, dtype=torch.float64, device="cuda")
                i, j = torch.arange(r, device="cuda").unsqueeze(1), torch.arange(n, device="cuda").unsqueeze(0)
                t[((i // 128) * ((n + 3) // 4) + j // 4) * 512 + (i % 32) * 16 + (i // 32 % 4) * 4 + j % 4] = sc
                sc = t
            out["scales"] = sc
        return out
    if c["op"] == "quantize":
        x = c["xv"].double()
        g = None
        if c["fmt"] == "nvfp4":
            g = torch.exp2(torch.ceil(torch.log2(x.abs().max() / 2688))) if c["dynamic"] else c["ts"][0].double()
        q, s = _exact_quantize(x, c["fmt"], g)
        v = q * s.repeat_interleave(BLOCK[c["fmt"]], dim=1)
        return {"values": v} if g is None else {"values": v * g, "tensor_scale": g.reshape(1)}
    if c["op"] == "product":
        return {"out": _exact_values(c["av"]) @ _exact_values(c["wv"]).t()}
    # one expert after another, the least index first among equals
    l = c["lv"].double()
    live = torch.isfinite(l)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        p = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    key = p + (0.0 if c["bv"] is None else c["bv"].double())
    key = torch.where(live, key, -math.inf)
    T, E = l.shape
    per, far = E // c["groups"], torch.arange(E, device="cuda")
    if c["groups"] > c["keep"]:
        left, total = key.clone(), torch.zeros(T, c["groups"], dtype=torch.float64, device="cuda")
        total[(~live).reshape(T, c["groups"], per).all(2)] = -math.inf
        for _ in range(min(c["gtop"], per)):
            best = left.reshape(T, c["groups"], per).max(2)
            total += torch.where(torch.isfinite(best.values), best.values, 0.0)
            left.reshape(T, c["groups"], per).scatter_(2, best.indices.unsqueeze(2), -math.inf)
        kept = torch.zeros(T, c["groups"], dtype=torch.bool, device="cuda")
        for _ in range(c["keep"]):
            top = total.max(1, keepdim=True).values
            at = torch.where(total == top, far[:c["groups"]], E).min(1, keepdim=True).values
            kept.scatter_(1, at, True)
            total = total.scatter(1, at, math.nan).nan_to_num(nan=-math.inf, neginf=-math.inf)
        key = torch.where(kept.repeat_interleave(per, dim=1), key, -math.inf)
    ws = []
    for _ in range(c["k"]):
        top = key.max(1, keepdim=True).values
        at = torch.where(key == top, far, E).min(1, keepdim=True).values
        ws.append(torch.where(torch.isfinite(top), p.gather(1, at), 0.0))
        key = key.scatter(1, at, -math.inf)
    w = torch.cat(ws, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return {"idx": None, "w": w}
