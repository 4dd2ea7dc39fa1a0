"""The handle-free operators (include/beam_ops.h, ops.py) on the GPU against
the 64-bit references in ops_ref.py: formats and layouts bit for bit, norms
and products within bounds counted in roundings, routing choices exactly; and
a run of them together with the MoE block."""
import math

import numpy as np
import pytest
import torch

import ops_ref as R
from group_limited_routing_sigmoid_b200 import ops
from group_limited_routing_sigmoid_b200.build import build

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half a step relative to a value just above a power of two: eps / 2
HALF = {t: torch.finfo(t).eps / 2 for t in HALF}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}   # half the least subnormal


def setup_module(_):
    build(quiet=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(rows, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * scale
    x[:, torch.rand(K, generator=g) < 0.05] *= 20
    return x.to(dtype).cuda()


def strided(x, pad):
    """The same values in rows that lie `pad` elements further apart, off any vector alignment."""
    b = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device=x.device)
    b[:, 1:1 + x.shape[1]] = x
    return b[:, 1:1 + x.shape[1]]


# --- formats ---------------------------------------------------------------------

def check_quantize(x, fmt, layout, g=None):
    q = ops.mx_quantize(x, fmt, layout, None if g is None else torch.tensor([g], device="cuda"))
    e, sb = R.quantize(f64(x), fmt, g)
    rows, K = x.shape
    got_sb = q.scales.cpu().numpy()
    np.testing.assert_array_equal(got_sb, sb.astype(np.uint8) if layout == "rows" else R.tile(sb))
    got = q.codes.cpu().numpy()
    # equal as values: a zero may carry either sign
    np.testing.assert_array_equal(R.elements(got, fmt), e)
    return q, e, sb


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("rows,K,layout,pad", [(1, 32, "rows", 0), (1, 32, "tiled", 0), (3, 96, "rows", 0), (5, 288, "tiled", 0),
                                               (129, 64, "tiled", 3), (130, 544, "rows", 5), (64, 1024, "tiled", 0),
                                               (300, 2592, "tiled", 0)])
def test_quantize(fmt, dtype, rows, K, layout, pad):
    x = rand(rows, K, dtype, rows + K)
    if pad:
        x = strided(x, pad)
    g = {"nvfp4": R.tensor_scale(f64(x))}.get(fmt)
    check_quantize(x, fmt, layout, g)


@pytest.mark.parametrize("g", [0.013, 1.0 / 3, 2.0 ** -9, 7e-7, 1e4, 2.0 ** -112, 2.0 ** 112])
def test_quantize_under_given_tensor_scales(g):
    # scales that saturate the block scale, leave it at zero, and lie between
    check_quantize(rand(40, 256, torch.float32, 3), "nvfp4", "rows", g)
    check_quantize(rand(40, 256, torch.bfloat16, 4, 2.0 ** -60), "nvfp4", "rows", g)


@pytest.mark.parametrize("g", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** -113, 2.0 ** 113])
def test_tensor_scale_out_of_range_reads_back_as_nan(g):
    q = ops.mx_quantize(rand(2, 64, torch.bfloat16, 0), "nvfp4", tensor_scale=torch.tensor([g], device="cuda"))
    assert (q.scales == 0x7f).all() and (q.codes == 0).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_edges(fmt, dtype):
    """Blocks of zeros, of one value, of ties, of the type's extremes and subnormals, of infinities and NaN."""
    big = torch.finfo(dtype).max
    rows = [torch.zeros(32), torch.full((32,), -0.0), torch.full((32,), 6.0), torch.full((32,), 448.0),
            torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4),
            torch.tensor([0.3125, 0.9375, 1.5625, 2.1875, 3.125, 4.375, 6.25, 7.5] * 4), torch.full((32,), big),
            torch.full((32,), 2.0 ** -126), torch.full((32,), 2.0 ** -133), torch.full((32,), 2.0 ** -100),
            torch.tensor([float("inf")] + [1.0] * 31), torch.tensor([1.0] * 31 + [float("nan")]),
            torch.tensor([-float("inf")] * 32), torch.arange(32.0) - 15.5, 2.0 ** -torch.arange(32.0)]
    x = torch.stack(rows).to(dtype).cuda()
    for layout in ("rows", "tiled"):
        if fmt == "nvfp4":
            for g in (2.0 ** -9, 1.0, 2.0 ** -100, 2.0 ** 110):
                check_quantize(x, fmt, layout, g)
        else:
            check_quantize(x, fmt, layout)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (0, 16, 0), (3, 7, 0), (77, 513, 2), (300, 1000, 0), (1, 100000, 0)])
def test_tensor_scale(dtype, rows, K, pad):
    x = rand(rows, K, dtype, K, 0.3)
    if pad:
        x = strided(x, pad)
    assert float(ops.mx_tensor_scale(x)) == R.tensor_scale(f64(x))


def test_tensor_scale_edges():
    for v in (0.0, 2688.0, 2688.0 * (1 + 2.0 ** -7), 2.0 ** -101, 2.0 ** -126, 3e38):
        x = torch.full((1, 8), v, device="cuda")
        assert float(ops.mx_tensor_scale(x)) == R.tensor_scale(f64(x)), v
    x = torch.tensor([[1.0, float("nan"), float("inf"), -5.0]], device="cuda")
    assert float(ops.mx_tensor_scale(x)) == R.tensor_scale(np.array([[5.0]]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt,layout,rows,K,pad", [("nvfp4", "rows", 5, 48, 0), ("nvfp4", "tiled", 131, 320, 0),
                                                   ("mxfp4", "rows", 40, 96, 0), ("mxfp4", "tiled", 3, 32, 5),
                                                   ("mxfp8", "rows", 7, 544, 3), ("mxfp8", "tiled", 200, 160, 0)])
def test_dequantize(fmt, layout, rows, K, pad, dtype):
    rng = np.random.default_rng(rows)
    # every code; scales around one, so that no type overflows
    c = rng.integers(0, 256, (rows, K if fmt == "mxfp8" else K // 2)).astype(np.uint8)
    if fmt == "mxfp8":
        c[(c & 127) == 127] = 0
    sb = (rng.integers(0, 0x50, (rows, K // R.BLOCK[fmt])) if fmt == "nvfp4"
          else rng.integers(117, 131, (rows, K // R.BLOCK[fmt]))).astype(np.uint8)
    g = 0.37 if fmt == "nvfp4" else None
    q = ops.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(sb if layout == "rows" else R.tile(sb)).cuda(), fmt,
                     layout, rows, K, None if g is None else torch.tensor([g], device="cuda"))
    out = None
    if pad:
        out = torch.full((rows, K + pad), 9.0, dtype=dtype, device="cuda")[:, :K]
    got = ops.mx_dequantize(q, dtype, out)
    want = R.values(R.elements(c, fmt), sb, fmt, 1.0 if g is None else float(np.float32(g)))
    # element x block scale is exact in FP32, one product with g, one rounding
    want32 = want.astype(np.float32)
    np.testing.assert_array_equal(got.float().cpu().numpy(), torch.from_numpy(want32).to(dtype).float().numpy())
    if pad:
        assert (out._base[:, K:] == 9.0).all()


def test_dequantize_nan_scales_and_the_least_power():
    q = ops.MxTensor(torch.full((1, 32), 0x22, dtype=torch.uint8, device="cuda"),
                     torch.tensor([[255, 0]], dtype=torch.uint8, device="cuda"), "mxfp4", "rows", 1, 64)
    v = ops.mx_dequantize(q, torch.float32)
    assert v[0, :32].isnan().all() and (v[0, 32:] == 2.0 ** -127).all()


@pytest.mark.parametrize("fmt,rows,K", [("nvfp4", 1, 16), ("nvfp4", 130, 208), ("mxfp4", 64, 96), ("mxfp8", 257, 1056)])
def test_tile_scales(fmt, rows, K):
    sb = np.random.default_rng(K).integers(0, 256, (rows, K // R.BLOCK[fmt])).astype(np.uint8)
    codes = torch.zeros(rows, K if fmt == "mxfp8" else K // 2, dtype=torch.uint8, device="cuda")
    q = ops.mx_tile_scales(ops.MxTensor(codes, torch.from_numpy(sb).cuda(), fmt, "rows", rows, K))
    np.testing.assert_array_equal(q.scales.cpu().numpy(), R.tile(sb))


def test_flattened_rows_past_32_bits():
    """More scales and codes than 31-bit offsets hold: the last rows come out as they do alone."""
    rows, K = 70000, 32768        # 2.3e9 elements
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand(3, K, torch.bfloat16, 1)
    g = torch.tensor([2.0 ** -5], device="cuda")
    for layout in ("rows", "tiled"):
        q = ops.mx_quantize(x, "nvfp4", layout, g)
        one = ops.mx_quantize(x[-3:], "nvfp4", "rows", g)
        assert torch.equal(q.codes[-3:], one.codes)
        v = ops.mx_dequantize(q)
        assert torch.equal(v[-3:], ops.mx_dequantize(one)) and not v[:-3].any()
        del q, v


# --- norm --------------------------------------------------------------------------

def norm_ref(x, r, gamma, alpha, beta, eps):
    a, b = float(np.float32(alpha)), float(np.float32(beta))
    s = b * f64(x) + (0.0 if r is None else a * f64(r))
    scale = 1 / np.sqrt((s * s).mean(1, keepdims=True) + float(np.float32(eps)))
    return s, s * scale * f64(gamma)


def check_norm(x, r, gamma, dtype, quantize, layout, alpha=1.0, beta=1.0, eps=1e-6, **kw):
    res = ops.rms_norm(x, gamma, residual=r, alpha=alpha, beta=beta, eps=eps, dtype=dtype, quantize=quantize, layout=layout, **kw)
    s, y = norm_ref(x, r, gamma, alpha, beta, eps)
    H = x.shape[1]
    u = 2.0 ** -24
    # s: two products and a sum, each rounded once
    ds = 2 * u * (np.abs(float(beta) * f64(x)) + (0 if r is None else np.abs(float(alpha) * f64(r))))
    if r is not None:
        got = f64(res.residual)
        t = res.residual.dtype
        assert np.all(np.abs(got - s) <= HALF[t] * (np.abs(s) + ds) + ds + TINY[t])
    # the mean square: a chain of at most 32 x 8 fused terms and 10 joins; its
    # square root, division and two products; half the mean's relative error
    # reaches y.  Cancellation in s enters through ds.
    rel = (0.5 * (32 * 8 + 10 + 2) + 5) * u
    ms = np.sqrt((s * s).mean(1, keepdims=True))
    ds_row = np.sqrt((ds * ds).mean(1, keepdims=True)) / np.maximum(ms, 1e-300)
    scale = np.abs(f64(gamma)) / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    dy = np.abs(y) * (rel + ds_row) + ds * scale
    if res.out is not None:
        assert res.out.dtype == dtype
        assert np.all(np.abs(f64(res.out) - y) <= HALF[dtype] * (np.abs(y) + dy) + dy + TINY[dtype])
    if quantize:
        q = res.quantized
        c = q.codes.cpu().numpy()
        T = x.shape[0]
        n = H // 32
        sb = q.scales.cpu().numpy()
        if layout == "tiled":
            t = sb.reshape((T + 127) // 128, (n + 3) // 4, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1, (n + 3) // 4 * 4)
            assert not t[T:].any() and not t[:, n:].any()
            sb = t[:T, :n]
        amax, damax = (np.abs(y).reshape(T, n, 32).max(-1), dy.reshape(T, n, 32).max(-1))
        k = sb.astype(int) - 127
        assert np.all(k >= R.pow2_exponent(amax - damax, 448.0)) and np.all(k <= R.pow2_exponent(amax + damax, 448.0))
        p = np.repeat(2.0 ** k.astype(float), 32, axis=1)
        v = R.elements(c, "mxfp8") * p
        # half a step of E4M3: 2^-4 of the value, 2^-10 where subnormal; a
        # value within dy above the top saturates
        assert np.all(np.abs(v - y) <= 2.0 ** -4 * (np.abs(y) + dy) + 2.0 ** -10 * p + dy)
        # and to nearest: no closer neighbour by more than dy
        e, _ = R.quantize(f64(res.out) if dtype == torch.float32 and res.out is not None else y, "mxfp8")
        if dtype == torch.float32 and res.out is not None:   # the FP32 rows themselves were quantised
            np.testing.assert_array_equal(R.elements(c, "mxfp8"), e)
    return res


TYPES = [(torch.bfloat16, None), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, None),
         (torch.float16, torch.float32), (torch.float16, torch.float16), (torch.float32, None), (torch.float32, torch.float32)]


@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (3, 7, 0), (2, 8, 0), (5, 264, 0), (4, 1000, 3), (3, 1032, 0), (7, 5120, 0),
                                     (2, 2563, 0), (2, 8200, 0), (1, 16392, 0), (1, 32768, 0), (2, 9001, 0)])
def test_norm(xt, rt, T, H, pad):
    g = torch.Generator().manual_seed(H)
    x, gamma = rand(T, H, xt, H), (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    r = None if rt is None else rand(T, H, rt, H + 1)
    if pad:
        x, r = strided(x, pad), None if r is None else strided(r, pad)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        check_norm(x, r, gamma, dtype, None, "rows", math.sqrt(19 / 20), math.sqrt(1 / 20))


@pytest.mark.parametrize("T,H,pad", [(1, 32, 0), (3, 96, 0), (130, 160, 0), (129, 5120, 0), (64, 2592, 0), (5, 1056, 1),
                                     (2, 8224, 0), (1, 32768, 0), (9, 9216, 3)])
@pytest.mark.parametrize("layout", ["rows", "tiled"])
def test_norm_mxfp8(T, H, pad, layout):
    x, r, gamma = rand(T, H, torch.bfloat16, H), rand(T, H, torch.float32, H + 1), torch.ones(H, device="cuda") * 1.25
    if pad:
        x = strided(x, pad)
    check_norm(x, r, gamma, torch.float32, "mxfp8", layout)
    a = check_norm(x, r, gamma, torch.bfloat16, "mxfp8", layout)
    b = check_norm(x, r, gamma, torch.bfloat16, "mxfp8", layout, want_out=False)
    assert b.out is None and torch.equal(a.quantized.codes, b.quantized.codes) and torch.equal(a.quantized.scales, b.quantized.scales)


def test_norm_in_place_and_given_buffers():
    x, r, gamma = rand(9, 512, torch.bfloat16, 1), rand(9, 512, torch.float32, 2), torch.ones(512, device="cuda")
    want = ops.rms_norm(x, gamma, residual=r, quantize="mxfp8")
    r2, out = r.clone(), torch.empty(9, 512, dtype=torch.bfloat16, device="cuda")
    q = ops.MxTensor(torch.zeros_like(want.quantized.codes), torch.zeros_like(want.quantized.scales), "mxfp8", "tiled", 9, 512)
    got = ops.rms_norm(x, gamma, residual=r2, residual_out=r2, out=out, quantize="mxfp8", quantized=q)
    assert got.residual is r2 and got.out is out
    assert torch.equal(r2, want.residual) and torch.equal(out, want.out)
    assert torch.equal(q.codes, want.quantized.codes) and torch.equal(q.scales, want.quantized.scales)


def test_norm_rows_of_zeros_infinities_and_nan():
    x = torch.zeros(5, 64, device="cuda")
    x[1] = 1.0
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 2e19                       # its square sum overflows FP32: the row is zero
    res = ops.rms_norm(x, torch.ones(64, device="cuda"), dtype=torch.float32, quantize="mxfp8", layout="rows")
    assert (res.out[0] == 0).all() and (res.quantized.scales[0] == 0).all()
    np.testing.assert_allclose(res.out[1].cpu(), 1.0, rtol=1e-6)
    assert res.out[2].isnan().all() and (res.quantized.scales[2] == 255).all() and (res.quantized.codes[2] == 0).all()
    assert res.out[3, 5].isnan() and (res.out[3, :5] == 0).all()
    assert res.quantized.scales[3, 0] == 255 and res.quantized.scales[3, 1] == 0
    assert (res.out[4] == 0).all()


# --- product -----------------------------------------------------------------------

PAIRS = [("nvfp4", "nvfp4"), ("mxfp4", "mxfp4"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp8")]


def operand(rows, K, fmt, seed, spread=3):
    """Random codes under scales within 2^spread of each other -> (MxTensor, values)."""
    rng = np.random.default_rng(seed)
    e = (R.E4M3 if fmt == "mxfp8" else R.E2M1)[rng.integers(0, 120 if fmt == "mxfp8" else 8, (rows, K))]
    e = e * rng.choice([-1.0, 1.0], (rows, K))
    n = K // R.BLOCK[fmt]
    sb = (rng.integers(0x30, 0x30 + 8 * spread, (rows, n)) if fmt == "nvfp4" else rng.integers(125, 125 + spread, (rows, n))).astype(np.uint8)
    g = 2.0 ** -3 if fmt == "nvfp4" else None
    q = ops.MxTensor(torch.from_numpy(R.codes(e, fmt)).cuda(), torch.from_numpy(R.tile(sb)).cuda(), fmt, "tiled", rows, K,
                     None if g is None else torch.tensor([g], device="cuda"))
    return q, R.values(e, sb, fmt, 1.0 if g is None else g)


def check_product(y, dtype, a, w, K):
    """FP32 sums: K products, each exact, joined in any order with at most one
    rounding (or truncation, two half-steps) a join; then one rounding."""
    want, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    tol = HALF[dtype] * np.abs(want) + (K / 32 + 40) * 2.0 ** -23 * mag + TINY[dtype]
    err = np.abs(f64(y) - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("af,wf", PAIRS)
@pytest.mark.parametrize("T,N,K", [(1, 1, 128), (1, 130, 256), (5, 128, 384), (16, 300, 1024), (17, 513, 640), (33, 64, 2048),
                                   (64, 1000, 512), (100, 257, 1152), (128, 128, 128), (129, 129, 256), (300, 7, 384),
                                   (200, 520, 1280), (513, 261, 256)])
def test_product(af, wf, T, N, K):
    a, av = operand(T, K, af, T)
    w, wv = operand(N, K, wf, N + 1000)
    for dtype in (torch.bfloat16, torch.float32):
        y = ops.mx_matmul(a, w, dtype)
        assert ops.ops_status() == 0
        check_product(y, dtype, av, wv, K)


@pytest.mark.parametrize("af,wf", [PAIRS[0], PAIRS[1]])
@pytest.mark.parametrize("T,N,K", [(3, 40, 64), (70, 200, 192), (140, 150, 320), (2, 3, 8256)])
def test_product_at_odd_multiples_of_64(af, wf, T, N, K):
    a, av = operand(T, K, af, 1)
    w, wv = operand(N, K, wf, 2)
    y = ops.mx_matmul(a, w, torch.float16)
    assert ops.ops_status() == 0
    check_product(y, torch.float16, av, wv, K)


@pytest.mark.parametrize("af,wf", PAIRS)
def test_product_of_whole_numbers_is_exact(af, wf):
    """Elements of 0, 1, 2 under scales of 1 and 2: every sum is a whole number below 2^24, so FP32 holds it exactly
    whatever the order, and each misplaced row, column, scale or K step shows."""
    for T, N, K in ((40, 300, 1024), (260, 384, 512), (3, 20, 4096)):
        rng = np.random.default_rng(T)
        ops_, vals = [], []
        for rows, fmt in ((T, af), (N, wf)):
            e = rng.integers(0, 3, (rows, K)).astype(float) * rng.choice([-1.0, 1.0], (rows, K))
            one = 0x38 if fmt == "nvfp4" else 127
            up = rng.integers(0, 2, (rows, K // R.BLOCK[fmt]))
            sb = (one + up * (8 if fmt == "nvfp4" else 1)).astype(np.uint8)
            ops_.append(ops.MxTensor(torch.from_numpy(R.codes(e, fmt)).cuda(), torch.from_numpy(R.tile(sb)).cuda(), fmt, "tiled", rows, K))
            vals.append(R.values(e, sb, fmt))
        y = ops.mx_matmul(*ops_, torch.float32)
        assert ops.ops_status() == 0
        np.testing.assert_array_equal(f64(y), vals[0] @ vals[1].T)


@pytest.mark.parametrize("T,N,K", [(8, 5120, 2560), (640, 5123, 768), (1021, 2563, 512), (2500, 1300, 256)])
def test_product_larger(T, N, K):
    for af, wf in (PAIRS[0], PAIRS[2]):
        a, av = operand(T, K, af, 5)
        w, wv = operand(N, K, wf, 6)
        out = torch.full((T, N + 5), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.mx_matmul(a, w, out=out[:, :N])
        assert ops.ops_status() == 0
        check_product(out[:, :N], torch.bfloat16, av, wv, K)
        assert (out[:, N:] == 7.0).all()          # what lies behind the rows stays
        again = ops.mx_matmul(a, w)
        assert torch.equal(again, out[:, :N])     # and the same bits every time


def test_product_nan_scales_stay_in_their_row():
    a, av = operand(6, 256, "mxfp8", 1)
    w, wv = operand(70, 256, "mxfp4", 2)
    sa = a.scales.clone()
    sa[(2 % 32) * 16] = 255                        # row 2, first block
    y = ops.mx_matmul(a._replace(scales=sa), w, torch.float32)
    assert y[2].isnan().all() and not y[[0, 1, 3, 4, 5]].isnan().any()
    assert ops.ops_status() == 0


# --- routing -----------------------------------------------------------------------

def check_route(l, k, score, bias=None, G=1, keep=1, gtop=2, renorm=True, scale=1.0):
    idx, w = ops.route_scores(l, k, score=score, bias=bias, n_group=G, topk_group=keep, group_top=gtop, renormalize=renorm, scale=scale)
    ri, rw = R.route(f64(l), k, score, None if bias is None else bias.cpu().numpy(), G, keep, gtop, renorm, scale)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    got = f64(w)
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    ok = ~np.isnan(rw)
    # exponential 2 ulps, sums of up to 38 joins, division, product
    np.testing.assert_allclose(got[ok], rw[ok], rtol=48 * 2.0 ** -23, atol=2.0 ** -149)
    return idx, w


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,keep,gtop", [(1, 1, 1, 1, 1, 2), (3, 2, 2, 1, 1, 2), (40, 8, 2, 1, 1, 1), (64, 60, 4, 1, 1, 1),
                                               (200, 64, 6, 8, 3, 1), (200, 256, 8, 8, 4, 2), (50, 317, 12, 1, 1, 2),
                                               (30, 512, 32, 32, 16, 2), (20, 1024, 8, 4, 2, 2), (33, 160, 8, 10, 3, 2),
                                               (9, 96, 32, 4, 4, 2), (300, 32, 8, 32, 8, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("coarse", [False, True])
def test_route(score, T, E, k, G, keep, gtop, with_bias, coarse):
    g = torch.Generator().manual_seed(T * E)
    l = torch.randn(T, E, generator=g) * 2
    if coarse:
        l = l.to(torch.bfloat16).float()
    l = l.cuda()
    bias = (torch.randn(E, generator=g) * 0.05).cuda() if with_bias else None
    for renorm in (False, True):
        check_route(l, k, score, bias, G, keep, gtop, renorm, 2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2)])
def test_route_masked_rows_and_experts(score, G, keep):
    g = torch.Generator().manual_seed(1)
    l = torch.randn(40, 64, generator=g)
    l[:, 5:20] = -math.inf
    l[3] = -math.inf                                   # nothing left
    l[4, 1:] = -math.inf                               # one left
    l[5, :32] = -math.inf
    l[6, 7] = math.nan
    l[7, 2] = math.inf
    l[8] = torch.finfo(torch.float32).min              # the type's lowest value is no mask
    l[9, :60] = torch.finfo(torch.float32).min
    l[10] = -200.0                                     # sigmoids that FP32 cannot hold
    l[10, 3] = -150.0
    l[11] = 60.0                                       # sigmoids that saturate
    l = l.cuda()
    for bias in (None, torch.linspace(-0.1, 0.1, 64).cuda()):
        for renorm in (False, True):
            check_route(l, 8, score, bias, G, keep, 2, renorm)
    bias = torch.zeros(64)
    bias[[0, 33]] = -math.inf
    bias[[40, 41]] = math.inf
    check_route(l, 8, score, bias.cuda(), G, keep)
    bias[2] = math.nan
    check_route(l, 8, score, bias.cuda(), G, keep)


def test_route_near_ties_are_decided_exactly():
    """Keys that differ by less than FP32 shows: logits one ulp apart under biases that nearly undo it."""
    g = torch.Generator().manual_seed(3)
    base = torch.randn(500, 1, generator=g)
    l = (base + torch.randn(500, 64, generator=g) * 3e-7).cuda()
    check_route(l, 8, "sigmoid")
    check_route(l, 8, "softmax", None, 8, 3, 2)
    bias = (torch.randn(64, generator=g) * 2e-8).cuda()
    check_route(l, 8, "sigmoid", bias)
    check_route(l, 8, "sigmoid", bias, 8, 3, 2)
    check_route(l, 8, "softmax", bias, 8, 3, 1)
    same = torch.zeros(10, 64, device="cuda")
    check_route(same, 8, "softmax")
    check_route(same, 8, "sigmoid", torch.zeros(64, device="cuda"), 8, 4)


def test_route_strided_logits_and_given_outputs():
    l = torch.randn(30, 70, generator=torch.Generator().manual_seed(0)).cuda()
    idx, w = ops.route_scores(l[:, 3:67], 5, score="softmax")
    want = ops.route_scores(l[:, 3:67].contiguous(), 5, score="softmax")
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    i2, w2 = torch.full((31, 5), 9, dtype=torch.int32, device="cuda"), torch.full((31, 5), 9.0, device="cuda")
    ops.route_scores(l[:, 3:67], 5, score="softmax", idx=i2[:30], w=w2[:30])
    assert torch.equal(i2[:30], idx) and (i2[30] == 9).all() and (w2[30] == 9).all()


def test_route_matches_the_handles_router():
    """The handle's routing from logits (beam_moe_route_logits) and this one agree on the Beam configuration."""
    import dataclasses

    from group_limited_routing_sigmoid_b200 import workloads as W
    from group_limited_routing_sigmoid_b200.binding import BeamMoE

    wl = dataclasses.replace(W.WORKLOADS["decode"], inter=128)
    g = W.generator(wl, "cuda")
    d = W.make_weights(wl, "cuda", g)
    d.update(W.make_tokens(wl, "cuda", g, T=300))
    moe = BeamMoE.from_workload(wl, d, max_tokens=300)
    l = moe.router_logits(d["x"])
    idx, w = moe.route_logits(l)
    i2, w2 = ops.route_scores(l, wl.top_k, bias=d["bias"], n_group=wl.n_group, topk_group=wl.topk_group)
    same = (idx == i2).all(1)
    assert same.float().mean() > 0.99              # the handle decides near-ties in FP32
    np.testing.assert_allclose(w2[same].cpu(), w[same].cpu(), rtol=1e-5)
    moe.close()


# --- together, streams, graphs ------------------------------------------------------

def test_a_layer_of_them():
    """Stream update and norm to MXFP8, a 4-bit gate and up, SwiGLU, NVFP4 tokens, a 4-bit down, against 64 bits step by step."""
    T, H, I = 37, 512, 1024
    x, r, gamma = rand(T, H, torch.bfloat16, 1, 0.1), rand(T, H, torch.float32, 2), torch.ones(H, device="cuda")
    wg, wu = (ops.mx_quantize(rand(I, H, torch.bfloat16, s, 0.05), "mxfp4", "tiled") for s in (3, 4))
    wd = ops.mx_quantize(rand(H, I, torch.bfloat16, 5, 0.05), "nvfp4", "tiled")
    n = ops.rms_norm(x, gamma, residual=r, quantize="mxfp8", want_out=False)
    gate, up = (ops.mx_matmul(n.quantized, w, torch.float32) for w in (wg, wu))
    nv = f64(ops.mx_dequantize(n.quantized, torch.float32))
    for y, w in ((gate, wg), (up, wu)):
        check_product(y, torch.float32, nv, f64(ops.mx_dequantize(w, torch.float32)), H)
    h = ops.mx_quantize(torch.nn.functional.silu(gate) * up, "nvfp4", "tiled")
    y = ops.mx_matmul(h, wd, torch.float32)
    check_product(y, torch.float32, f64(ops.mx_dequantize(h, torch.float32)), f64(ops.mx_dequantize(wd, torch.float32)), I)
    assert ops.ops_status() == 0


def test_quantized_weights_run_the_nvfp4_block():
    """Weights made here, in rows, feed BeamMoE.nvfp4; the block agrees with the oracle on what they stand for."""
    from group_limited_routing_sigmoid_b200 import workloads as W
    from group_limited_routing_sigmoid_b200.binding import BeamMoE
    from parity import check_block

    wl = W.WORKLOADS["tiny_nvfp4"]
    d = W.make_inputs(wl, "cuda")
    E, I, H = wl.n_experts, wl.inter, wl.hidden
    for i, (n, R_, K) in enumerate((("gate", I, H), ("up", I, H), ("down", H, I))):
        q = ops.mx_quantize(rand(E * R_, K, torch.bfloat16, 10 + i, 0.02), "nvfp4", "rows")
        d[n + "_codes"], d[n + "_scales"] = q.codes.view(E, R_, K // 2), q.scales.view(E, R_, K // 16)
        d[n + "_global"] = float(q.tensor_scale)
    moe = BeamMoE.from_workload(wl, d)
    rep = check_block(wl, d, moe)
    moe.close()
    assert rep.ok(), rep


def run_all(x, r, gamma, w, l, stream=None):
    n = ops.rms_norm(x, gamma, residual=r, quantize="mxfp8", stream=stream)
    y = ops.mx_matmul(n.quantized, w, stream=stream)
    q = ops.mx_quantize(y, "nvfp4", "tiled", stream=stream)
    v = ops.mx_dequantize(q, stream=stream)
    idx, wt = ops.route_scores(l, 4, score="softmax", stream=stream)
    return [n.out, n.residual, n.quantized.codes, n.quantized.scales, y, q.codes, q.scales, q.tensor_scale, v, idx, wt]


def run_inputs(seed=0, T=70):
    w = ops.mx_quantize(rand(384, 512, torch.bfloat16, 7, 0.05), "mxfp4", "tiled")
    return (rand(T, 512, torch.bfloat16, seed), rand(T, 512, torch.float32, seed + 1), torch.ones(512, device="cuda"), w,
            rand(T, 60, torch.float32, seed + 2))


def test_other_streams_and_two_at_once():
    args = [run_inputs(s) for s in (0, 50)]
    want = [run_all(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run_all(*a, stream=s) for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            assert torch.equal(x, y)
    raw = run_all(*args[0], stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(raw, want[0]))


def test_captured_and_replayed():
    args = run_inputs()
    want = [t.clone() for t in run_all(*args)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run_all(*args)
    other = run_inputs(9)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    args[0].copy_(other[0])                           # new tokens in the captured buffers
    g.replay()
    torch.cuda.synchronize()
    want = run_all(args[0], *args[1:])
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_bindings_refuse_mismatches():
    x = rand(4, 64, torch.bfloat16, 0)
    q = ops.mx_quantize(x, "mxfp4", "rows")
    with pytest.raises(ValueError):
        ops.mx_matmul(q, q)                            # scales not tiled
    t = ops.mx_tile_scales(q)
    with pytest.raises(ops.BeamMoEError):
        ops.mx_matmul(t, ops.mx_quantize(x, "mxfp8", "tiled"))
    with pytest.raises(TypeError):
        ops.mx_matmul(t, t, out=torch.empty(4, 5, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        ops.mx_quantize(x.t(), "mxfp4")
    with pytest.raises(TypeError):
        ops.mx_quantize(x[:1].expand(4, 64), "mxfp4")
    with pytest.raises(ops.BeamMoEError):
        ops.mx_quantize(rand(4, 48, torch.bfloat16, 0), "mxfp8")
    with pytest.raises(ValueError):
        ops.mx_quantize(x, "mxfp4", tensor_scale=torch.ones(1, device="cuda"))
    with pytest.raises(TypeError):
        ops.rms_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        ops.rms_norm(x, torch.ones(64, device="cuda"), residual=x.half())
    with pytest.raises(ops.BeamMoEError):
        ops.route_scores(torch.zeros(2, 8, device="cuda"), 9)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(64, 1, 1), (256, 8, 4), (480, 6, 2), (1000, 1, 1)])
def test_route_many_experts_of_one_lane_and_ties_at_the_border(score, E, G, keep):
    """The best experts side by side (one lane's whole list), and equal keys around the last place with a third one near."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn(24, E, generator=g)
    l[:8] = l[:8].sort(dim=1, descending=True).values
    l[8:12] = l[8:12].sort(dim=1).values
    l[12:16, :40] = 3.0                                # equal, more than are chosen
    l[16:20, 5:12] = 3.0
    l[20:22, 7:15] = 3.0
    l[20:22, 15] = 3.0 + 2.0 ** -22                    # one ulp above the equal ones
    l[22, :] = torch.linspace(2.0, 2.0 + 1e-5, E)
    l = l.cuda()
    bias = torch.randn(E, generator=g).cuda() * 1e-8
    for k in (1, 8, 32):
        for b in (None, torch.zeros(E, device="cuda"), bias):
            for renorm in (False, True):
                check_route(l, k, score, b, G, keep, 2, renorm)


def test_route_long_batch_strided_rows():
    """More rows than warps in flight, in rows off any vector alignment, against the same rows alone."""
    l = torch.randn(9000, 256, generator=torch.Generator().manual_seed(2)).cuda()
    bias = (torch.randn(256, generator=torch.Generator().manual_seed(3)) * 0.05).cuda()
    want = ops.route_scores(l, 8, bias=bias, n_group=8, topk_group=4)
    got = ops.route_scores(strided(l, 3), 8, bias=bias, n_group=8, topk_group=4)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    some = ops.route_scores(l[8500:8600], 8, bias=bias, n_group=8, topk_group=4)
    assert torch.equal(some[0], want[0][8500:8600]) and torch.equal(some[1], want[1][8500:8600])
    check_route(l[:700], 8, "sigmoid", bias, 8, 4)


@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 9), (3, 255), (5, 261), (4, 1031), (3, 2563), (2, 8191), (2, 9001)])
def test_norm_writes_its_rows_alone(xt, rt, T, H):
    """Rows at every offset from a vector's alignment, in and out: the bytes around them stay, and the residual may be
    updated in place."""
    gamma = (1 + 0.1 * torch.randn(H + 1, generator=torch.Generator().manual_seed(H))).cuda()[1:]
    x0, r0 = rand(T, H, xt, H), None if rt is None else rand(T, H, rt, H + 1)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        for off in (0, 1, 2, 3, 5, 7):
            def room(t, like=None):
                b = torch.full((T, H + 9), 7.0, dtype=t, device="cuda")
                if like is not None:
                    b[:, off:off + H] = like
                return b

            def kept(b):
                return (b[:, :off] == 7.0).all() and (b[:, off + H:] == 7.0).all()
            bx, bo = room(xt, x0), room(dtype)
            br = None if rt is None else room(rt, r0)
            r = None if rt is None else br[:, off:off + H]
            want = ops.rms_norm(x0, gamma, residual=r0, alpha=0.9, beta=0.3, dtype=dtype)
            ops.rms_norm(bx[:, off:off + H], gamma, residual=r, alpha=0.9, beta=0.3, dtype=dtype, out=bo[:, off:off + H],
                         residual_out=r)
            assert torch.equal(bo[:, off:off + H], want.out) and kept(bo) and kept(bx)
            if rt is not None:
                assert torch.equal(r, want.residual) and kept(br)


@pytest.mark.parametrize("af,wf", PAIRS)
@pytest.mark.parametrize("T,N", [(1, 1280), (16, 1281), (17, 1505), (64, 2000), (65, 1600), (128, 3333), (128, 5120)])
def test_product_wide_tiles(af, wf, T, N):
    """Few tokens against many weight rows."""
    K = 640
    a, av = operand(T, K, af, T, 2)
    w, wv = operand(N, K, wf, N, 2)
    out = torch.full((T + 1, N + 3), 7.0, dtype=torch.float32, device="cuda")
    ops.mx_matmul(a, w, torch.float32, out=out[:T, :N])
    assert ops.ops_status() == 0
    check_product(out[:T, :N], torch.float32, av, wv, K)
    assert (out[T] == 7.0).all() and (out[:, N:] == 7.0).all()


@pytest.mark.parametrize("af,wf", PAIRS)
@pytest.mark.parametrize("T,N", [(2100, 1200), (1024, 2565), (1021, 5123), (600, 4097), (4096, 513), (1300, 3500)])
def test_product_pair_tiles(af, wf, T, N):
    """Pairs of CTAs with every tile width, whole numbers (exact in any order), aligned and odd rows of out."""
    K = 256
    rng = np.random.default_rng(T)
    opnds, vals = [], []
    for rows, fmt in ((T, af), (N, wf)):
        e = rng.integers(0, 3, (rows, K)).astype(float) * rng.choice([-1.0, 1.0], (rows, K))
        one = 0x38 if fmt == "nvfp4" else 127
        up = rng.integers(0, 2, (rows, K // R.BLOCK[fmt]))
        sb = (one + up * (8 if fmt == "nvfp4" else 1)).astype(np.uint8)
        opnds.append(ops.MxTensor(torch.from_numpy(R.codes(e, fmt)).cuda(), torch.from_numpy(R.tile(sb)).cuda(), fmt, "tiled", rows, K))
        vals.append(R.values(e, sb, fmt))
    want = vals[0] @ vals[1].T
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        out = torch.full((T, N + 1), 7.0, dtype=dtype, device="cuda")
        ops.mx_matmul(*opnds, dtype, out=out[:, :N])
        assert ops.ops_status() == 0
        np.testing.assert_array_equal(out[:, :N].float().cpu().numpy(), torch.from_numpy(want).to(dtype).float().numpy())
        assert (out[:, N] == 7.0).all()
        assert torch.equal(ops.mx_matmul(*opnds, dtype), out[:, :N])


@pytest.mark.parametrize("af,wf", PAIRS)
@pytest.mark.parametrize("T,N,K", [(150, 150, 1280), (129, 449, 256), (500, 500, 512), (1000, 100, 512), (90, 140, 1152),
                                   (200, 2000, 1024), (3000, 300, 256), (333, 65, 768), (8200, 70, 256)])
def test_product_of_middling_sizes(af, wf, T, N, K):
    """Tiles of 64 columns that start in the middle of a 128-row block of scales, split 1 to 8 ways."""
    a, av = operand(T, K, af, T, 2)
    w, wv = operand(N, K, wf, N, 2)
    out = torch.full((T + 1, N + 3), 7.0, dtype=torch.float16, device="cuda")
    ops.mx_matmul(a, w, torch.float16, out=out[:T, :N])
    y = ops.mx_matmul(a, w, torch.float32)
    assert ops.ops_status() == 0
    check_product(y, torch.float32, av, wv, K)
    assert torch.equal(out[:T, :N], y.half())
    assert (out[T] == 7.0).all() and (out[:, N:] == 7.0).all()


def test_operands_of_impossible_sizes_are_refused():
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    for rows, K in ((1 << 40, 1 << 24), (1 << 34, 1 << 30), (-1, 64), (4, 0)):
        with pytest.raises(ops.BeamMoEError):
            ops.mx_dequantize(ops.MxTensor(e, e, "mxfp4", "rows", rows, K))
        with pytest.raises((ops.BeamMoEError, ValueError)):
            ops.mx_tile_scales(ops.MxTensor(e, e, "mxfp4", "rows", rows, K))
    t = ops.mx_quantize(rand(4, 128, torch.bfloat16, 0), "mxfp4", "tiled")
    with pytest.raises((TypeError, ValueError)):
        ops.mx_matmul(t._replace(rows=1 << 40), t)
    with pytest.raises(TypeError):
        ops.mx_matmul(t._replace(rows=5), t)           # not the codes' size
    with pytest.raises(ops.BeamMoEError):
        ops.mx_matmul(t._replace(codes=torch.empty(257, dtype=torch.uint8, device="cuda")[1:]), t)   # 32-byte alignment


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_empty_operands(fmt):
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    for layout in ("rows", "tiled"):
        q = ops.mx_quantize(x, fmt, layout)
        assert q.rows == 0 and q.scales.numel() == 0 and ops.mx_dequantize(q).shape == (0, 128)
    a, w = (ops.mx_tile_scales(ops.mx_quantize(t, fmt)) for t in (x, rand(70, 128, torch.bfloat16, 1)))
    assert ops.mx_matmul(a, w).shape == (0, 70) and ops.mx_matmul(w, a).shape == (70, 0)
    n = ops.rms_norm(x, torch.ones(128, device="cuda"), residual=x, quantize="mxfp8")
    assert n.out.shape == n.residual.shape == (0, 128) and n.quantized.rows == 0
    idx, w = ops.route_scores(torch.empty(0, 8, device="cuda"), 2)
    assert idx.shape == w.shape == (0, 2)


@pytest.mark.parametrize("T,H", [(70, 512), (300, 1000)])
def test_offset_views_give_the_same(T, H):
    """Contiguous tensors that start off their allocation's alignment: the same bits, but for the norm, whose squares are
    summed in the order of its vectors (within check_norm's bound of the exact sum either way)."""
    b = torch.randn(T * H + 8, generator=torch.Generator().manual_seed(1)).cuda()
    gamma = torch.ones(H + 8, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        base = b.to(dt)
        for off in (1, 4, 8):
            v = base[off:off + T * H].view(T, H)
            a = v.clone()
            for t, g in ((v, gamma[off:off + H]), (a, gamma[:H])):
                check_norm(t, None, g, torch.bfloat16, None, "rows")
            if H % 32 == 0:
                for fmt in ("nvfp4", "mxfp4", "mxfp8"):
                    for layout in ("rows", "tiled"):
                        p, q = ops.mx_quantize(v, fmt, layout), ops.mx_quantize(a, fmt, layout)
                        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
                        out = torch.empty(T * H + 8, dtype=dt, device="cuda")[off:off + T * H].view(T, H)
                        assert torch.equal(ops.mx_dequantize(q, dt, out), ops.mx_dequantize(q, dt))
            if dt == torch.float32:
                i, j = (ops.route_scores(t, 8, score="softmax") for t in (v[:, :512], a[:, :512]))
                assert torch.equal(i[0], j[0]) and torch.equal(i[1], j[1])


@pytest.mark.parametrize("af,wf", PAIRS)
@pytest.mark.parametrize("T,N,K", [(1, 18945, 128), (3, 18960, 256), (16, 19000, 640), (33, 20480, 384), (64, 20480, 1152),
                                   (64, 21313, 256), (20, 23680, 256), (64, 23681, 128)])
def test_product_a_few_tiles_more_than_sms(af, wf, T, N, K):
    """One to 37 weight tiles more than one for every SM; whole numbers, exact in any order."""
    rng = np.random.default_rng(N)
    opnds, vals = [], []
    for rows, fmt in ((T, af), (N, wf)):
        e = rng.integers(0, 3, (rows, K)).astype(float) * rng.choice([-1.0, 1.0], (rows, K))
        one = 0x38 if fmt == "nvfp4" else 127
        up = rng.integers(0, 2, (rows, K // R.BLOCK[fmt]))
        sb = (one + up * (8 if fmt == "nvfp4" else 1)).astype(np.uint8)
        opnds.append(ops.MxTensor(torch.from_numpy(R.codes(e, fmt)).cuda(), torch.from_numpy(R.tile(sb)).cuda(), fmt, "tiled", rows, K))
        vals.append(R.values(e, sb, fmt))
    want = vals[0] @ vals[1].T
    out = torch.full((T + 1, N + 5), 7.0, dtype=torch.float32, device="cuda")
    ops.mx_matmul(*opnds, torch.float32, out=out[:T, :N])
    assert ops.ops_status() == 0
    np.testing.assert_array_equal(f64(out[:T, :N]), want)
    assert (out[T] == 7.0).all() and (out[:, N:] == 7.0).all()


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is captured: nothing that loads on first use may break the capture."""
    import os
    import subprocess
    import sys
    import textwrap

    code = textwrap.dedent("""
        import torch
        from group_limited_routing_sigmoid_b200 import ops
        T, H = 70, 512
        x = torch.randn(T, H, device="cuda").bfloat16()
        r, gamma, l = torch.randn(T, H, device="cuda"), torch.ones(H, device="cuda"), torch.randn(T, 60, device="cuda")
        wide = torch.randn(600, H, device="cuda").bfloat16()
        torch.cuda.synchronize()
        def run():
            n = ops.rms_norm(x, gamma, residual=r, quantize="mxfp8")
            w = ops.mx_tile_scales(ops.mx_quantize(wide, "mxfp4"))
            y = ops.mx_matmul(n.quantized, w)
            q = ops.mx_quantize(wide, "nvfp4", "tiled")
            return [n.out, y, ops.mx_matmul(q, q), ops.mx_dequantize(q), *ops.route_scores(l, 4, score="softmax")]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run()))
        assert ops.ops_status() == 0
    """)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0, done.stderr[-2000:]


def test_two_threads_at_once():
    """Calls of several threads, each on its own stream, one of them refused: results and error texts are the thread's own."""
    import threading

    args = [run_inputs(s) for s in (0, 50, 90)]
    want = [run_all(*a) for a in args]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.default_stream())
            for _ in range(20):
                got = run_all(*args[i], stream=s)
                with pytest.raises(ops.BeamMoEError, match="top_k"):
                    ops.route_scores(args[i][4], 61 + i)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                bad.append(i)
        except BaseException as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and ops.ops_status() == 0
