"""The references of the handle-free operators against independent forms, and
the refusals of the operators' entry points: host checks run before any CUDA
call, so all of this needs no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import ops_ref as R
from group_limited_routing_sigmoid_b200 import binding, ops
from group_limited_routing_sigmoid_b200.build import build

INVALID, UNSUPPORTED, OK = binding.BEAM_ERR_INVALID_ARG, binding.BEAM_ERR_UNSUPPORTED, binding.BEAM_OK
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build(quiet=True)
    return binding.library()


# --- references ------------------------------------------------------------------

def test_e4m3_reference_matches_torch():
    v = np.concatenate([np.linspace(-460, 460, 20001), R.E4M3, (R.E4M3[1:] + R.E4M3[:-1]) / 2]).astype(np.float32)
    got = np.copysign(R.E4M3[R.nearest_code(v.astype(np.float64), R.E4M3)], v)
    want = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, want)


def test_e2m1_ties_go_to_the_even_code():
    mid = (R.E2M1[1:] + R.E2M1[:-1]) / 2
    np.testing.assert_array_equal(R.nearest_code(mid, R.E2M1), [0, 2, 2, 4, 4, 6, 6])


def test_pow2_exponent_is_the_least():
    for top in (6.0, 448.0):
        a = np.concatenate([top * 2.0 ** np.arange(-130, 120), top * 2.0 ** np.arange(-130.0, 120) * (1 + 2.0 ** -23),
                            [0.0, 1.0, 3.4e38]])
        k = R.pow2_exponent(a, top)
        assert np.all((a <= top * 2.0 ** k) | (k == 127))
        assert np.all((a > top * 2.0 ** (k - 1.0)) | (k == -127))


@pytest.mark.parametrize("rows,n", [(1, 1), (128, 4), (130, 6), (257, 9)])
def test_tile_is_a_permutation(rows, n):
    sb = np.random.default_rng(0).integers(1, 255, (rows, n)).astype(np.uint8)
    t = R.tile(sb)
    r, c = (rows + 127) // 128 * 128, (n + 3) // 4 * 4
    back = t.reshape(r // 128, c // 4, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(r, c)
    np.testing.assert_array_equal(back[:rows, :n], sb)
    assert back[rows:].sum() == 0 and back[:, n:].sum() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
def test_codes_round_trip(fmt):
    rng = np.random.default_rng(1)
    e, sb = R.quantize(rng.standard_normal((5, 96)).astype(np.float32).astype(np.float64), fmt, 2.0 ** -9)
    np.testing.assert_array_equal(R.elements(R.codes(e, fmt), fmt), e)


def test_route_reference_matches_torch_softmax():
    l = np.random.default_rng(2).standard_normal((20, 24))
    idx, w = R.route(l, 4, "softmax", None, 1, 1, 2, False, 1.0)
    p, i = torch.topk(torch.softmax(torch.from_numpy(l), 1), 4)
    np.testing.assert_array_equal(idx, i.numpy())
    np.testing.assert_allclose(w, p.numpy(), rtol=1e-12)


# --- refusals ----------------------------------------------------------------------

def test_scale_bytes(lib):
    for fmt, f in ops.FORMATS.items():
        for layout, l in ops.LAYOUTS.items():
            for rows in (0, 1, 128, 129, 1000):
                assert ops.scale_bytes(fmt, rows, 96, layout) == lib.beam_mx_scale_bytes(f, rows, 96, l)
    assert lib.beam_mx_scale_bytes(0, 3, 64, 0) == 12
    assert lib.beam_mx_scale_bytes(0, 3, 64, 1) == 512
    assert lib.beam_mx_scale_bytes(0, 129, 80, 1) == 2 * 2 * 512
    assert lib.beam_mx_scale_bytes(2, 128, 128, 1) == 512
    assert lib.beam_mx_scale_bytes(1, 0, 32, 1) == 0
    for bad in ((3, 1, 32, 0), (0, -1, 32, 0), (0, 1, 24, 0), (1, 1, 16, 0), (1, 1, 0, 0), (1, 1, 32, 2)):
        assert lib.beam_mx_scale_bytes(*bad) == INVALID


def test_sizes_past_memory_are_refused(lib):
    """Products of sizes that wrap around in 64 bits do not pass for small tensors."""
    assert lib.beam_mx_scale_bytes(1, 1 << 40, 1 << 30, 0) == INVALID
    assert lib.beam_mx_quantize(None, P(32), 0, 1 << 40, 1 << 30, 1 << 30, 1, 0, None, P(32), P(32)) == INVALID
    assert lib.beam_mx_dequantize(None, P(32), P(32), None, 1, 0, 1 << 40, 1 << 30, P(32), 0, 1 << 30) == INVALID
    assert lib.beam_mx_tile_scales(None, 1, P(32), 1 << 40, 1 << 30, P(32)) == INVALID
    assert lib.beam_mx_tensor_scale(None, P(32), 0, 1 << 40, 1 << 30, 1 << 30, P(32)) == INVALID


def quantize(lib, x=16, dtype=0, rows=4, K=64, ldx=64, fmt=1, layout=0, g=None, codes=16, scales=16):
    return lib.beam_mx_quantize(None, x and P(x), dtype, rows, K, ldx, fmt, layout, g and P(g), codes and P(codes),
                                scales and P(scales))


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(codes=None), dict(scales=None), dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(K=48),
    dict(K=0), dict(ldx=32), dict(fmt=3), dict(layout=2), dict(g=16), dict(fmt=0), dict(x=17), dict(codes=24),
    dict(scales=18), dict(dtype=2, x=18), dict(fmt=0, g=18),
])
def test_quantize_refuses(lib, kw):
    assert quantize(lib, **kw) == INVALID
    assert lib.beam_ops_error()


def test_empty_calls_do_nothing(lib):
    assert quantize(lib, rows=0, x=None, codes=None, scales=None) == OK
    assert lib.beam_mx_dequantize(None, None, None, None, 1, 0, 0, 32, None, 0, 32) == OK
    assert lib.beam_mx_tile_scales(None, 1, None, 0, 32, None) == OK
    assert matmul(lib, T=0) == OK and matmul(lib, N=0, ldo=0) == OK
    assert norm(lib, T=0, x=None, gamma=None, out=None) == OK
    assert route(lib, T=0, logits=None) == OK


@pytest.mark.parametrize("args", [
    (None, 16, None, 1, 0, 4, 64, 16, 0, 64), (16, None, None, 1, 0, 4, 64, 16, 0, 64),
    (16, 16, None, 1, 0, 4, 64, None, 0, 64), (16, 16, None, 3, 0, 4, 64, 16, 0, 64),
    (16, 16, None, 1, 0, 4, 48, 16, 0, 64), (16, 16, None, 1, 0, 4, 64, 16, 0, 63),
    (16, 16, None, 1, 0, 4, 64, 17, 0, 64), (24, 16, None, 1, 0, 4, 64, 16, 0, 64),
    (16, 16, None, 1, 0, 4, 64, 16, 5, 64), (16, 16, 18, 1, 0, 4, 64, 16, 0, 64),
])
def test_dequantize_refuses(lib, args):
    c, s, g, fmt, layout, rows, K, out, dtype, ldo = args
    assert lib.beam_mx_dequantize(None, c and P(c), s and P(s), g and P(g), fmt, layout, rows, K, out and P(out), dtype,
                                  ldo) == INVALID


def test_tensor_scale_and_tile_refuse(lib):
    assert lib.beam_mx_tensor_scale(None, P(16), 0, 4, 0, 64, P(16)) == INVALID
    assert lib.beam_mx_tensor_scale(None, P(16), 0, -1, 64, 64, P(16)) == INVALID
    assert lib.beam_mx_tensor_scale(None, None, 0, 4, 64, 64, P(16)) == INVALID
    assert lib.beam_mx_tensor_scale(None, P(16), 0, 4, 64, 63, P(16)) == INVALID
    assert lib.beam_mx_tensor_scale(None, P(16), 0, 4, 64, 64, None) == INVALID
    assert lib.beam_mx_tensor_scale(None, P(16), 7, 4, 64, 64, P(16)) == INVALID
    assert lib.beam_mx_tile_scales(None, 1, P(16), 4, 48, P(16)) == INVALID
    assert lib.beam_mx_tile_scales(None, 1, None, 4, 64, P(16)) == INVALID
    assert lib.beam_mx_tile_scales(None, 1, P(16), 4, 64, P(18)) == INVALID


def matmul(lib, af=0, ac=32, asc=32, ag=None, wf=0, wc=32, wsc=32, wg=None, T=4, N=8, K=128, out=16, dtype=0, ldo=8):
    p = lambda v: v and P(v)
    return lib.beam_mx_matmul(None, af, p(ac), p(asc), p(ag), wf, p(wc), p(wsc), p(wg), T, N, K, p(out), dtype, ldo)


@pytest.mark.parametrize("kw,code", [
    (dict(ac=None), INVALID), (dict(asc=None), INVALID), (dict(wc=None), INVALID), (dict(wsc=None), INVALID),
    (dict(out=None), INVALID), (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(T=1 << 27), INVALID),
    (dict(K=0), INVALID), (dict(K=96), UNSUPPORTED), (dict(af=2, wf=1, K=64), UNSUPPORTED),
    (dict(af=1), UNSUPPORTED), (dict(wf=2), UNSUPPORTED), (dict(af=2, wf=0), UNSUPPORTED), (dict(af=5), INVALID),
    (dict(dtype=3), INVALID), (dict(ldo=7), INVALID), (dict(ac=48), INVALID), (dict(wsc=40), INVALID),
    (dict(out=17), INVALID), (dict(ag=18), INVALID),
])
def test_matmul_refuses(lib, kw, code):
    assert matmul(lib, **kw) == code
    assert lib.beam_ops_error()


def norm(lib, x=16, xd=0, ldx=64, r=None, rd=0, ldr=64, ro=None, ldro=64, alpha=1.0, beta=1.0, gamma=16, eps=1e-6, T=4,
         H=64, out=16, od=0, ldo=64, codes=None, scales=None, layout=0):
    p = lambda v: v and P(v)
    return lib.beam_rms_norm(None, p(x), xd, ldx, p(r), rd, ldr, p(ro), ldro, alpha, beta, p(gamma), eps, T, H, p(out), od,
                             ldo, p(codes), p(scales), layout)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(gamma=None), INVALID), (dict(out=None), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(T=2 ** 31 - 1), UNSUPPORTED), (dict(H=32769, ldx=32769, ldo=32769), UNSUPPORTED), (dict(xd=3), INVALID),
    (dict(od=3), INVALID), (dict(r=16), INVALID), (dict(ro=16), INVALID), (dict(r=16, ro=32, rd=1), INVALID),
    (dict(ldx=63), INVALID), (dict(ldo=63), INVALID), (dict(r=16, ro=32, rd=2, ldr=60), INVALID),
    (dict(codes=16), INVALID), (dict(scales=16), INVALID), (dict(codes=16, scales=16, layout=2), INVALID),
    (dict(codes=16, scales=16, H=48), INVALID), (dict(codes=24, scales=16), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(alpha=float("inf")), INVALID), (dict(beta=float("nan")), INVALID),
    (dict(x=17), INVALID), (dict(gamma=18), INVALID),
])
def test_norm_refuses(lib, kw, code):
    assert norm(lib, **kw) == code
    assert lib.beam_ops_error()


def route(lib, logits=16, T=4, E=64, ldl=64, score=0, bias=None, G=1, keep=1, gtop=2, k=4, renorm=1, scale=1.0, idx=16,
          w=16):
    p = lambda v: v and P(v)
    return lib.beam_route_scores(None, p(logits), T, E, ldl, score, p(bias), G, keep, gtop, k, renorm, scale, p(idx), p(w))


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(idx=None), dict(w=None), dict(T=-1), dict(E=0), dict(E=1025, ldl=1025), dict(ldl=63),
    dict(score=2), dict(G=0), dict(G=3), dict(G=64), dict(G=8, keep=9), dict(keep=0), dict(gtop=0), dict(gtop=3),
    dict(k=0), dict(k=33), dict(G=16, keep=1, k=5), dict(scale=float("nan")), dict(logits=18), dict(bias=17),
])
def test_route_refuses(lib, kw):
    assert route(lib, **kw) == INVALID
    assert lib.beam_ops_error()


def test_bindings_refuse_what_is_no_cuda_matrix():
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        ops.mx_quantize(x, "mxfp4")
    with pytest.raises(TypeError):
        ops.rms_norm(x, torch.zeros(64))
    with pytest.raises(TypeError):
        ops.route_scores(x, 2)
    with pytest.raises(ValueError):
        ops.scale_bytes("fp4", 4, 64, "rows")
    q = ops.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), "mxfp4", "rows", 4, 64)
    with pytest.raises(TypeError):
        ops.mx_dequantize(q)


def test_binding_turns_refusals_into_exceptions():
    """The compiled binding's own checks: what is no tensor, wrong counts, integers and reals out of place."""
    f = ops._native()
    x = torch.zeros(4, 64)
    q = ops.MxTensor(x, x, "mxfp4", "rows", 4, 64)
    for call, args in ((f.quantize, (x, 1)), (f.quantize, (3, 1, 0, None, None, None, "mxfp4", "rows")),
                       (f.quantize, (None,) * 8),
                       (f.rms_norm, (x,) * 15), (f.matmul, ("a",) * 4), (f.matmul, (x, x, 0, None)),
                       (f.dequantize, ((x, x, "mxfp4", "rows", 4, 64, None), 0, None)), (f.dequantize, (q, 0, None)),
                       (f.dequantize, (q._replace(K="K"), 0, None)), (f.matmul, (q._replace(layout="tiled"),) * 2 + (0, None)),
                       (f.tile_scales, (x, 1, 2.5, 64)), (f.route_scores, (x,) * 11), (f.tensor_scale, (x, None))):
        with pytest.raises(TypeError):
            call(*args)
    with pytest.raises(ValueError):
        f.tile_scales(x, 1 << 40, 4, 64)
    for call, args in ((f.dequantize, (q._replace(format="fp4"), 0, None)), (f.dequantize, (q._replace(layout=1), 0, None)),
                       (f.dequantize, (q._replace(K=1 << 40), 0, None)), (f.matmul, (q, q, 0, None)),
                       (f.matmul, (q._replace(layout="tiled"), q._replace(layout="tiled", K=32), 0, None)),
                       (f.matmul, (q._replace(layout="tiled", rows=1 << 33),) * 2 + (0, None))):
        with pytest.raises(ValueError):
            call(*args)
    with pytest.raises(OverflowError):
        f.tile_scales(x, 1, 1 << 80, 64)
