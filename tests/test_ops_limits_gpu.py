"""The handle-free operators at the ends of their documented ranges and in calls that run beside others, on the GPU,
against the 64-bit references in ops_ref.py."""
import numpy as np
import pytest
import torch

import ops_ref as R
from group_limited_routing_sigmoid_b200 import ops
from group_limited_routing_sigmoid_b200.binding import BEAM_ERR_INVALID_ARG, BEAM_ERR_TIMEOUT, library
from group_limited_routing_sigmoid_b200.build import build

pytestmark = pytest.mark.gpu


def setup_module(_):
    build(quiet=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def test_small_tensor_scales_beside_other_work():
    """Tensors of one cluster's size while other kernels hold the SMs, so that the cluster's blocks start at different times."""
    g = torch.Generator().manual_seed(0)
    big = torch.randn(4096, 4096, generator=g).cuda()
    small = [torch.randn(1 + i % 7, 1 + 37 * i, generator=g).cuda() * 10.0 ** (i % 9 - 4) for i in range(60)]
    want = [R.tensor_scale(f64(t)) for t in small]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            busy = [ops.mx_quantize(big, "mxfp8", "tiled") for _ in range(10)]
        got = [ops.mx_tensor_scale(t) for t in small]
        torch.cuda.synchronize()
        assert [float(t) for t in got] == want
    del busy


def check_route(l, k, score, bias=None, G=1, keep=1, gtop=2, renorm=True, scale=1.0):
    idx, w = ops.route_scores(l, k, score=score, bias=bias, n_group=G, topk_group=keep, group_top=gtop, renormalize=renorm, scale=scale)
    ri, rw = R.route(f64(l), k, score, None if bias is None else bias.cpu().numpy(), G, keep, gtop, renorm, scale)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    got = f64(w)
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    ok = ~np.isnan(rw)
    # two exponentials of 2 ulps, E / lanes + 5 <= 69 partial sums and two roundings, in units of half an ulp
    np.testing.assert_allclose(got[ok], rw[ok], rtol=(8 + 69 + 2) * 2.0 ** -24, atol=2.0 ** -149)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(720, 10, 4), (960, 10, 3), (1000, 5, 2), (1017, 9, 8), (561, 17, 1), (1020, 17, 16),
                                      (1023, 3, 2), (930, 31, 30), (1015, 29, 5), (768, 24, 7), (1020, 20, 19), (510, 30, 2)])
def test_route_group_counts_that_are_no_power_of_two(score, E, G, keep):
    """Up to 60 experts a lane; the best ones lie last in their lanes in some rows, NaN and masks too."""
    g = torch.Generator().manual_seed(E + G)
    l = torch.randn(40, E, generator=g) * 2
    size = E // G
    l[8:16, size - 1::size] += 6.0                     # the last expert of every group
    l[16:20] = l[16:20].sort(dim=1).values
    l[20, E - 1] = float("nan")
    l[21, size - 1] = float("nan")
    l[22] = -float("inf")
    l[23, : E - 1] = -float("inf")
    l[24] = l[24].to(torch.bfloat16).float()
    l[25] = 0.0
    l = l.cuda()
    k = min(8, keep * size)
    for bias in (None, (torch.randn(E, generator=g) * 0.05).cuda()):
        for gtop in (1, 2):
            for renorm in (False, True):
                check_route(l, k, score, bias, G, keep, gtop, renorm, 2.5)


def test_route_sums_that_lose_their_small_terms():
    """A lane that adds 59 terms of 0.9 x 2^-24 to one keeps none of them in FP32; a key 47 steps of 2^-24 below one comes
    before the first expert's, 53 below, only in exact arithmetic."""
    E, G = 1020, 17
    l = torch.full((4, E), -100.0)
    l[:, 960:] = -float("inf")                         # the group that is dropped
    l[:, 0] = 0.0
    l[:, 1:60] = float(np.log(0.9 * 2.0 ** -24))
    bias = torch.zeros(E)
    bias[200], bias[300] = 1 - 47 * 2.0 ** -24, 0.5    # the second: what is not chosen lies far below
    check_route(l.cuda(), 2, "softmax", bias.cuda(), G, 16, 2, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("layout", ["rows", "tiled"])
@pytest.mark.parametrize("rows", [3, 700])
def test_found_scales_stay_in_the_quantisers_range(dtype, layout, rows):
    """NVFP4 of tensors that hold their type's largest or lowest value (a mask's, say), the scale found: no finite element
    reads back as NaN or infinity, and the blocks without it are quantised under the scale that is returned."""
    K = 1024                                           # 700 rows: more than one cluster finds the scale of
    for big in (torch.finfo(dtype).max, torch.finfo(dtype).min, 1.5e37, 1.0):
        x = torch.randn(rows, K, generator=torch.Generator().manual_seed(rows)) * 3
        x[rows // 2, K - 1] = big
        x = x.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max).to(dtype).cuda()
        q = ops.mx_quantize(x, "nvfp4", layout)
        g = min(R.tensor_scale(f64(x)), 2.0 ** 112)
        assert float(q.tensor_scale) == g
        e, sb = R.quantize(f64(x), "nvfp4", g)
        np.testing.assert_array_equal(q.scales.cpu().numpy(), sb.astype(np.uint8) if layout == "rows" else R.tile(sb))
        np.testing.assert_array_equal(R.elements(q.codes.cpu().numpy(), "nvfp4"), e)
        v = ops.mx_dequantize(q, torch.float32)
        assert v.isfinite().all() and (v[rows // 2, K - 1] > 0) == (big > 0)
        given = ops.mx_quantize(x, "nvfp4", layout, tensor_scale=q.tensor_scale)
        assert torch.equal(given.codes, q.codes) and torch.equal(given.scales, q.scales)


def test_found_scales_captured():
    """The scale of a tensor above one cluster's size is a memset and a kernel; both and the quantiser replay on new values."""
    x = torch.randn(300, 4096, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = ops.mx_quantize(x, "nvfp4", "tiled")
        v = ops.mx_dequantize(q)
    for scale in (1.0, 30.0, 0.01):
        x.mul_(scale)
        g.replay()
        torch.cuda.synchronize()
        want = ops.mx_quantize(x, "nvfp4", "tiled")
        assert torch.equal(q.tensor_scale, want.tensor_scale) and torch.equal(q.codes, want.codes)
        assert torch.equal(q.scales, want.scales) and torch.equal(v, ops.mx_dequantize(want))


def test_status_is_refused_in_a_capture_that_goes_on():
    x = torch.randn(64, 512, generator=torch.Generator().manual_seed(1)).cuda()
    want = ops.mx_quantize(x, "mxfp8")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert ops.ops_status() == BEAM_ERR_INVALID_ARG
        q = ops.mx_quantize(x, "mxfp8")
    g.replay()
    assert ops.ops_status() == 0
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("T,N,K,stages", [(1, 256, 2048, (0, 5)), (20, 300, 1024, (0, 3)), (64, 200, 256, (0,)),
                                          (300, 300, 512, (0, 1)), (64, 40000, 512, (0, 1)), (1000, 3333, 512, (1,)),
                                          (2100, 1200, 512, (0, 1))])
def test_waits_that_run_out_end_and_are_reported_once(fmt, T, N, K, stages):
    """Bytes that do not come, in a product's first stage (nothing issued yet) and in a later one (copies and MMAs in flight):
    split tiles, whole ones, persistent ones and pairs.  The next product is skipped, the one after the report is right."""
    g = torch.Generator().manual_seed(T + N)
    a, w = (ops.mx_quantize(torch.randn(n, K, generator=g).bfloat16().cuda(), fmt, "tiled") for n in (T, N))
    want = ops.mx_matmul(a, w)
    assert ops.ops_status() == 0
    for stage in stages:
        assert library().beam_ops_debug_withhold(stage, 5) == 0
        ops.mx_matmul(a, w)
        skipped = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.mx_matmul(a, w, out=skipped)
        assert ops.ops_status() == BEAM_ERR_TIMEOUT
        assert ops.ops_status() == 0
        assert (skipped == 7.0).all()
        assert torch.equal(ops.mx_matmul(a, w), want)
        assert ops.ops_status() == 0


def test_one_of_two_callers_gets_an_event():
    import threading

    a = ops.mx_quantize(torch.randn(64, 512, generator=torch.Generator().manual_seed(1)).cuda(), "mxfp8", "tiled")
    want = ops.mx_matmul(a, a)
    for _ in range(10):
        library().beam_ops_debug_withhold(0, 1)
        ops.mx_matmul(a, a)
        torch.cuda.synchronize()
        got, streams = [], [torch.cuda.Stream() for _ in range(4)]
        threads = [threading.Thread(target=lambda s=s: got.append(ops.ops_status(stream=s))) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(got) == [BEAM_ERR_TIMEOUT, 0, 0, 0]
    assert torch.equal(ops.mx_matmul(a, a), want)


@pytest.mark.parametrize("E", [2, 3, 8, 60, 256, 1000])
@pytest.mark.parametrize("spread", [1.0, 4.0, 12.0, 30.0])
@pytest.mark.parametrize("renorm", [False, True])
def test_softmax_weights_far_below_the_largest(E, spread, renorm):
    """Scores of every size: the rounding of logit - maximum does not reach the weights.  In half ulps: the exponential 4, its
    correction 1, what the sum's terms hold 4 + 10 and its additions ceil(E / 32) + 4, the division and the scale 2."""
    g = torch.Generator().manual_seed(E)
    l = (torch.randn(3000, E, generator=g) * spread).cuda()
    k = min(4, E)
    for bias in (None, (torch.rand(E, generator=g) * 1e-3).cuda()):
        idx, w = ops.route_scores(l, k, score="softmax", bias=bias, renormalize=renorm)
        x = l.double()
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = (p / p.sum(1, keepdim=True)).gather(1, idx.long())
        if renorm:
            p = p / p.sum(1, keepdim=True)
        tol = (4 + 1 + 14 + (E + 31) // 32 + 4 + 2) * 2.0 ** -24 * p + 2.0 ** -149
        assert ((w.double() - p).abs() <= tol).all(), float(((w.double() - p).abs() / tol).max())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(32, 1, 1), (33, 1, 1), (40, 1, 1), (64, 1, 1), (256, 1, 1), (256, 8, 4), (1000, 1, 1), (720, 10, 4)])
def test_route_of_the_largest_top_k_with_a_bias(score, E, G, keep):
    """32 chosen leave no lane for the best that is not: ties and near ties across that border, masks that leave 31 to 33."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn(64, E, generator=g)
    order = l[8:24].argsort(dim=1, descending=True)
    for i, n in enumerate((31, 32, 33, 34) * 4):       # the n best alone are not masked
        l[8 + i].scatter_(0, order[i, n:], -float("inf"))
    l[24:32] = l[24:32].to(torch.bfloat16).float()
    l[32:40] = torch.round(l[32:40])
    l[40:48] = 0.5 + torch.arange(E) * 2.0 ** -24      # neighbours one ulp apart
    l = l.cuda()
    for bias in (torch.zeros(E), torch.randn(E, generator=g) * 0.05, torch.randn(E, generator=g) * 1e-8):
        check_route(l, 32, score, bias.cuda(), G, keep)


@pytest.mark.parametrize("af,wf", [("nvfp4", "nvfp4"), ("mxfp4", "mxfp4"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp8")])
@pytest.mark.parametrize("T,N,K", [(6, 70, 256), (70, 6, 256), (300, 300, 512), (2100, 1200, 256)])
def test_values_that_are_not_finite_reach_their_row_and_column_alone(af, wf, T, N, K):
    """What the quantiser writes for a block with an infinity or a NaN, codes of zero under a scale of NaN, makes the whole row
    (of a) or column (of w) of the product NaN, and nothing else; so does a tensor scale out of range."""
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, K, generator=g).cuda(), torch.randn(N, K, generator=g).cuda()
    x[2, 5], w[3, K - 1] = float("nan"), float("inf")
    a, b = ops.mx_quantize(x, af, "tiled"), ops.mx_quantize(w, wf, "tiled")
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 3] = True, True
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(ops.mx_matmul(a, b, dtype).isnan(), bad)
    if af == "nvfp4":
        far = ops.mx_quantize(x, af, "tiled", torch.full((1,), 2.0 ** 113, device="cuda"))
        assert ops.mx_matmul(far, b).isnan().all()
    assert ops.ops_status() == 0


def test_norm_repeats_itself_and_its_codes_differ_next_to_ties_alone():
    """The same bits every time; and where a code or a scale is not that of the exact row, the exact value lies within the FP32
    row's own error of the border between the two."""
    T, H = 2048, 5120
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(T, H, generator=g, device="cuda") * 3).bfloat16()
    r = torch.randn(T, H, generator=g, device="cuda")
    gamma = 1 + 0.02 * torch.randn(H, generator=g, device="cuda")
    alpha, beta = float(np.float32(np.sqrt(19 / 20))), float(np.float32(np.sqrt(1 / 20)))
    runs = [ops.rms_norm(x, gamma, residual=r, alpha=alpha, beta=beta, quantize="mxfp8", layout="rows") for _ in range(4)]
    for o in runs[1:]:
        assert torch.equal(o.out, runs[0].out) and torch.equal(o.residual, runs[0].residual)
        assert torch.equal(o.quantized.codes, runs[0].quantized.codes) and torch.equal(o.quantized.scales, runs[0].quantized.scales)
    q = runs[0].quantized
    s = beta * x.double() + alpha * r.double()
    scale = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + float(np.float32(1e-6)))
    y = s * scale * gamma.double()
    # s: two products and a sum; the mean of squares: at most 16 fused terms and 10 joins a thread, twice what s is off, and half
    # of both reaches y; root, division and two products
    u = 2.0 ** -24
    ds = 2 * u * ((beta * x.double()).abs() + (alpha * r.double()).abs())
    ds_row = (ds * ds).mean(1, keepdim=True).sqrt() * scale
    dy = y.abs() * ((0.5 * (16 + 10 + 2) + 5) * u + ds_row) + ds * scale * gamma.double()
    amax, damax = y.abs().view(T, -1, 32).amax(-1), dy.view(T, -1, 32).amax(-1)

    def exponent(a):                                   # least k with a <= 448 x 2^k
        m, e = torch.frexp(a)
        return torch.where(m <= 0.875, e - 9, e - 8)
    k = q.scales.int() - 127
    assert ((k == exponent(amax)) | (exponent(amax - damax) != exponent(amax + damax))).all()
    p = torch.exp2(k.double()).repeat_interleave(32, dim=1)
    grid = torch.from_numpy(R.E4M3).cuda()
    code = (q.codes & 127).long()
    mid = (grid[1:] + grid[:-1]) / 2
    border = torch.cat([torch.tensor([0.0], dtype=torch.float64, device="cuda"), mid, torch.tensor([1e9], dtype=torch.float64, device="cuda")])
    assert (y.abs() + dy >= border[code] * p).all() and (y.abs() - dy <= border[code + 1] * p).all()
    off = (y.abs() < border[code] * p) | (y.abs() > border[code + 1] * p)
    assert off.double().mean() < 1e-4


def test_route_refuses_a_top_k_before_it_makes_outputs():
    l = torch.randn(60000, 64, device="cuda")
    some = torch.empty(60000, 33, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocated_bytes.all.allocated"]
    for k in (2 ** 31 - 1, 33, 0, -1):
        for idx in (None, some):
            with pytest.raises(ops.BeamMoEError, match="top_k"):
                ops.route_scores(l, k, idx=idx)
    assert torch.cuda.memory_stats()["allocated_bytes.all.allocated"] == before


def test_inputs_that_require_a_gradient_give_results_that_do_not():
    x = torch.randn(8, 256, device="cuda", requires_grad=True)
    gamma = torch.nn.Parameter(torch.ones(256, device="cuda"))
    n = ops.rms_norm(x, gamma, residual=x, quantize="mxfp8")
    q = ops.mx_quantize(x, "mxfp8", "tiled")
    results = [n.out, n.residual, ops.mx_matmul(n.quantized, q), ops.mx_dequantize(q), *ops.route_scores(x, 4), ops.mx_tensor_scale(x)]
    assert not any(t.requires_grad for t in results)
    with torch.no_grad():
        again = ops.rms_norm(x, gamma, residual=x)
    assert torch.equal(again.out, n.out)


@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_weights_down_to_the_least_subnormal(renorm):
    """exp(-x) overflows below -88.7, the score only vanishes below -104.  In half ulps: the exponential 4, sum, division, scale
    and, renormalised, up to 5 joins and another division; half the least subnormal each where the result is one."""
    l = torch.cat([torch.linspace(-106, -80, 500), torch.linspace(-1, 40, 140)]).view(-1, 1).repeat(1, 4)
    l += torch.arange(4) * -0.37
    idx, w = ops.route_scores(l.cuda(), 4, renormalize=renorm)
    assert (idx == torch.arange(4, device="cuda")).all()
    p = 1 / (1 + torch.exp(-l.double()))
    if renorm:
        p = p / p.sum(1, keepdim=True)
    assert ((w.cpu().double() - p).abs() <= 14 * 2.0 ** -24 * p + 4 * 2.0 ** -149).all()


@pytest.mark.parametrize("name", ["decode_small", "decode_small_nvfp4", "dense_tiny"])
def test_beside_a_handles_block_on_another_stream(name):
    """A block's forward and the operators at once, each on its own stream: both use tensor memory, and give what they give alone."""
    from group_limited_routing_sigmoid_b200 import workloads as W
    from group_limited_routing_sigmoid_b200.binding import BeamMoE

    wl = W.WORKLOADS[name]
    d = W.make_inputs(wl, "cuda")
    if name.endswith("nvfp4"):
        E, I, H = wl.n_experts, wl.inter, wl.hidden
        for n, rows, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            q = ops.mx_quantize(torch.randn(E * rows, K, device="cuda").mul_(0.02).bfloat16(), "nvfp4")
            d[n + "_codes"], d[n + "_scales"] = q.codes.view(E, rows, K // 2), q.scales.view(E, rows, K // 16)
            d[n + "_global"] = float(q.tensor_scale)
    moe = BeamMoE.from_workload(wl, d)
    out = torch.empty_like(d["x"])
    moe.forward(d["x"], out=out)
    want = out.clone()
    g = torch.Generator().manual_seed(2)
    pairs = [tuple(ops.mx_quantize(torch.randn(n, K, generator=g).bfloat16().cuda(), fmt, "tiled") for n in (T, N))
             for fmt, T, N, K in (("nvfp4", 1, 5120, 5120), ("mxfp8", 64, 20480, 640), ("mxfp4", 500, 500, 512), ("nvfp4", 2048, 2048, 512))]
    alone = [ops.mx_matmul(a, w) for a, w in pairs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        moe.forward(d["x"], out=out)
        with torch.cuda.stream(side):
            got = [ops.mx_matmul(a, w) for a, w in pairs]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and moe.get_status() == 0 and ops.ops_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, alone))
    moe.close()
