"""The handle-free operators at the ends of their documented ranges and in calls that run beside others, on the GPU,
against the 64-bit references in ops_ref.py."""
import numpy as np
import pytest
import torch

import ops_ref as R
from group_limited_routing_sigmoid_b200 import ops
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
