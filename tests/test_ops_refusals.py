"""Refusals of the handle-free operators' entry points: host checks run before any CUDA call, so none of this needs a GPU."""
import ctypes

import pytest
import torch

from group_limited_routing_sigmoid_b200 import binding, ops
from group_limited_routing_sigmoid_b200.build import build

INVALID = binding.BEAM_ERR_INVALID_ARG
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build(quiet=True)
    return binding.library()


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(codes=None), dict(scales=None), dict(g=None), dict(dtype=3), dict(rows=-1), dict(K=24), dict(K=0),
    dict(ldx=32), dict(layout=2), dict(x=17), dict(codes=24), dict(scales=18), dict(g=18), dict(rows=1 << 40, K=1 << 30, ldx=1 << 30),
])
def test_quantize_nvfp4_refuses(lib, kw):
    a = dict(x=16, dtype=0, rows=4, K=64, ldx=64, layout=0, g=16, codes=16, scales=16)
    a.update(kw)
    x, g, codes, scales = (a[n] and P(a[n]) for n in ("x", "g", "codes", "scales"))
    assert lib.beam_mx_quantize_nvfp4(None, x, a["dtype"], a["rows"], a["K"], a["ldx"], a["layout"], g, codes, scales) == INVALID
    assert lib.beam_ops_error()


def test_withhold_refuses(lib):
    for stage, ms in ((-2, 10), (0, 0), (0, -1), (0, 2001)):
        assert lib.beam_ops_debug_withhold(stage, ms) == INVALID
    assert lib.beam_ops_debug_withhold(-1, 1) == binding.BEAM_OK


def test_an_operand_to_write_into_has_codes_and_scales():
    x, some = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.uint8)
    for codes, scales in ((None, some), (some, None)):
        with pytest.raises(TypeError, match="codes and scales"):
            ops.mx_quantize(x, "mxfp4", out=ops.MxTensor(codes, scales, "mxfp4", "rows", 4, 64))
