"""What the handle-free operators decide on the host or lay down in the source, checked without a GPU: synchronisation,
lane layouts and plans over their documented ranges."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "group_limited_routing_sigmoid_b200", "csrc")

HOST = r"""
#include "mx_plan.h"
#include "route_layout.h"
#include <cstdint>
#include <cstring>
using namespace beam;
// 0, or what is wrong with a row's layout: 1 registers, 2 an expert read by no lane or twice, 3 one out of range, 4 a group
// that does not lie in its own lanes.
extern "C" int walk(int E, int G, int keep, int *at)
{
    const RouteLayout l = route_layout(E, G, keep);
    bool known = false;
    for (int r = 1; r <= 64; r *= 2) known |= l.regs == r;
    if (!known || l.epl > l.regs) return at[0] = l.epl, at[1] = l.regs, 1;
    uint8_t seen[1024];
    memset(seen, 0, sizeof(seen));
    for (int lane = 0; lane < 32; ++lane) {
        const Span my(lane, l.lanes_log, l.size, l.epl, E);
        for (int i = 0; i < l.regs; ++i) {
            if (i >= my.mine) continue;
            const int e = my.e0 + i;
            if (e < 0 || e >= E) return at[0] = lane, at[1] = e, 3;
            if (keep < G && e / (E / G) != lane >> l.lanes_log) return at[0] = lane, at[1] = e, 4;
            ++seen[e];
        }
    }
    for (int e = 0; e < E; ++e)
        if (seen[e] != 1) return at[0] = e, at[1] = seen[e], 2;
    return 0;
}

// A plan's width, split and whether it is a pair's.
extern "C" void make_plan(int kind, int P, int Q, int nst, int swap, int vec, int sms, int *out)
{
    const mx::Plan p = mx::plan(kind, P, Q, nst, swap != 0, vec != 0, sms);
    out[0] = p.bn, out[1] = p.split, out[2] = p.pair;
}
"""


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_block_writes_to_another_before_all_have_started():
    """A store into another block's shared memory needs a cluster barrier before it: nothing else says that the block exists."""
    kernel = source("mx_quant.cu").split("void __launch_bounds__(kThreadsQ) mx_amax_kernel", 1)[1].split("\ntemplate", 1)[0]
    store = kernel.index("st.shared::cluster")
    assert "barrier.cluster.wait" in kernel[:store] or "cluster_sync()" in kernel[:store]
    assert kernel.count("barrier.cluster.arrive") == kernel.count("barrier.cluster.wait")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """The headers' host functions, compiled for the CPU."""
    d = tmp_path_factory.mktemp("host")
    with open(d / "host.cpp", "w") as f:
        f.write(HOST)
    so = str(d / "host.so")
    subprocess.check_call([shutil.which("g++") or os.environ.get("CXX", "c++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                           "-o", so, str(d / "host.cpp")])
    return ctypes.CDLL(so)


def test_every_expert_has_one_lane_and_one_register(host):
    """All (E, n_group) that the header documents, groups dropped or not, as the kernel's lanes and loops walk them."""
    bad = np.zeros(4, np.int32)
    count = 0
    for E in range(1, 1025):
        for G in range(1, 33):
            if E % G:
                continue
            for keep in {1, G}:
                count += 1
                assert host.walk(E, G, keep, bad.ctypes.data_as(ctypes.c_void_p)) == 0, (E, G, keep, bad)
    assert count > 5000


@pytest.mark.parametrize("sms", [1, 2, 7, 16, 74, 132, 148, 152, 160, 208])
def test_every_product_has_a_plan(host, sms):
    """Whatever the device's SM count: a width, a split of no more parts than K has stages, one B tile below 64 columns."""
    out = np.zeros(3, np.int32)
    at = out.ctypes.data_as(ctypes.c_void_p)
    edges = {1, 2, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 1000, 4097, 37888, 37889, 38000, 38912, 38913, 100000, (1 << 27) - 1}
    edges |= {128 * n + d for n in (sms, 2 * sms, 45, 93) for d in (-1, 0, 1)}
    for T in (1, 5, 16, 17, 32, 33, 64, 65, 128, 129, 1021, 8192, 38000, 50000, (1 << 27) - 1):
        for N in sorted(e for e in edges if e > 0):
            swap = N >= T if T <= 128 or N <= 128 else False
            P, Q = (N, T) if swap else (T, N)
            for nst in (1, 2, 3, 7, 8, 80):
                for kind in range(3):
                    for vec in (0, 1):
                        host.make_plan(kind, P, Q, nst, int(swap), vec, sms, at)
                        bn, split, pair = out
                        what = (kind, T, N, nst, vec, list(out))
                        assert bn in ((256,) if pair else (16, 32, 64, 128)), what
                        assert 1 <= split <= min(8, nst) and (bn >= 64 or bn >= Q), what
                        assert not (pair and (swap or split > 1 or P <= 128 or Q <= 128)), what
