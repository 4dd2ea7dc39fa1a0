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
