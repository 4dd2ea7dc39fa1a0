"""What the handle-free operators decide on the host or lay down in the source, checked without a GPU: synchronisation,
lane layouts and plans over their documented ranges."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "group_limited_routing_sigmoid_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_block_writes_to_another_before_all_have_started():
    """A store into another block's shared memory needs a cluster barrier before it: nothing else says that the block exists."""
    kernel = source("mx_quant.cu").split("void __launch_bounds__(kThreadsQ) mx_amax_kernel", 1)[1].split("\ntemplate", 1)[0]
    store = kernel.index("st.shared::cluster")
    assert "barrier.cluster.wait" in kernel[:store] or "cluster_sync()" in kernel[:store]
    assert kernel.count("barrier.cluster.arrive") == kernel.count("barrier.cluster.wait")
