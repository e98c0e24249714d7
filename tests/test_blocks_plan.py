"""Block attention's layout is one of a device: its SMs and the clusters that it runs at once (no GPU needed)."""
import ctypes

import pytest

from speculative_decoding_tree_05_gb300 import ddtree

CLUSTERS = [0, 0, 76, 50, 34, 30, 24, 20, 16]


@pytest.fixture(scope="module")
def plan():
    from speculative_decoding_tree_05_gb300 import build
    build.build()
    fn = ddtree.lib().ddtree_internal_blocks_plan

    def call(dims, block, topk, sms, clusters):
        out, n = (ctypes.c_int32 * 3)(), ctypes.c_int64()
        rc = fn(ctypes.byref(dims), block, topk, sms, (ctypes.c_int32 * 9)(*clusters), out, ctypes.byref(n))
        return rc, tuple(out), n.value
    return call


def dims(batch=16, nodes=1, heads=16, n=32768):
    return ddtree.make_dims(batch, nodes, heads, 1 << 19, n, n)


def test_devices_do_not_share_a_layout(plan):
    """The same sizes on two devices in turn, one of which runs no clusters: each keeps its own."""
    d = dims()
    a, b = plan(d, 32, 32, 152, CLUSTERS), plan(d, 32, 32, 152, [0] * 9)
    assert a[0] == b[0] == 0
    assert a[1][2] == 1 and b[1][2] == 0
    assert b[2] > a[2]                      # partial results lie in the workspace only where a merge kernel joins them
    assert plan(d, 32, 32, 152, CLUSTERS) == a and plan(d, 32, 32, 152, [0] * 9) == b


@pytest.mark.parametrize("batch,nodes,heads", [(1, 1, 1), (16, 1, 16), (4, 9, 16), (8, 33, 16), (1, 65, 128), (40, 1, 32)])
def test_splits_and_workspace(plan, batch, nodes, heads):
    for clusters in (CLUSTERS, [0] * 9):
        rc, (groups, splits, clustered), n = plan(dims(batch, nodes, heads), 64, 32, 152, clusters)
        assert rc == 0 and 1 <= splits <= 32
        rows = min(64, heads * nodes if heads <= 64 else 64)
        assert groups == (-(-nodes // (64 // heads)) if heads <= 64 else nodes * -(-heads // 64))
        if clustered:
            assert 2 <= splits <= 8 and rows <= 32 and batch * groups <= clusters[splits]
        part = batch * splits * nodes * heads * (512 + 1) * 4
        if splits > 1 and not clustered:      # the partials have their room
            assert n >= part


def test_refusals(plan):
    assert plan(dims(), 48, 32, 152, CLUSTERS)[0] == -2
    assert plan(dims(), 64, 0, 152, CLUSTERS)[0] == -2
