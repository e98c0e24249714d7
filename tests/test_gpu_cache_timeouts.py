"""A bounded wait that runs out in the kernels of the cache-size and block operators: the status word says so, the context
stays usable and the next call is right.  A test build (short limits) keeps one buffer back, so that the wait for it
runs out; no load is left out, and every copy lands before its CTA exits."""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import build_and_load, require_cuda
import test_gpu_block_attn as attn
import test_gpu_block_select as select
import test_gpu_key_weight as weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks():
    require_cuda()
    build_and_load()
    return build_and_load("testhooks")


def status_of(hooks, buffer, call, status):
    """The status words of a call that keeps a buffer back, and of the same call after it."""
    hooks.ddtree_test_set_keep_back(buffer)
    try:
        call()
        first = status()
    finally:
        hooks.ddtree_test_set_keep_back(-1)
    result = call()
    return first, status(), result


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("buffer", [0, 1, 3])
def test_block_summary(hooks, monkeypatch, block, buffer):
    kv, slot, n = select.pool_of([60000, 20000], seed=block)
    want, want_scale = ddtree.block_summary(kv, slot, n, block)
    monkeypatch.setattr(ddtree, "_lib", hooks)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    first, after, (got, scale) = status_of(hooks, buffer, lambda: ddtree.block_summary(kv, slot, n, block, workspace=ws),
                                           lambda: ddtree.read_device_status(ws))
    assert first & ddtree.STATUS_TIMEOUT and after == 0
    assert torch.equal(got, want) and torch.equal(scale, want_scale)


@pytest.mark.parametrize("lens,chosen,buffer", [
    ([2000], None, 0), ([2000], None, 1), ([9000, 300], None, 0), ([9000, 300], None, 4), ([9000, 300], 40, 1),
    ([9000, 300], 40, 4)])
def test_key_weights(hooks, lens, chosen, buffer):
    """65 x 64 rows are 33 tiles, 20 for 40 chosen nodes; one request of 2000 shares them out, three or four to a unit.

    Tile buffer + 2 waits for what is kept back.
    """
    d = weight.make(len(lens), lens, 65, 64, seed=1)
    sel = None
    if chosen:
        sel = torch.arange(chosen, dtype=torch.int32, device="cuda").expand(len(lens), chosen).contiguous()
    k = ddtree.KeyWeights(len(lens), 65, 64, d["kv"].shape[0], max(lens), library=hooks)
    first, after, out = status_of(hooks, buffer, lambda: k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], weight.SCALE,
                                                           node_idx=sel), k.status)
    assert first & ddtree.STATUS_TIMEOUT and after == 0
    weight.check(d, out, sel=sel)


@pytest.mark.parametrize("buffer", [0, 1])
def test_block_selector(hooks, buffer):
    """8 x 65 x 16 rows against 1250 blocks: 9 tiles of rows a request."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(8, 65, 16, 576, generator=g, device="cuda").to(torch.bfloat16)
    summary = torch.randint(-127, 128, (8, 1250, 576), generator=g, device="cuda").to(torch.bfloat16)
    scale = torch.rand(8, 1250, generator=g, device="cuda")
    n = torch.full((8,), 20000, dtype=torch.int32, device="cuda")
    want = ddtree.BlockSelector(8, 65, 16, 20000, 16, 32)(q, summary, scale, n)
    s = ddtree.BlockSelector(8, 65, 16, 20000, 16, 32, library=hooks)
    first, after, got = status_of(hooks, buffer, lambda: s(q, summary, scale, n), s.status)
    assert first & ddtree.STATUS_TIMEOUT and after == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("buffer", [0, 1])
@pytest.mark.parametrize("batch,nodes,heads,topk", [
    (16, 1, 16, 32),        # few rows: the splits are clusters
    (4, 1, 16, 160),        # more splits than a cluster has, and a merge kernel
    (2, 8, 16, 100),        # 64 rows
    (40, 9, 16, 12),        # 120 groups: one split
    (1, 2, 128, 160)])      # slices of one node's heads
def test_block_verifier(hooks, buffer, batch, nodes, heads, topk):
    """A key list long enough that every split has the three tiles that the wait takes."""
    lens = [topk * 64] * batch
    d = attn.make(lens, nodes, heads, 64, topk, seed=3, lists="all")
    v = ddtree.BlockVerifier(batch, nodes, heads, d["kv"].shape[0], max(lens), 64, topk, library=hooks)
    first, after, (out, lse) = status_of(
        hooks, buffer, lambda: v(d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], d["idx"], attn.SCALE),
        v.status)
    assert first & ddtree.STATUS_TIMEOUT and after == 0
    attn.check(d, out, lse)
