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
