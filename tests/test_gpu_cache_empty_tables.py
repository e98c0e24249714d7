"""Tables without a position (max_prefix_len 0): nothing is written, and lengths and nodes are still reported."""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def lengths(bad):
    return torch.tensor([0, 3 if bad else 0], **I32)


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("stride", [0, 8])
def test_key_weights(bad, stride):
    k = ddtree.KeyWeights(2, 3, 16, 10, stride, 0)
    q = torch.randn(2, 3, 16, 576, device="cuda").to(torch.bfloat16)
    a = (q, torch.zeros(10, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, stride, **I32), lengths(bad),
         torch.zeros(2, 3, 16, device="cuda"), 0.1)
    out = torch.full((2, stride), 5.0, device="cuda")
    k(*a, out=out)
    assert k.status() == (ddtree.STATUS_BAD_PREFIX if bad else 0)
    k(*a, out=out, node_idx=torch.tensor([[0, -1], [2, 3 if bad else 1]], **I32))
    assert k.status() == (ddtree.STATUS_BAD_PREFIX | ddtree.STATUS_BAD_NODE if bad else 0)
    assert bool((out == 5).all())


@pytest.mark.parametrize("bad", [False, True])
def test_block_summary(bad):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    s, c = ddtree.block_summary(torch.zeros(10, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, **I32),
                                lengths(bad), 16, max_prefix_len=0, workspace=ws)
    assert s.shape == (2, 0, 576) and c.shape == (2, 0)
    assert ddtree.read_device_status(ws) == (ddtree.STATUS_BAD_PREFIX if bad else 0)


@pytest.mark.parametrize("bad", [False, True])
def test_block_selector(bad):
    s = ddtree.BlockSelector(2, 3, 16, 0, 16, 4)
    q = torch.randn(2, 3, 16, 576, device="cuda").to(torch.bfloat16)
    got = s(q, torch.zeros(2, 0, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 0, device="cuda"), lengths(bad))
    assert bool((got == -1).all())
    assert s.status() == (ddtree.STATUS_BAD_PREFIX if bad else 0)


@pytest.mark.parametrize("bad", [False, True])
def test_evict(bad):
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    slots, weight, n, freed = ddtree.kv_evict(torch.zeros(2, 4, device="cuda"), torch.zeros(2, 4, **I32), lengths(bad),
                                              torch.tensor([2, 2], **I32), max_prefix_len=0, workspace=ws)
    assert n.tolist() == [0, 0]
    assert ddtree.read_device_status(ws) == (ddtree.STATUS_BAD_PREFIX if bad else 0)


@pytest.mark.parametrize("bad", [False, True])
def test_block_verifier(bad):
    """The tree alone."""
    v = ddtree.BlockVerifier(2, 2, 16, 10, 0, 16, 3)
    kv = torch.randn(10, 576, device="cuda").to(torch.bfloat16)
    q = torch.randn(2, 2, 16, 576, device="cuda").to(torch.bfloat16)
    idx = torch.full((2, 2, 3), -1, **I32)
    out, lse = v(q, kv, torch.zeros(2, 0, **I32), lengths(bad), torch.tensor([[-1, 0]] * 2, **I32),
                 torch.tensor([[1, 2], [3, 4]], **I32), idx, 0.1)
    assert v.status() == (ddtree.STATUS_BAD_PREFIX if bad else 0)
    assert float((out[:, 0].float() - kv[[1, 3], None, :512].float()).abs().max()) == 0     # its only key: weight 1
    assert bool(torch.isfinite(lse).all())
