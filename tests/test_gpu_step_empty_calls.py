"""A call without rows or requests reports nothing, whatever the call before it on the same workspace has reported."""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def empty(*shape, dtype=torch.int32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def test_rows():
    pool, scale = ddtree.kv8_pool(10)
    rows, slots = torch.ones(2, 576, dtype=torch.bfloat16, device="cuda"), torch.tensor([3, 10], dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ddtree.kv8_write(rows, slots, pool, scale, workspace=ws)
    assert ddtree.read_device_status(ws) == ddtree.STATUS_BAD_SLOT
    ddtree.kv8_write(rows[:0], slots[:0], pool, scale, workspace=ws)
    assert ddtree.read_device_status(ws) == 0
    ddtree.kv8_read(pool, scale, slots, workspace=ws)
    assert ddtree.read_device_status(ws) == ddtree.STATUS_BAD_SLOT
    ddtree.kv8_read(pool, scale, slots[:0], workspace=ws)
    assert ddtree.read_device_status(ws) == 0


def test_attention_without_requests():
    v = ddtree.Kv8Verifier(0, 9, 16, 10, 64)
    v.workspace[:] = 255
    pool, scale = ddtree.kv8_pool(10)
    out, lse = v(empty(0, 9, 16, 576, dtype=torch.bfloat16), pool, scale, empty(0, 64), empty(0), empty(0, 9), empty(0, 9), 0.1)
    assert v.status() == 0 and out.shape == (0, 9, 16, 512) and lse.shape == (0, 9, 16)


def test_drafted_tokens_without_requests():
    a = ddtree.TreeAcceptor(0, 9, 100)
    a.workspace[:] = 255
    path, length, token = a(empty(0, 9, 100, dtype=torch.bfloat16), empty(0, 9), empty(0, 9), empty(0, 9, dtype=torch.float32),
                            empty(0, dtype=torch.float32))
    assert a.status() == 0 and path.shape == (0, 9) and length.shape == token.shape == (0,)
