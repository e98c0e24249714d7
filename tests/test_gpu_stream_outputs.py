"""Calls on a stream of the caller's that make their own outputs, while the current stream is kept busy.

The outputs belong to the call's stream: no fill on the current stream may come after the kernels, and no memory may be
taken that earlier work of the current stream still reads.
"""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
SCALE = 0.07
BUSY = 200_000_000   # cycles of the current stream: about a tenth of a second


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def inputs():
    g = torch.Generator(device="cuda").manual_seed(0)
    n, nodes, heads = 1000, 5, 16
    kv = torch.randn(n + nodes, 576, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, nodes, heads, 576, generator=g, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=q, kv=kv, slot=torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous(), lens=i32([n]),
                lse=torch.full((1, nodes, heads), 4.0, device="cuda"), weight=torch.rand(1, n, generator=g, device="cuda"),
                keep=i32([300]), parent=i32([[-1, 0, 1, 2, 3]]), tree=i32([[n + t for t in range(nodes)]]),
                idx=torch.arange(8, dtype=torch.int32, device="cuda").expand(1, nodes, 8).contiguous())


def calls(d):
    """name -> (function of the stream that returns the call's outputs)"""
    n = d["kv"].shape[0]
    weigh = ddtree.KeyWeights(1, 5, 16, n, 1000)
    select = ddtree.BlockSelector(1, 5, 16, 1000, 64, 8)
    attend = ddtree.BlockVerifier(1, 5, 16, n, 1000, 64, 8)
    summary, scale = ddtree.block_summary(d["kv"], d["slot"], d["lens"], 64)
    return {
        "KeyWeights": lambda s: (weigh(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, stream=s),),
        "kv_evict": lambda s: ddtree.kv_evict(d["weight"], d["slot"], d["lens"], d["keep"], 4, 8, stream=s),
        "block_summary": lambda s: ddtree.block_summary(d["kv"], d["slot"], d["lens"], 64, stream=s),
        "BlockSelector": lambda s: (select(d["q"], summary, scale, d["lens"], stream=s),),
        "BlockVerifier": lambda s: attend(d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], d["idx"], SCALE,
                                          stream=s),
    }


NAMES = ["KeyWeights", "kv_evict", "block_summary", "BlockSelector", "BlockVerifier"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_made_by_the_call(name):
    d = inputs()
    call = calls(d)[name]
    want = [x.clone() for x in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads(name):
    d = inputs()
    call = calls(d)[name]
    sizes = [(x.shape, x.dtype) for x in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full(shape, 3, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    seen = [x.clone() for x in old]
    del old                              # free for later work of the current stream only
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(bool((x == 3).all()) for x in seen)
    del got
