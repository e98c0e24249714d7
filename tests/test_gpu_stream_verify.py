"""Verify calls and kv_compact on a stream of the caller's, making their own outputs while the current stream is busy."""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree, workloads as wl
from parity_util import build_and_load, require_cuda

pytestmark = pytest.mark.gpu
BUSY = 200_000_000   # cycles of the current stream: about a tenth of a second
NAMES = ["Verifier", "ragged", "verify_attn", "SparseVerifier", "kv_compact"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    build_and_load()


def call_of(name):
    """A function of the stream that returns the call's outputs."""
    w = wl.make_workload("tiny", prefix=(777,))
    d = wl.to_device(w, "cuda")
    a = (d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], d["tree_parent"], d["tree_slot_idx"], w.sm_scale)
    if name in ("Verifier", "ragged"):
        v = ddtree.Verifier(w.batch, w.nodes, w.heads, w.pool_slots, w.slot_stride, w.max_prefix_len)
        n = torch.full((w.batch,), w.nodes, dtype=torch.int32, device="cuda") if name == "ragged" else None
        return lambda s: v(*a, stream=s, tree_len=n)
    if name == "verify_attn":
        return lambda s: ddtree.verify_attn(*a, max_prefix_len=w.max_prefix_len, stream=s)
    if name == "SparseVerifier":
        v = ddtree.SparseVerifier(w.batch, w.nodes, w.heads, w.pool_slots, 64)
        idx = d["slot_idx"][:, None, :64].expand(w.batch, w.nodes, 64).contiguous()
        return lambda s: v(d["q"], d["kv_pool"], idx, w.sm_scale, stream=s)
    start = torch.arange(w.batch, dtype=torch.int64, device="cuda") * w.slot_stride
    to = torch.zeros(max(w.pool_slots, w.batch * w.slot_stride), 576, dtype=torch.bfloat16, device="cuda")[:w.pool_slots]
    return lambda s: (ddtree.kv_compact(d["kv_pool"], to, d["slot_idx"], d["prefix_len"], start, stream=s,
                                        max_prefix_len=w.max_prefix_len),)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_made_by_the_call(name):
    call = call_of(name)
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
    call = call_of(name)
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


def test_workspace_of_a_single_call_outlives_it():
    """verify_attn's workspace is dropped on return: work of the current stream must not get it while the call runs."""
    call = call_of("verify_attn")
    want = [x.clone() for x in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    got = call(s)
    for mib in (1, 2, 4, 8, 16):         # take whatever memory is free now, and overwrite it
        [torch.full((mib << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
