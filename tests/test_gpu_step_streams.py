"""The 8-bit cache, its attention and the check of drafted tokens on streams of the caller's.

Outputs that a call makes belong to its stream, two calls with workspaces of their own run at once, and a call that is
captured while eager ones run gives what they give.
"""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
SCALE = 0.07
BUSY = 200_000_000   # cycles of the current stream: about a tenth of a second
B, T, H, V, LEN = 3, 9, 16, 5003, 700


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def inputs(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    slots = B * LEN + B * T
    order = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    pool, scale = ddtree.kv8_pool(slots)
    rows = torch.randn(slots, 576, generator=g, device="cuda").to(torch.bfloat16)
    ddtree.kv8_write(rows, torch.arange(slots, dtype=torch.int32, device="cuda"), pool, scale)
    up = torch.tensor([[-1] + [i // 2 for i in range(T - 1)]] * B, dtype=torch.int32, device="cuda")
    return dict(pool=pool, scale=scale, rows=rows, order=order, slot=order[:B * LEN].reshape(B, LEN).contiguous(),
                tree=order[B * LEN:].reshape(B, T).contiguous(), parent=up,
                lens=torch.tensor([LEN, 13, 300], dtype=torch.int32, device="cuda"),
                q=torch.randn(B, T, H, 576, generator=g, device="cuda").to(torch.bfloat16),
                logits=4 * torch.randn(B, T, V, generator=g, device="cuda"),
                tokens=torch.randint(0, V, (B, T), generator=g, device="cuda").to(torch.int32),
                uniform=torch.rand(B, T, generator=g, device="cuda"), heat=torch.ones(B, device="cuda"))


def calls(d):
    """name -> function of the stream, and of outputs, that returns the call's outputs"""
    attend, accept = ddtree.Kv8Verifier(B, T, H, d["pool"].shape[0], LEN), ddtree.TreeAcceptor(B, T, V)

    def read(s, out=(None,)):
        return (ddtree.kv8_read(d["pool"], d["scale"], d["order"], out=out[0], stream=s),)

    def verify(s, out=(None, None)):
        return attend(d["q"], d["pool"], d["scale"], d["slot"], d["lens"], d["parent"], d["tree"], SCALE, out=out[0],
                      lse=out[1], stream=s)

    def check(s, out=(None, None, None)):
        return accept(d["logits"], d["tokens"], d["parent"], d["uniform"], d["heat"], path=out[0], path_len=out[1],
                      next_token=out[2], stream=s)

    return {"kv8_read": read, "Kv8Verifier": verify, "TreeAcceptor": check}


NAMES = ["kv8_read", "Kv8Verifier", "TreeAcceptor"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads(name):
    d = inputs()
    call = calls(d)[name]
    want = [x.clone() for x in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full(x.shape, 3, dtype=x.dtype, device="cuda") for x in want for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    seen = [x.clone() for x in old]
    del old                              # free for later work of the current stream only
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(bool((x == 3).all()) for x in seen)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_two_at_once(name):
    """Calls with workspaces of their own, side by side on two streams, over and over."""
    d, e = inputs(1), inputs(2)
    first, second = calls(d)[name], calls(e)[name]
    want = [[x.clone() for x in f(None)] for f in (first, second)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[torch.zeros_like(x) for x in w] for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for f, s, out in zip((first, second), streams, got):
            f(s, out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, got) for a, b in zip(w, o))


@pytest.mark.parametrize("name", NAMES)
def test_a_captured_call_among_eager_ones(name):
    """One workspace, in order: eager, replayed, eager with other inputs in the same tensors, replayed."""
    d, e = inputs(3), inputs(4)
    call, other = calls(d)[name], calls(e)[name]
    want, fresh = [x.clone() for x in call(None)], [x.clone() for x in other(None)]
    out = [torch.zeros_like(x) for x in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(None, out)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(None), want))
        for x in out:
            x.zero_()
        graph.replay()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    for k in d:
        d[k].copy_(e[k])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, fresh))
    assert all(torch.equal(a, b) for a, b in zip(call(None), fresh))


def test_a_slot_that_stands_twice():
    """A prefix that lists a slot more than once weighs it as often, and reading it twice gives it twice."""
    d = inputs(5)
    d["slot"][0, 100:200] = d["slot"][0, 0]
    out, lse = calls(d)["Kv8Verifier"](None)
    pool, scale = d["pool"].clone(), d["scale"].clone()
    # the same rows in slots of their own
    n = pool.shape[0]
    more = torch.cat([pool, pool[d["slot"][0, 0].long()].expand(100, -1)]).contiguous()
    more_scale = torch.cat([scale, scale[d["slot"][0, 0].long()].expand(100)]).contiguous()
    slot = d["slot"].clone()
    slot[0, 100:200] = torch.arange(n, n + 100, dtype=torch.int32, device="cuda")
    v = ddtree.Kv8Verifier(B, T, H, n + 100, LEN)
    out2, lse2 = v(d["q"], more, more_scale, slot, d["lens"], d["parent"], d["tree"], SCALE)
    assert v.status() == 0 and torch.equal(out, out2) and torch.equal(lse, lse2)
    twice = ddtree.kv8_read(d["pool"], d["scale"], d["slot"][0])
    assert torch.equal(twice[100:200], twice[:1].expand(100, -1))
