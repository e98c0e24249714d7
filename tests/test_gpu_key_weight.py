"""Accumulated attention weights of the prefix keys (ddtree_kv_weight) against fp64 on the GPU.

Tolerance per key, from the arithmetic: the exponent sm_scale q.k - lse carries at most 36 accumulation
roundings of the dot product (one per 16-wide tensor-core step, each up to two units of 2^-24 of the sum of
|q_i k_i| because the adder may truncate) plus four roundings of s and lse themselves, and 2^x adds 2^-22; a
relative error of the exponential of at most e times that, and the sum over rows at most doubles it.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
SCALE = 1.0 / np.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def make(batch, lens, nodes, heads, seed=0, stride=None, pool=None, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = max(1, max(lens)) if stride is None else stride
    pool = sum(lens) + 7 if pool is None else pool
    order = torch.randperm(pool, generator=g, device="cuda")
    slot = torch.full((batch, stride), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        slot[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    kv = torch.randn(pool, 576, generator=g, device="cuda", dtype=torch.bfloat16)
    q = (amp * torch.randn(batch, nodes, heads, 576, generator=g, device="cuda")).to(torch.bfloat16)
    lse = 3.0 + torch.rand(batch, nodes, heads, generator=g, device="cuda")
    return dict(q=q, kv=kv, slot=slot, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=lse)


def reference(d, b, sel=None, decay=0.0, old=None):
    """(weights, tolerance) of request b in fp64."""
    n = int(d["lens"][b])
    nodes = list(range(d["q"].shape[1])) if sel is None else [t for t in sel if 0 <= t < d["q"].shape[1]]
    slots = d["slot"][b, :n].long()
    good = (slots >= 0) & (slots < d["kv"].shape[0])
    k = d["kv"][slots.clamp(0, d["kv"].shape[0] - 1)].double()
    w = torch.zeros(n, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(w)
    for t in nodes:
        lse = d["lse"][b, t].double()
        live = lse.abs() != float("inf")
        q, lse = d["q"][b, t].double()[live], lse[live]
        p = torch.exp(SCALE * (k @ q.T) - lse)
        mag = SCALE * (k.abs() @ q.abs().T)
        w += p.sum(1)
        tol += (p * (2 * 2.718 * (72 * mag + 4 * lse.abs()) * 2.0 ** -24 + 2.0 ** -21)).sum(1)
    w, tol = torch.where(good, w, 0.0), torch.where(good, tol, 0.0)
    if old is not None and decay:
        w = w + decay * old[b, :n].double()
        tol = tol + 2.0 ** -23 * w.abs()
    return w, tol


def check(d, out, sel=None, decay=0.0, old=None, before=None):
    for b in range(d["q"].shape[0]):
        n = int(d["lens"][b])
        w, tol = reference(d, b, None if sel is None else sel[b].tolist(), decay, old)
        err = (out[b, :n].double() - w).abs()
        assert bool((err <= tol + 1e-30).all()), (b, float((err / (tol + 1e-30)).max()))
        if before is not None:
            assert torch.equal(out[b, n:], before[b, n:])


CASES = [
    (1, [1], 1, 1), (1, [2], 9, 16), (2, [127, 0], 1, 16), (2, [128, 129], 5, 3), (3, [300, 1, 257], 9, 16),
    (1, [513], 65, 16), (1, [260], 3, 128), (1, [200], 128, 2), (2, [64, 700], 2, 200), (1, [140], 1, 1024),
    (9, [33 * i for i in range(9)], 4, 24), (1, [20000], 7, 16),
]


@pytest.mark.parametrize("batch,lens,nodes,heads", CASES)
def test_every_node(batch, lens, nodes, heads):
    d = make(batch, lens, nodes, heads, stride=max(lens) + 5)
    out = torch.full((batch, max(lens) + 5), 7.5, device="cuda")
    before = out.clone()
    k = ddtree.KeyWeights(batch, nodes, heads, d["kv"].shape[0], max(lens) + 5)
    got = k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, out=out)
    assert k.status() == 0
    check(d, got, before=before)
    again = k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, out=torch.full_like(out, 7.5))
    assert torch.equal(got, again)   # a fixed order of summation


@pytest.mark.parametrize("heads", [1, 16, 40])
def test_chosen_nodes_and_decay_in_place(heads):
    lens = [400, 90]
    d = make(2, lens, 9, heads, seed=3)
    sel = torch.tensor([[0, 2, 2, -1], [8, -1, 5, 1]], dtype=torch.int32, device="cuda")
    old = torch.rand(2, 400, device="cuda")
    acc = old.clone()
    k = ddtree.KeyWeights(2, 9, heads, d["kv"].shape[0], 400)
    k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, weight=acc, decay=0.75, node_idx=sel, out=acc)
    assert k.status() == 0
    check(d, acc, sel=sel, decay=0.75, old=old, before=old)


def test_bad_node_is_left_out_and_reported():
    d = make(1, [50], 4, 16, seed=4)
    sel = torch.tensor([[1, 4, -2, 3]], dtype=torch.int32, device="cuda")
    k = ddtree.KeyWeights(1, 4, 16, d["kv"].shape[0], 50)
    out = k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, node_idx=sel)
    assert k.status() == ddtree.STATUS_BAD_NODE
    check(d, out, sel=sel)


def test_bad_slots_lengths_and_rows_that_do_not_count():
    d = make(2, [300, 200], 6, 16, seed=5)
    d["slot"][0, 7], d["slot"][0, 130], d["slot"][1, 199] = -1, d["kv"].shape[0], 1 << 30
    d["lse"][0, 2] = float("-inf")           # an inactive node: its query may hold anything
    d["q"][0, 2] = float("nan")
    d["lse"][1, 5, 3] = float("inf")
    d["q"][1, 5, 3] = float("inf")
    out = torch.zeros(2, 300, device="cuda")
    k = ddtree.KeyWeights(2, 6, 16, d["kv"].shape[0], 300)
    k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, out=out)
    assert k.status() == ddtree.STATUS_BAD_SLOT
    check(d, out)
    lens = torch.tensor([-3, 1 << 20], dtype=torch.int32, device="cuda")
    d["slot"][1, 200:] = 0
    k(d["q"], d["kv"], d["slot"], lens, d["lse"], SCALE, out=out)
    assert k.status() & ddtree.STATUS_BAD_PREFIX
    d["lens"] = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    check(d, out)


def test_a_non_finite_key_row_stays_its_own():
    d = make(1, [200], 3, 16, seed=6)
    clean = ddtree.KeyWeights(1, 3, 16, d["kv"].shape[0], 200)
    want = clean(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE)
    d["kv"][int(d["slot"][0, 77]), 5] = float("nan")
    got = clean(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE)
    assert bool(torch.isnan(got[0, 77]))
    keep = torch.arange(200, device="cuda") != 77
    assert torch.equal(got[0, keep], want[0, keep])


def test_weights_of_a_verify_call_sum_to_its_rows():
    """Prefix weights plus the tree's own softmax mass are one per row."""
    from speculative_decoding_tree_05_gb300 import workloads as wl
    w = wl.make_workload("tiny", prefix=(777,), nodes=1, max_depth=0)
    d = wl.to_device(w, "cuda")
    v = ddtree.Verifier(1, 1, w.heads, w.pool_slots, w.slot_stride, w.max_prefix_len)
    _, lse = v(d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], d["tree_parent"], d["tree_slot_idx"], w.sm_scale)
    k = ddtree.KeyWeights(1, 1, w.heads, w.pool_slots, w.slot_stride, w.max_prefix_len)
    weight = k(d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], lse, w.sm_scale)
    own = d["kv_pool"][int(d["tree_slot_idx"][0, 0])].double()
    tail = torch.exp(w.sm_scale * (d["q"][0, 0].double() @ own) - lse[0, 0].double())
    total = weight[0, :777].double().sum() + tail.sum()
    assert abs(float(total) - w.heads) <= w.heads * 2e-3   # the verify lse is good to 1e-3


def test_other_stream_and_graph_replay():
    d = make(2, [300, 150], 5, 16, seed=8)
    k = ddtree.KeyWeights(2, 5, 16, d["kv"].shape[0], 300)
    out = torch.zeros(2, 300, device="cuda")
    want = k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    d["lens"][0] = 120       # new lengths in place
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0, :120], want[0, :120]) and not bool(out[0, 120:].any()) and torch.equal(out[1], want[1])


def test_chosen_nodes_in_a_graph():
    """The packed rows are made by a kernel of the same graph, which the scores follow as a dependent launch."""
    d = make(2, [700, 350], 9, 16, seed=9)
    sel = torch.tensor([[0, 2, 5], [1, -1, -1]], dtype=torch.int32, device="cuda")
    k = ddtree.KeyWeights(2, 9, 16, d["kv"].shape[0], 700)
    out = torch.zeros(2, 700, device="cuda")
    call = lambda: k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, node_idx=sel, out=out)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    sel.copy_(torch.tensor([[8, 3, -1], [4, 4, 0]], dtype=torch.int32, device="cuda"))
    d["q"].copy_(torch.randn(d["q"].shape, device="cuda").to(torch.bfloat16))
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    check(d, out, sel=sel)


def test_slots_behind_four_gigabytes():
    """Row offsets past 32 bits: the used rows are the last of a pool of 4.2 million."""
    rows = 4_200_000
    d = make(1, [500], 3, 16, seed=10)
    big = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
    n = d["kv"].shape[0]
    big[rows - n:] = d["kv"]
    d["kv"], d["slot"] = big, (d["slot"] + (rows - n)).contiguous()
    k = ddtree.KeyWeights(1, 3, 16, rows, 500)
    out = k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE)
    check(d, out)
    summary, scale = ddtree.block_summary(d["kv"], d["slot"], d["lens"], 64)
    small, small_scale = ddtree.block_summary(big[rows - n:].clone(), d["slot"] - (rows - n), d["lens"], 64)
    assert torch.equal(summary, small) and torch.equal(scale, small_scale)
    parent = torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda")
    tree = torch.tensor([[rows - 1, rows - 2, rows - 3]], dtype=torch.int32, device="cuda")
    idx = torch.arange(8, dtype=torch.int32, device="cuda").expand(1, 3, 8).contiguous()
    a = ddtree.BlockVerifier(1, 3, 16, rows, 500, 64, 8)(d["q"], big, d["slot"], d["lens"], parent, tree, idx, SCALE)
    b = ddtree.BlockVerifier(1, 3, 16, n, 500, 64, 8)(d["q"], big[rows - n:].clone(), d["slot"] - (rows - n), d["lens"],
                                                      parent, tree - (rows - n), idx, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_empty_prefixes():
    d = make(2, [0, 0], 3, 16, seed=11, stride=64)
    k = ddtree.KeyWeights(2, 3, 16, d["kv"].shape[0], 64)
    out = torch.full((2, 64), 3.0, device="cuda")
    k(d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE, out=out)
    assert k.status() == 0 and bool((out == 3.0).all())


def test_refusals():
    d = make(1, [64], 2, 16)
    k = ddtree.KeyWeights(1, 2, 16, d["kv"].shape[0], 64)
    a = (d["q"], d["kv"], d["slot"], d["lens"], d["lse"], SCALE)
    with pytest.raises(ValueError):
        k(d["q"].half(), *a[1:])
    with pytest.raises(ValueError):
        k(d["q"][..., :512], *a[1:])
    with pytest.raises(ValueError):
        k(d["q"].transpose(1, 2), *a[1:])
    with pytest.raises(ValueError):
        k(*a, out=torch.zeros(1, 64))
    with pytest.raises(ValueError):
        k(*a, node_idx=torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ddtree.DDTError):
        ddtree.KeyWeights(1, 0, 16, 10, 64)
