"""The operators in the order a serving step uses them, each fed by the one before."""
import numpy as np
import pytest
import torch

import oracle
from parity_util import LSE_MAX, OUT_MAX, require_cuda
from speculative_decoding_tree_05_gb300 import ddtree, workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def batch():
    w = wl.make_workload("tiny", batch=3, prefix=("list", 3000, 700, 1500), nodes=9, heads=16, pool_slots=16384)
    return w, wl.to_device(w, "cuda")


def verify(w, d, slot_idx, prefix_len):
    v = ddtree.Verifier(w.batch, w.nodes, w.heads, w.pool_slots, slot_idx.shape[1])
    return v(d["q"], d["kv_pool"], slot_idx, prefix_len, d["tree_parent"], d["tree_slot_idx"], w.sm_scale)


def test_weigh_evict_compact_verify():
    """verify -> weights of the accepted nodes -> eviction -> compaction; the next verify sees the kept keys only."""
    w, d = batch()
    stride = d["slot_idx"].shape[1]
    _, lse = verify(w, d, d["slot_idx"], d["prefix_len"])
    accepted = torch.tensor([[0, 1, 3], [0, 2, -1], [0, -1, -1]], dtype=torch.int32, device="cuda")
    weigh = ddtree.KeyWeights(w.batch, w.nodes, w.heads, w.pool_slots, stride)
    weight = weigh(d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], lse, w.sm_scale, node_idx=accepted)
    weight = weigh(d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], lse, w.sm_scale, weight=weight, decay=0.5,
                   node_idx=accepted, out=weight)
    assert weigh.status() == 0
    keep = (d["prefix_len"] // 3).to(torch.int32)
    slots, kept, length, freed = ddtree.kv_evict(weight, d["slot_idx"], d["prefix_len"], keep, sink=4, recent=32)
    assert torch.equal(length, keep)
    for b in range(w.batch):
        n, m = int(d["prefix_len"][b]), int(length[b])
        both = torch.cat([slots[b, :m], freed[b, :n - m]]).sort().values
        assert torch.equal(both, d["slot_idx"][b, :n].sort().values)     # every slot once: kept or freed
        mid = d["slot_idx"][b, 4:n - 32]
        gone = torch.isin(mid, freed[b, :n - m])
        assert float(weight[b, 4:n - 32][gone].max()) <= float(kept[b, 4:m - 32].min())
    out, lse2 = verify(w, d, slots, length)
    # the oracle on the kept keys: a request cut to them is the same request with a shorter prefix
    pool = d["kv_pool"].view(torch.int16).cpu().numpy().view(np.uint16)
    ref_o, ref_l, st = oracle.verify_attn(d["q"].view(torch.int16).cpu().numpy().view(np.uint16), pool,
                                          slots.cpu().numpy(), length.cpu().numpy(), d["tree_parent"].cpu().numpy(),
                                          d["tree_slot_idx"].cpu().numpy(), w.sm_scale)
    assert st == 0
    assert np.abs(out.cpu().numpy().reshape(ref_o.shape) - ref_o).max() <= OUT_MAX
    assert np.abs(lse2.cpu().numpy().reshape(ref_l.shape) - ref_l).max() <= LSE_MAX
    # the freed rows may be overwritten, and the kept ones moved together
    for b in range(w.batch):
        d["kv_pool"][freed[b, :int(d["prefix_len"][b]) - int(length[b])].long()] = float("nan")
    free = np.ones(w.pool_slots, bool)
    free[0] = False
    free[w.tree_slot_idx.reshape(-1)] = False
    start = []
    for m in length.tolist():   # the lowest run of m slots that holds no tree row
        s = next(x for x in range(1, w.pool_slots - m) if free[x:x + m].all())
        free[s:s + m] = False
        start.append(s)
    start = torch.tensor(start, dtype=torch.int64, device="cuda")
    moved = torch.zeros_like(d["kv_pool"])
    moved[d["tree_slot_idx"].long()] = d["kv_pool"][d["tree_slot_idx"].long()]
    new = ddtree.kv_compact(d["kv_pool"], moved, slots, length, start)
    e = dict(d, kv_pool=moved)
    out3, lse3 = verify(w, e, new, length)
    assert torch.equal(out3, out) and torch.equal(lse3, lse2)


@pytest.mark.parametrize("block", [16, 64])
def test_summarise_select_attend(block):
    """summary -> selection -> attention over the selection, in one captured graph; with every block selected it is
    verify attention."""
    w, d = batch()
    stride = d["slot_idx"].shape[1]
    n = -(-stride // block)
    want, want_l = verify(w, d, d["slot_idx"], d["prefix_len"])
    pick = ddtree.BlockSelector(w.batch, w.nodes, w.heads, stride, block, n)
    attend = ddtree.BlockVerifier(w.batch, w.nodes, w.heads, w.pool_slots, stride, block, n)
    summary, scale = ddtree.block_summary(d["kv_pool"], d["slot_idx"], d["prefix_len"], block)
    idx = pick(d["q"], summary, scale, d["prefix_len"])
    out, lse = attend(d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], d["tree_parent"], d["tree_slot_idx"], idx,
                      w.sm_scale)
    assert attend.status() == 0
    assert float((out.float() - want).abs().max()) <= OUT_MAX + 2.0 ** -8 * float(want.abs().max())
    assert float((lse - want_l).abs().max()) <= LSE_MAX
    # a narrower selection, captured with its summary update and replayed after the pool has changed
    few = ddtree.BlockSelector(w.batch, w.nodes, w.heads, stride, block, 6, first=1, last=1)
    narrow = ddtree.BlockVerifier(w.batch, w.nodes, w.heads, w.pool_slots, stride, block, 6)
    idx6 = torch.zeros(w.batch, w.nodes, 6, dtype=torch.int32, device="cuda")
    o6, l6 = torch.zeros_like(out), torch.zeros_like(lse)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def step():
        ddtree.block_summary(d["kv_pool"], d["slot_idx"], d["prefix_len"], block, summary=summary, scale=scale, workspace=ws)
        few(d["q"], summary, scale, d["prefix_len"], out=idx6)
        narrow(d["q"], d["kv_pool"], d["slot_idx"], d["prefix_len"], d["tree_parent"], d["tree_slot_idx"], idx6,
               w.sm_scale, out=o6, lse=l6)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    d["kv_pool"].copy_(torch.randn(d["kv_pool"].shape, device="cuda").to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    got = o6.clone(), l6.clone(), idx6.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], o6) and torch.equal(got[1], l6) and torch.equal(got[2], idx6)
    assert bool((idx6[:, :, 0] == 0).all())      # the first block is always read
    # node by node in fp64
    for b, t in ((0, 0), (1, 4), (2, 8)):
        L = int(d["prefix_len"][b])
        pos = [p for x in idx6[b, t].tolist() if x >= 0 for p in range(x * block, min(L, (x + 1) * block))]
        up, u = [], t
        while u >= 0:
            up.append(u)
            u = int(d["tree_parent"][b, u])
        rows = torch.cat([d["slot_idx"][b][torch.tensor(pos, device="cuda")], d["tree_slot_idx"][b][torch.tensor(up, device="cuda")]])
        k = d["kv_pool"][rows.long()].double()
        s = w.sm_scale * (d["q"][b, t].double() @ k.T)
        ref = torch.softmax(s, -1) @ k[:, :512]
        assert float((o6[b, t].double() - ref).abs().max()) <= 2.0 ** -7 * float(k.abs().max())
        assert float((l6[b, t].double() - torch.logsumexp(s, -1)).abs().max()) <= 1e-4
