"""Tree attention over each node's own blocks (ddtree_verify_attn_blocks) against fp64 on the GPU.

Tolerances, from the arithmetic.  lse: each score carries at most 36 accumulation roundings (up to two units of
2^-24 of the sum of |q_i k_i| each), two of its scaling and one against the running max; the log-sum-exp moves by
at most the largest of them, plus 2^-21 for the exponentials, sums and logarithms.  out: each weight is rounded to
bf16 (half a step, 2^-8 of the value at most) and the result to
bf16 (half a step, 2^-8 of the value at most), so |error| <= 2^-8 (sum of weight |v|) + 2^-8 |out| plus the score
error times the same sum.
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


def make(lens, nodes, heads, block, topk, seed=0, amp=1.0, stride=None, lists="random"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = np.random.default_rng(seed)
    batch, stride = len(lens), max(1, max(lens)) if stride is None else stride
    pool = sum(lens) + batch * nodes + 5
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    slot = torch.full((batch, stride), 1 << 28, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        slot[b, :n] = order[at:at + n]
        at += n
    tree = order[at:at + batch * nodes].reshape(batch, nodes).contiguous()
    kv = torch.randn(pool, 576, generator=g, device="cuda").to(torch.bfloat16)
    q = (amp * torch.randn(batch, nodes, heads, 576, generator=g, device="cuda")).to(torch.bfloat16)
    parent = np.full((batch, nodes), -1, np.int32)
    for i in range(1, nodes):
        parent[:, i] = h.integers(0, i, batch)
    idx = np.full((batch, nodes, topk), -1, np.int32)
    for b, n in enumerate(lens):
        nb = -(-n // block)
        for t in range(nodes):
            m = min(topk, nb)
            if lists == "random":
                m = int(h.integers(0, m + 1)) if t % 3 == 2 else m
            pick = h.permutation(nb)[:m]
            idx[b, t, h.permutation(topk)[:m]] = pick      # any order, holes anywhere
    return dict(q=q, kv=kv, slot=slot, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                parent=torch.tensor(parent, device="cuda"), tree=tree, idx=torch.tensor(idx, device="cuda"), block=block)


def call(d, **kw):
    batch, nodes, heads, _ = d["q"].shape
    v = ddtree.BlockVerifier(batch, nodes, heads, d["kv"].shape[0], d["slot"].shape[1], d["block"], d["idx"].shape[2])
    out, lse = v(d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], d["idx"], SCALE, **kw)
    return out, lse, v.status()


def check(d, out, lse, skip=()):
    batch, nodes, heads, _ = d["q"].shape
    block = d["block"]
    idx, parent = d["idx"].cpu().numpy(), d["parent"].cpu().numpy()
    for b in range(batch):
        n = int(d["lens"][b])
        nb = -(-n // block)
        for t in range(nodes):
            if (b, t) in skip:
                continue
            blocks = sorted({int(x) for x in idx[b, t] if 0 <= x < nb})
            pos = [p for x in blocks for p in range(x * block, min(n, (x + 1) * block))]
            slots = d["slot"][b][torch.tensor(pos, dtype=torch.long, device="cuda")].long()
            slots = slots[(slots >= 0) & (slots < d["kv"].shape[0])]
            up, u = [], t
            while u >= 0:
                up.append(u)
                u = parent[b, u]
            slots = torch.cat([slots, d["tree"][b][torch.tensor(up, device="cuda")].long()])
            k, q = d["kv"][slots].double(), d["q"][b, t].double()
            s = SCALE * (q @ k.T)
            want_l = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            want = p @ k[:, :512]
            err_s = (SCALE * (q.abs() @ k.abs().T) * 72 + 3 * s.abs()).max() * 2.0 ** -24
            tol_l = err_s + 2.0 ** -21 * (1 + want_l.abs())
            assert bool(((lse[b, t].double() - want_l).abs() <= tol_l).all()), (b, t)
            mass = p @ k[:, :512].abs()
            tol = (2.0 ** -8 + 2 * 2.718 * err_s) * mass + 2.0 ** -8 * want.abs() + 1e-30
            err = (out[b, t].double() - want).abs()
            assert bool((err <= tol).all()), (b, t, float((err / tol).max()))


CASES = [
    ([1], 1, 1, 16, 1), ([16], 1, 16, 16, 1), ([63, 64, 65], 1, 16, 16, 4), ([300, 0, 17], 9, 16, 16, 5),
    ([1000, 640], 5, 3, 32, 12), ([1000], 33, 16, 64, 9), ([2049, 100], 7, 16, 128, 6), ([700], 3, 64, 64, 7),
    ([700, 130], 3, 128, 32, 9), ([500], 2, 100, 64, 4), ([400], 65, 1, 16, 7), ([400], 128, 2, 16, 3),
    ([9000], 4, 24, 16, 300), ([5000, 4000, 3000, 1], 13, 16, 64, 32), ([300], 1, 1024, 32, 4),
    ([40000], 6, 16, 16, 40),
]


@pytest.mark.parametrize("lens,nodes,heads,block,topk", CASES)
def test_against_fp64(lens, nodes, heads, block, topk):
    d = make(lens, nodes, heads, block, topk, seed=nodes + heads, stride=max(lens) + 3)
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)
    out2, lse2, _ = call(d)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("heads", [1, 16, 32, 33, 64])
@pytest.mark.parametrize("batch,topk,block", [(4, 60, 16), (16, 40, 32), (30, 9, 64), (3, 6, 128)])
def test_splits_with_and_without_keys(batch, topk, block, heads):
    """Requests of very different lengths share one choice of key splits: some splits hold no key."""
    lens = [[2600, 0, 40, 1, 63, 1500][b % 6] for b in range(batch)]
    d = make(lens, 1, heads, block, topk, seed=heads + topk, lists="all")
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)
    d["kv"][int(d["slot"][0, 2500])] = float("nan")    # in one split of one request
    out2, lse2, _ = call(d)
    reads = 2500 // block in d["idx"][0, 0].tolist()
    assert bool(torch.isnan(out2[0]).all()) == reads and bool(torch.isnan(lse2[0]).all()) == reads
    assert torch.equal(out2[1:], out[1:]) and torch.equal(lse2[1:], lse[1:])


@pytest.mark.parametrize("amp", [4.0, 16.0])
def test_large_scores_raise_the_running_max(amp):
    d = make([3000], 9, 16, 64, 20, seed=5, amp=amp)
    # scores that grow along the prefix: the max is raised again and again
    k = d["kv"][d["slot"][0].long()].float()
    ramp = torch.linspace(0.1, 2.0, 3000, device="cuda")[:, None]
    d["kv"][d["slot"][0].long()] = (k * 0.3 + ramp * d["q"][0, 0, 0].float() / amp).to(torch.bfloat16)
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


def test_very_low_scores_are_not_lost():
    d = make([640], 4, 16, 64, 6, seed=6)
    row = d["q"][0, 0, 0].float()
    d["q"][:] = row.to(torch.bfloat16)
    d["kv"][:] = (-4.0 * row + 0.05 * torch.randn_like(d["kv"].float())).to(torch.bfloat16)   # scores near -170 nats
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


def test_every_block_listed_is_verify_attention():
    lens = [777, 64, 130]
    d = make(lens, 9, 16, 64, 13, seed=7, lists="all")
    out, lse, _ = call(d)
    v = ddtree.Verifier(3, 9, 16, d["kv"].shape[0], 777)
    d["slot"][d["slot"] == 1 << 28] = 0
    want, want_l = v(d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], SCALE)
    assert float((out.float() - want).abs().max()) <= 2e-2 + 2.0 ** -8 * float(want.abs().max())
    assert float((lse - want_l).abs().max()) <= 1e-3


def test_repeats_and_bad_blocks():
    d = make([500], 5, 16, 32, 8, seed=8)
    d["idx"][0, 0] = torch.tensor([3, 3, 3, -1, 7, 7, 15, 15], dtype=torch.int32, device="cuda")
    d["idx"][0, 1] = torch.tensor([16, -2, 1 << 30, -1, 2, 0, 0, 1], dtype=torch.int32, device="cuda")
    d["idx"][0, 2] = -1
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_BLOCK
    check(d, out, lse)


def test_bad_slots():
    d = make([500], 5, 16, 32, 8, seed=9, lists="all")
    d["slot"][0, 5], d["slot"][0, 77], d["slot"][0, 499] = -1, 1 << 30, d["kv"].shape[0]
    d["slot"][0, 128:192] = -9
    out, lse, st = call(d)
    assert st in (0, ddtree.STATUS_BAD_SLOT)
    check(d, out, lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_non_finite_row_reaches_only_the_nodes_that_read_it(value):
    d = make([640], 8, 16, 64, 4, seed=10)
    idx = np.array([[0, 1, 2, 3], [0, 2, 4, 6], [5, 6, 7, 8], [1, 3, 5, 7], [4, 4, 4, 9], [0, 1, 8, 9], [2, 3, 4, 5],
                    [6, 7, 8, 9]], np.int32)
    d["idx"] = torch.tensor(idx[None], device="cuda")
    d["kv"][int(d["slot"][0, 64 * 4 + 11]), 100] = value    # block 4
    out, lse, _ = call(d)
    readers = [t for t in range(8) if 4 in idx[t]]
    for t in readers:
        assert not bool(torch.isfinite(out[0, t, :, 100]).any())
    check(d, out, lse, skip={(0, t) for t in readers})


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [1, 16, 64])
def test_a_non_finite_query_row_spoils_only_itself(value, heads):
    d = make([640], 8, heads, 64, 4, seed=15, lists="random")
    d["q"][0, 2, heads // 2, 7] = value
    d["q"][0, 5] = value
    out, lse, st = call(d)
    assert st == 0
    assert not bool(torch.isfinite(out[0, 5]).any()) and not bool(torch.isfinite(out[0, 2, heads // 2]).any())
    others = [h for h in range(heads) if h != heads // 2]
    assert bool(torch.isfinite(out[0, 2, others]).all()) and bool(torch.isfinite(lse[0, 2, others]).all())
    check(d, out, lse, skip={(0, 2), (0, 5)})
    # beside a non-finite key row, which still reaches only its readers
    d["kv"][int(d["slot"][0, 64 * 4 + 11]), 100] = value
    out, lse, _ = call(d)
    idx = d["idx"][0].cpu().numpy()
    readers = [t for t in range(8) if 4 in idx[t]]
    assert readers and len(readers) < 8
    for t in readers:
        assert not bool(torch.isfinite(out[0, t, :, 100]).any())
    check(d, out, lse, skip={(0, t) for t in readers} | {(0, 2), (0, 5)})


def test_a_non_finite_tree_row_reaches_only_its_descendants():
    d = make([300], 6, 16, 64, 3, seed=12)
    d["parent"] = torch.tensor([[-1, 0, 0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    d["kv"][int(d["tree"][0, 1])] = float("nan")
    out, lse, st = call(d)
    assert st == 0
    for t in (1, 3, 5):
        assert bool(torch.isnan(out[0, t]).all()) and bool(torch.isnan(lse[0, t]).all())
    check(d, out, lse, skip={(0, 1), (0, 3), (0, 5)})


def test_bad_parents_and_tree_slots():
    d = make([300], 6, 16, 64, 3, seed=13)
    d["parent"] = torch.tensor([[-1, 0, 1, 5, 3, -2]], dtype=torch.int32, device="cuda")
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_PARENT
    # a bad link ends the walk: node 3 sees itself, node 4 node 3 and itself, node 5 itself
    d["parent"] = torch.tensor([[-1, 0, 1, -1, 3, -1]], dtype=torch.int32, device="cuda")
    check(d, out, lse)
    d["parent"] = torch.tensor([[-1, 0, 1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    keep = d["tree"].clone()
    d["tree"][0, 2] = d["kv"].shape[0] + 5
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_SLOT
    d["tree"] = keep
    check(d, out, lse, skip={(0, t) for t in (2, 3, 4, 5)})


@pytest.mark.parametrize("nodes", [1, 2, 65, 128])
def test_trees_alone(nodes):
    """No prefix: the tree rows are the only keys; a chain of them, and none at all when its slots are bad."""
    d = make([0], nodes, 16, 16, 2, seed=14)
    d["parent"] = torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda")[None].contiguous()
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)
    d["tree"][:] = -1
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_SLOT and not bool(out.any()) and bool((lse == float("-inf")).all())


def test_slot_layout_graph_and_stream():
    d = make([900, 300], 9, 16, 64, 6, seed=11)
    out, lse, _ = call(d)
    # the same logical data in another slot order
    perm = torch.randperm(d["kv"].shape[0], device="cuda")
    e = dict(d)
    e["kv"] = torch.empty_like(d["kv"])
    e["kv"][perm] = d["kv"]
    e["slot"] = torch.where(d["slot"] < 1 << 28, perm[d["slot"].clamp(max=perm.numel() - 1).long()].to(torch.int32), d["slot"])
    e["tree"] = perm[d["tree"].long()].to(torch.int32)
    out2, lse2, _ = call(e)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    v = ddtree.BlockVerifier(2, 9, 16, d["kv"].shape[0], 900, 64, 6)
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v(d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], d["idx"], SCALE, out=o, lse=l)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    s = torch.cuda.Stream()
    o.zero_()
    torch.cuda.synchronize()
    v(d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], d["idx"], SCALE, out=o, lse=l, stream=s)
    s.synchronize()
    assert torch.equal(o, out)


def test_refusals():
    d = make([100], 2, 16, 16, 3)
    with pytest.raises(ddtree.DDTError):
        ddtree.BlockVerifier(1, 2, 16, 100, 100, 48, 3)
    with pytest.raises(ddtree.DDTError):
        ddtree.BlockVerifier(1, 2, 16, 100, 100, 16, 0)
    v = ddtree.BlockVerifier(1, 2, 16, d["kv"].shape[0], 100, 16, 3)
    a = [d["q"], d["kv"], d["slot"], d["lens"], d["parent"], d["tree"], d["idx"], SCALE]
    for i, bad in ((0, d["q"].half()), (1, d["kv"][:, :512]), (6, d["idx"][..., :2].contiguous()), (6, d["idx"].long())):
        b = list(a)
        b[i] = bad
        with pytest.raises(ValueError):
            v(*b)
    with pytest.raises(ValueError):
        v(*a, out=torch.empty(1, 2, 16, 512, device="cuda"))
