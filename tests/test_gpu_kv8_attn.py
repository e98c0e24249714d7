"""Verify attention over the 8-bit latent cache (ddtree_verify_attn_kv8) against fp64 on the GPU.

Tolerances, from the arithmetic.  A query value enters as two 8-bit parts: exactly, or where it is below 2^-10.8 of the
row's largest latent value with half a step of 2^-9 e, e being at most 1/224 of that value: 2^-17.8 of it.  A score adds at
most 40 partial sums, each rounded (up to two units of 2^-24) in the size of sum |q k|, and the steps from there to the
weight's exponent round three values of the size of score, log of the scale and reference (2^-23 each).  The
log-sum-exp moves by at most the largest of these, plus 2^-20 for the exponentials, sums and logarithms.  out: each weight
is cut to 8 bits (2^-8 of it at most; parts below e5m2's reach: 2^-21 of the largest weight times scale), the result rounded
to bf16 (2^-8), and the score error counts twice (in the weight and in their sum).
"""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import build_and_load, require_cuda

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def make(lens, nodes, heads, seed=0, amp=1.0, stride=None, tree="random", spread=0.0, extra=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = np.random.default_rng(seed)
    batch, stride = len(lens), max(lens) if stride is None else stride
    slots = sum(lens) + batch * nodes + extra
    order = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    slot = torch.full((batch, stride), 1 << 28, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        slot[b, :n] = order[at:at + n]
        at += n
    treeslot = order[at:at + batch * nodes].reshape(batch, nodes).contiguous()
    rows = torch.randn(slots, 576, generator=g, device="cuda")
    if spread:   # rows of very different sizes: their keys' scores stay comparable through the queries' rope part
        rows[:, :512] *= torch.exp2(torch.randint(-int(spread), int(spread) + 1, (slots, 1), generator=g, device="cuda").float())
    pool, scale = ddtree.kv8_pool(slots)
    ddtree.kv8_write(rows.to(torch.bfloat16), torch.arange(slots, dtype=torch.int32, device="cuda"), pool, scale)
    q = (amp * torch.randn(batch, nodes, heads, 576, generator=g, device="cuda")).to(torch.bfloat16)
    parent = np.full((batch, nodes), -1, np.int32)
    for i in range(1, nodes):
        parent[:, i] = i - 1 if tree == "chain" else 0 if tree == "star" else h.integers(0, i, batch)
    return dict(q=q, pool=pool, scale=scale, slot=slot, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                parent=torch.tensor(parent, device="cuda"), tree=treeslot, tree_len=None)


def call(d, library=None, **kw):
    batch, nodes, heads, _ = d["q"].shape
    v = ddtree.Kv8Verifier(batch, nodes, heads, d["pool"].shape[0], d["slot"].shape[1], library=library,
                           prefix_len_sum=d.get("sum", 0))
    out, lse = v(d["q"], d["pool"], d["scale"], d["slot"], d["lens"], d["parent"], d["tree"], d.get("sm", SCALE),
                 tree_len=d["tree_len"], **kw)
    return out, lse, v.status()


def values(d):
    latent = d["pool"][:, :512].view(torch.float8_e4m3fn).double()
    rope = d["pool"][:, 512:].contiguous().view(torch.bfloat16).double()
    return torch.cat([latent, rope], 1) * d["scale"].double()[:, None]


def check(d, out, lse, skip=(), requests=None):
    batch, nodes, heads, _ = d["q"].shape
    sm = d.get("sm", SCALE)
    table, parent = values(d), d["parent"].cpu().numpy()
    slots_n = d["pool"].shape[0]
    for b in range(batch) if requests is None else requests:
        L = min(max(int(d["lens"][b]), 0), d["slot"].shape[1])
        active = nodes if d["tree_len"] is None else min(max(int(d["tree_len"][b]), 0), nodes)
        if active < nodes:
            assert not bool(out[b, active:].any()) and bool((lse[b, active:] == -math.inf).all())
        prefix = d["slot"][b, :L].long()
        prefix = prefix[(prefix >= 0) & (prefix < slots_n)]
        for t in range(active):
            if (b, t) in skip:
                continue
            up, u, hops = [], t, 0
            while u >= 0:
                up.append(u)
                nxt = int(parent[b, u])
                if (u == 0 and nxt != -1) or (u > 0 and not 0 <= nxt < u):
                    break
                u = nxt
            mine = d["tree"][b, torch.tensor(up, device="cuda")].long()
            k = table[torch.cat([prefix, mine[(mine >= 0) & (mine < slots_n)]])]
            q = d["q"][b, t].double()
            if k.shape[0] == 0:
                assert not bool(out[b, t].any()) and bool((lse[b, t] == -math.inf).all())
                continue
            s = sm * (q @ k.T)
            ref_l = torch.logsumexp(s, -1)
            w = torch.softmax(s, -1)
            ref_o = w @ k[:, :512]
            both = abs(sm) * (q.abs() @ k.abs().T)
            key_scale = torch.log2(k[:, :512].abs().amax(1).clamp(min=2.0 ** -60)).abs().amax()
            near = s.abs().amax(1) + math.log(2.0) * (key_scale + 10)
            cut = abs(sm) * q[:, :512].abs().amax(1) * 2.0 ** -17.8 * k.abs().sum(1).amax()
            err = 80 * 2.0 ** -24 * both.amax(1) + 8 * 2.0 ** -23 * near + cut + 2.0 ** -20
            e = (lse[b, t].double() - ref_l).abs()
            assert bool((e <= err).all()), (b, t, float((e - err).max()))
            size = w @ k[:, :512].abs()
            big = (w * k[:, :512].abs().amax(1)).amax(1)[:, None] * k.shape[0] * 2.0 ** -20
            tol = 2.0 ** -8 * size + 2.0 ** -8 * ref_o.abs() + 2 * err[:, None] * size + big
            e = (out[b, t].double() - ref_o).abs()
            assert bool((e <= tol).all()), (b, t, float((e / tol).max()))


@pytest.mark.parametrize("lens,nodes,heads,tree", [
    ([0], 1, 1, "chain"), ([1], 1, 16, "chain"), ([63], 1, 16, "chain"), ([64], 2, 3, "random"), ([65], 9, 16, "random"),
    ([256], 9, 16, "chain"), ([700, 0, 1, 64], 33, 16, "random"), ([1000], 65, 16, "random"), ([300, 77], 128, 5, "random"),
    ([500], 128, 64, "chain"), ([130, 900], 5, 100, "random"), ([333], 3, 128, "star"), ([200], 2, 200, "chain"),
    ([4097, 5, 1300], 1, 16, "chain"), ([20000], 9, 16, "chain"), ([100], 1, 1024, "chain"), ([64, 128], 64, 1, "star")])
def test_sizes(lens, nodes, heads, tree):
    d = make(lens, nodes, heads, seed=nodes + heads, tree=tree)
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


@pytest.mark.parametrize("lens,heads,tree_len", [([700, 90, 3000], 16, [33, 1, 17]), ([64, 0, 500, 10], 100, [0, 1, 2, 33]),
                                                 ([900, 900], 3, [33, 32])])
def test_ragged_trees(lens, heads, tree_len):
    d = make(lens, 33, heads, seed=5)
    d["tree_len"] = torch.tensor(tree_len, dtype=torch.int32, device="cuda")
    for b, n in enumerate(tree_len):       # what is not active is not read
        d["q"][b, n:] = math.nan
        d["parent"][b, n:] = 77
        d["tree"][b, n:] = 1 << 29
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


@pytest.mark.parametrize("batch", [8, 32, 33])
def test_ragged_trees_over_long_prefixes(batch):
    """Trees' lengths that the division into units follows (up to 32 requests), among them trees of no node."""
    h = np.random.default_rng(batch)
    d = make([int(x) for x in h.integers(0, 12000 if batch == 8 else 2500, batch)], 33, 16, seed=batch)
    for tree_len in (h.integers(0, 34, batch), np.where(np.arange(batch) == 5, 33, 0), np.full(batch, 33), np.zeros(batch)):
        d["tree_len"] = torch.from_numpy(tree_len.astype(np.int32)).cuda()
        out, lse, st = call(d)
        assert st == 0
        check(d, out, lse, requests=[0, 4, 5, batch - 1])


@pytest.mark.parametrize("amp,sm", [(8.0, SCALE), (0.01, SCALE), (1.0, -0.2), (1.0, 0.0), (30.0, 0.5)])
def test_amplitudes_and_scales(amp, sm):
    d = make([900], 9, 16, seed=2, amp=amp)
    d["sm"] = sm
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


@pytest.mark.parametrize("spread", [4, 12, 30])
def test_rows_of_very_different_scales(spread):
    """The sums of weights and of weighted values have their own sizes where scales differ."""
    d = make([700, 100], 9, 16, seed=3, spread=spread, amp=2.0 ** -spread)
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


def test_any_positive_scale():
    d = make([500], 4, 16, seed=4)
    d["scale"] *= 0.3 + torch.rand(d["scale"].shape, device="cuda")
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


def test_queries_with_large_channels():
    d = make([600], 9, 16, seed=6)
    d["q"][..., 7] *= 50
    d["q"][..., 300] = 0
    d["q"][0, 2, 3] = 0
    d["q"][0, 3, 3, :512] = 0
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


def test_equal_scores_over_a_long_prefix():
    """Every key the same: the output is the key, the log-sum-exp the logarithm of their number."""
    d = make([30000], 1, 16, seed=7)
    d["pool"][:] = d["pool"][3].clone()
    d["scale"][:] = d["scale"][3].clone()
    out, lse, st = call(d)
    assert st == 0
    k = values(d)[0]
    assert bool(((out[0, 0].double() - k[:512]).abs() <= 2.0 ** -7 * k[:512].abs()).all())
    s = SCALE * (d["q"][0, 0].double() @ k)
    assert bool(((lse[0, 0].double() - s - math.log(30001)).abs() <= 1e-4).all())


def test_bad_slots_parents_and_lengths():
    d = make([300, 200, 100], 9, 16, seed=8, stride=310)
    n = d["pool"].shape[0]
    d["slot"][0, 5], d["slot"][0, 77], d["slot"][1, 199] = -1, n, -2 ** 31
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_SLOT
    check(d, out, lse)
    d["tree"][2, 4], d["tree"][2, 0] = n, -3
    d["parent"][1, 0], d["parent"][1, 3], d["parent"][2, 8] = 0, 3, 100
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_SLOT | ddtree.STATUS_BAD_PARENT
    check(d, out, lse)
    d = make([300, 200, 100], 9, 16, seed=9)
    d["lens"][1], d["lens"][2] = 301, -4
    d["slot"][1] = d["slot"][0]
    d["tree_len"] = torch.tensor([9, 10, -1], dtype=torch.int32, device="cuda")
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_PREFIX | ddtree.STATUS_BAD_TREE_LEN
    check(d, out, lse)


def test_no_visible_key():
    d = make([2, 0], 3, 16, seed=10)
    n = d["pool"].shape[0]
    d["slot"][0, :2] = n
    d["tree"][:] = n
    out, lse, st = call(d)
    assert st == ddtree.STATUS_BAD_SLOT
    assert not bool(out.any()) and bool((lse == -math.inf).all())


def test_values_that_are_not_finite_stay_where_they_belong():
    d = make([400, 300], 9, 16, seed=11, tree="star")
    d["q"][0, 2, 5, 100], d["q"][0, 3, 0, 570] = math.nan, math.inf
    tree_row = int(d["tree"][1, 4])
    d["scale"][tree_row] = math.nan
    d["pool"][tree_row] = 0
    out, lse, st = call(d)
    assert st == 0
    for b, t, h in ((0, 2, 5), (0, 3, 0)):
        assert bool(torch.isnan(out[b, t, h]).all()) and math.isnan(float(lse[b, t, h]))
    assert bool(torch.isnan(out[1, 4]).all()) and bool(torch.isnan(lse[1, 4]).all())
    fine = torch.isfinite(lse)
    assert int((~fine).sum()) == 2 + 16 and bool(torch.isfinite(out[fine]).all())
    check(d, out, lse, skip={(0, 2), (0, 3), (1, 4)})
    row = int(d["slot"][0, 17])                    # a prefix key: all of its request, and nothing else
    for bad in (math.nan, 0.0, -1.0, math.inf):
        d["scale"][row] = bad
        out, lse, st = call(d)
        assert st == 0 and bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
        check(d, out, lse, skip={(1, 4)}, requests=[1])


def test_any_slot_order_gives_the_same_bits():
    d = make([3000, 50], 9, 16, seed=12)
    out, lse, _ = call(d)
    order = torch.randperm(d["pool"].shape[0], device="cuda")
    e = dict(d)
    e["pool"], e["scale"] = torch.empty_like(d["pool"]), torch.empty_like(d["scale"])
    e["pool"][order], e["scale"][order] = d["pool"], d["scale"]
    e["slot"] = d["slot"].clone()
    for b in range(2):
        n = int(d["lens"][b])
        e["slot"][b, :n] = order[d["slot"][b, :n].long()].to(torch.int32)
    e["tree"] = order[d["tree"].long()].to(torch.int32)
    out2, lse2, st = call(e)
    assert st == 0 and torch.equal(out, out2) and torch.equal(lse, lse2)
    out3, lse3, _ = call(d)
    assert torch.equal(out, out3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("batch", [64, 1024, 1025, 1500])
def test_large_batches(batch):
    """Up to 1024 requests share their tiles out; more have a unit each."""
    h = np.random.default_rng(batch)
    lens = [int(x) for x in h.integers(0, 150, batch)]
    lens[3] = 2000 if batch < 2000 else 150
    d = make(lens, 2, 4, seed=13)
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse, requests=[0, 1, 2, 3, 40, 63, batch - 1])


@pytest.mark.parametrize("batch,most,nodes,heads,ragged", [(40, 20, 9, 64, False), (24, 500, 7, 128, True), (60, 90, 12, 24, True),
                                                           (170, 300, 1, 16, False), (9, 40, 40, 100, False)])
def test_many_groups_over_short_prefixes(batch, most, nodes, heads, ragged):
    """More groups than SMs and no request split: the units cut their query rows themselves."""
    h = np.random.default_rng(batch)
    d = make([most] + [int(x) for x in h.integers(0, most + 1, batch - 1)], nodes, heads, seed=batch, tree="chain" if nodes > 20 else "random")
    if ragged:
        n = h.integers(0, nodes + 1, batch)
        n[1] = nodes
        d["tree_len"] = torch.from_numpy(n.astype(np.int32)).cuda()
    d["q"][0, 0, heads - 1, 5], d["q"][2, 0, 0, 570] = math.nan, -math.inf
    d["q"][1, 0, 0] = 0
    d["q"][1, nodes - 1] *= 2.0 ** -100
    d["q"][3, 0, 0, 100] = 1000
    out, lse, st = call(d)
    assert st == 0
    active = d["tree_len"] is None or int(d["tree_len"][0]) > 0
    if active:
        assert bool(torch.isnan(out[0, 0, heads - 1]).all()) and bool(torch.isfinite(out[0, 0, :heads - 1]).all())
    check(d, out, lse, skip={(0, 0), (2, 0)}, requests=[0, 1, 2, 3, batch // 2, batch - 1])
    again, lse2, _ = call(d)
    assert torch.equal(out.nan_to_num(1.5), again.nan_to_num(1.5)) and torch.equal(lse.nan_to_num(1.5), lse2.nan_to_num(1.5))


@pytest.mark.parametrize("hint", [0, 1, 2500, 2 ** 31 - 1])
def test_length_hints(hint):
    d = make([2000, 500], 9, 16, seed=14, stride=60000)
    d["sum"] = hint
    out, lse, st = call(d)
    assert st == 0
    check(d, out, lse)


def test_equals_attention_over_the_rows_read_back():
    """The cache read back as bf16 rows gives the other verify call the same keys."""
    d = make([1500, 300], 9, 16, seed=15)
    out, lse, st = call(d)
    n = d["pool"].shape[0]
    rows = ddtree.kv8_read(d["pool"], d["scale"], torch.arange(n, dtype=torch.int32, device="cuda"))
    v = ddtree.Verifier(2, 9, 16, n, d["slot"].shape[1])
    out2, lse2 = v(d["q"], rows, d["slot"], d["lens"], d["parent"], d["tree"], SCALE)
    assert st == 0 and v.status() == 0
    assert float((lse - lse2).abs().max()) <= 1e-3          # (that call's partial scores are rounded to 16 bits)
    assert float((out.double() - out2.double()).norm() / out2.double().norm()) <= 2.0 ** -7


def test_slots_beyond_31_bits_of_bytes():
    slots = (1 << 31) // 640 + 5000
    d = make([3000], 4, 16, seed=16)
    n = d["pool"].shape[0]
    out, lse, _ = call(d)
    pool, scale = ddtree.kv8_pool(slots)
    pool[slots - n:], scale[slots - n:] = d["pool"], d["scale"]
    e = dict(d, pool=pool, scale=scale, slot=d["slot"] + (slots - n), tree=d["tree"] + (slots - n))
    out2, lse2, st = call(e)
    assert st == 0 and torch.equal(out, out2) and torch.equal(lse, lse2)


def test_captured_with_changing_lengths_and_two_graphs():
    d = make([3000, 900], 9, 16, seed=17)
    v = ddtree.Kv8Verifier(2, 9, 16, d["pool"].shape[0], 3000)
    w = ddtree.Kv8Verifier(2, 9, 16, d["pool"].shape[0], 3000)
    args = (d["q"], d["pool"], d["scale"], d["slot"], d["lens"], d["parent"], d["tree"], SCALE)
    v(*args)
    torch.cuda.synchronize()
    outs = [torch.zeros(2, 9, 16, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.zeros(2, 9, 16, device="cuda") for _ in range(2)]
    graphs = []
    for u, o, l in zip((v, w), outs, lses):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            u(*args, out=o, lse=l)
    side = torch.cuda.Stream()
    for lens in ([3000, 900], [10, 0], [2999, 901]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        d["slot"][1, 900] = d["slot"][0, 0]
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert v.status() == 0 and w.status() == 0
        assert torch.equal(outs[0], outs[1]) and torch.equal(lses[0], lses[1])
        check(d, outs[0], lses[0])


def test_on_a_stream_of_its_own_while_the_current_one_is_busy():
    d = make([2000], 9, 16, seed=18)
    out, lse, _ = call(d)
    v = ddtree.Kv8Verifier(1, 9, 16, d["pool"].shape[0], 2000)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got, got_l = v(d["q"], d["pool"], d["scale"], d["slot"], d["lens"], d["parent"], d["tree"], SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got, out) and torch.equal(got_l, lse)
    assert v.status(side) == 0


@pytest.mark.parametrize("lens,buffer", [([6000], 0), ([6000, 300], 1)])
def test_a_wait_that_runs_out(lens, buffer):
    """A test build keeps a score buffer back: the status word says so, and the next call is right."""
    build_and_load()
    hooks = build_and_load("testhooks")
    d = make(lens, 65, 128, seed=19)
    want, want_l, _ = call(d)
    hooks.ddtree_test_set_keep_back(buffer)
    try:
        _, _, st = call(d, library=hooks)
    finally:
        hooks.ddtree_test_set_keep_back(-1)
    assert st & ddtree.STATUS_TIMEOUT
    out, lse, st = call(d, library=hooks)
    assert st == 0 and torch.equal(out, want) and torch.equal(lse, want_l)
