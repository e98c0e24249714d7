"""Block summaries and block selection against their definitions, exactly (integers and fixed fp32 roundings)."""
import numpy as np
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


def pool_of(lens, seed=0, extra=9, heavy=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool, stride = sum(lens) + extra, max(lens)
    order = torch.randperm(pool, generator=g, device="cuda")
    slot = torch.full((len(lens), stride), 1 << 29, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        slot[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    kv = torch.randn(pool, 576, generator=g, device="cuda")
    if heavy:   # values over many binades: a plain fp32 sum would lose the small ones
        kv = kv * torch.exp2(torch.randint(-20, 21, kv.shape, generator=g, device="cuda").float())
    return kv.to(torch.bfloat16), slot, torch.tensor(lens, dtype=torch.int32, device="cuda")


def plain_summary(kv, slots):
    """One block's (integers, scale) from its rows' slots, in fp64 up to the mean."""
    slots = slots[(slots >= 0) & (slots < kv.shape[0])]
    if not len(slots):
        return torch.zeros(576, dtype=torch.float32), 0.0
    mean = (kv[slots.long()].double().sum(0) / len(slots)).float().cpu()
    scale = mean.abs().max() * torch.tensor(np.float32(1) / np.float32(127))
    if not torch.isfinite(scale):
        return torch.zeros(576, dtype=torch.float32), float("nan")
    if scale == 0:
        return torch.zeros(576, dtype=torch.float32), 0.0
    return torch.round(mean / scale).clamp(-127, 127), float(scale)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("heavy", [False, True])
def test_summary(block, heavy):
    lens = [1, 15, 16, 17, 129, 500, 0 + 1]
    kv, slot, n = pool_of(lens, seed=block, heavy=heavy)
    nb = -(-max(lens) // block)
    summary = torch.full((len(lens), nb, 576), 99.0, dtype=torch.bfloat16, device="cuda")
    scale = torch.full((len(lens), nb), 99.0, device="cuda")
    ddtree.block_summary(kv, slot, n, block, summary=summary, scale=scale)
    for b, L in enumerate(lens):
        for j in range(nb):
            if j * block >= L:
                assert bool((summary[b, j] == 99).all()) and float(scale[b, j]) == 99
                continue
            want, s = plain_summary(kv, slot[b, j * block:min(L, (j + 1) * block)])
            assert float(scale[b, j]) == s
            assert torch.equal(summary[b, j].float().cpu(), want)


@pytest.mark.parametrize("block", [16, 64, 128])
def test_summary_of_many_blocks(block):
    """Enough blocks that every stage buffer is used many times over."""
    lens = [60000, 9000, 31]
    kv, slot, n = pool_of(lens, seed=block)
    summary, scale = ddtree.block_summary(kv, slot, n, block)
    for b, L in enumerate(lens):
        whole = L // block * block
        mean = kv[slot[b, :whole].long()].double().reshape(-1, block, 576).mean(1).float()
        want = mean.abs().amax(-1) * (torch.ones((), device="cuda") / torch.full((), 127.0, device="cuda"))
        assert torch.equal(scale[b, :L // block], want)
        assert torch.equal(summary[b, :L // block].float(), torch.round(mean / want[:, None]).clamp(-127, 127))


def test_summary_update_after_a_step():
    lens = [200, 64, 65, 33]
    kv, slot, n = pool_of(lens, seed=9)
    summary, scale = ddtree.block_summary(kv, slot, n, 64)
    kv2 = torch.randn_like(kv.float()).to(torch.bfloat16)
    s2, c2 = summary.clone(), scale.clone()
    start = torch.tensor([190, 64, 64, -5], dtype=torch.int32, device="cuda")
    ddtree.block_summary(kv2, slot, n, 64, from_len=start, summary=s2, scale=c2)
    full, fscale = ddtree.block_summary(kv2, slot, n, 64)
    for b, first in enumerate([2, 1, 1, 0]):
        nb = -(-lens[b] // 64)
        assert torch.equal(s2[b, :first], summary[b, :first]) and torch.equal(c2[b, :first], scale[b, :first])
        assert torch.equal(s2[b, first:nb], full[b, first:nb]) and torch.equal(c2[b, first:nb], fscale[b, first:nb])


def test_summary_of_bad_slots_and_values():
    kv, slot, n = pool_of([256], seed=2)
    slot[0, 3], slot[0, 70] = -1, kv.shape[0]
    slot[0, 128:192] = -2
    kv[int(slot[0, 200]), 7] = float("inf")
    kv[slot[0, 64:128].clamp(0, kv.shape[0] - 1).long()] = 0
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    summary, scale = ddtree.block_summary(kv, slot, n, 64, workspace=ws)
    assert ddtree.read_device_status(ws) == ddtree.STATUS_BAD_SLOT
    for j in range(4):
        want, s = plain_summary(kv, slot[0, j * 64:(j + 1) * 64])
        assert torch.equal(summary[0, j].float().cpu(), want), j
        got = float(scale[0, j])
        assert got == s or (np.isnan(got) and np.isnan(s)), j


def plain_select(q, summary, scale, n, topk, first, last):
    """Blocks of one node, ascending: q [H, 576] bf16, summary [n, 576], scale [n] (numpy, fp32 roundings)."""
    qf = q.float().cpu().numpy()
    amax = np.abs(qf).max(1)
    with np.errstate(all="ignore"):
        qs = (amax * (np.float32(1) / np.float32(127))).astype(np.float32)
        ok = np.isfinite(amax)
        qi = np.where((qs > 0)[:, None] & ok[:, None], np.clip(np.rint(qf / qs[:, None]), -127, 127), 0)
        dots = (qi.astype(np.float64) @ summary.float().cpu().numpy().astype(np.float64).T).astype(np.float32)
        per = np.where(ok[:, None], dots * qs[:, None], -np.inf).astype(np.float32)
        score = per.max(0) * scale.cpu().numpy().astype(np.float32)
    at = np.arange(n)
    key = np.where(np.isnan(score), -np.inf, score.astype(np.float64)) + 0.0
    held = (at < first) | (at >= n - last)
    order = np.lexsort((at, np.where(held, 0.0, -key), ~held))
    best = np.sort(order[:topk])
    return np.concatenate([best, np.full(topk - len(best), -1)])


def select_case(batch, lens, nodes, heads, block, topk, first, last, seed=0, tweak=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-max(lens) // block)
    q = torch.randn(batch, nodes, heads, 576, generator=g, device="cuda").to(torch.bfloat16)
    mean = torch.randn(batch, nb, 576, generator=g, device="cuda")
    scale = mean.abs().amax(-1) / 127
    summary = torch.round(mean / scale[..., None]).to(torch.bfloat16)
    if tweak:
        tweak(q, summary, scale)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s = ddtree.BlockSelector(batch, nodes, heads, max(lens), block, topk, first=first, last=last)
    got = s(q, summary, scale, n).cpu().numpy()
    assert s.status() == 0
    for b in range(batch):
        m = -(-lens[b] // block)
        for t in range(nodes):
            want = plain_select(q[b, t], summary[b, :m], scale[b, :m], m, topk, first, last)
            assert np.array_equal(got[b, t], want), (b, t, got[b, t], want)


@pytest.mark.parametrize("batch,lens,nodes,heads,block,topk,first,last", [
    (1, [1], 1, 1, 16, 1, 0, 0), (1, [5000], 3, 16, 16, 8, 0, 1), (2, [2048, 100], 9, 16, 64, 4, 1, 2),
    (1, [9000], 2, 3, 16, 40, 0, 0), (1, [4097], 5, 24, 32, 17, 2, 2), (1, [4096], 2, 128, 32, 32, 1, 1),
    (1, [3000], 2, 300, 32, 9, 0, 0), (1, [3000], 2, 1024, 64, 9, 0, 0), (3, [1, 17, 40000], 4, 16, 16, 300, 0, 0),
    (1, [2000], 9, 40, 32, 11, 0, 0), (1, [2000], 40, 7, 32, 11, 0, 0), (1, [900], 3, 72, 16, 7, 0, 0),
    (2, [640, 64], 65, 16, 64, 20, 0, 0), (1, [300], 4, 16, 16, 3, 5, 5), (1, [280000], 1, 2, 16, 64, 1, 4),
])
def test_select(batch, lens, nodes, heads, block, topk, first, last):
    select_case(batch, lens, nodes, heads, block, topk, first, last)


def test_select_ties_take_the_lowest_blocks():
    def tweak(q, summary, scale):
        summary[:, 10:] = summary[:, 3:4]
        scale[:, 10:] = scale[:, 3:4]
    select_case(1, [6400], 4, 16, 64, 37, 0, 0, tweak=tweak)

    def zeros(q, summary, scale):
        summary.zero_()
        scale.zero_()
    select_case(1, [6400], 2, 16, 64, 30, 0, 3, tweak=zeros)


def test_select_non_finite_values():
    def tweak(q, summary, scale):
        q[0, 0, 3, 5] = float("nan")
        q[0, 1, :, 0] = float("inf")     # no head left: every block ranks the same
        q[0, 2, 2] = 0
        scale[0, 7] = float("nan")
        summary[0, 7] = 0
    select_case(1, [3200], 4, 16, 32, 20, 0, 1, tweak=tweak)


def test_select_empty_prefix_and_graph():
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 3, 16, 576, generator=g, device="cuda").to(torch.bfloat16)
    summary = torch.randint(-127, 128, (2, 20, 576), generator=g, device="cuda").to(torch.bfloat16)
    scale = torch.rand(2, 20, generator=g, device="cuda")
    n = torch.tensor([0, 320], dtype=torch.int32, device="cuda")
    s = ddtree.BlockSelector(2, 3, 16, 320, 16, 5)
    got = s(q, summary, scale, n)
    assert bool((got[0] == -1).all()) and bool((got[1] >= 0).all())
    out = torch.zeros_like(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s(q, summary, scale, n, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)


def test_refusals():
    with pytest.raises(ddtree.DDTError):
        ddtree.BlockSelector(1, 1, 16, 320, 24, 5)
    s = ddtree.BlockSelector(1, 1, 16, 320, 16, 5)
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(1, 20, 576, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(1, 20, device="cuda")
    n = torch.tensor([320], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        s(q, m[:, :19].contiguous(), c, n)
    with pytest.raises(ValueError):
        s(q.float(), m, c, n)
    with pytest.raises(ddtree.DDTError):
        ddtree.BlockSelector(1, 1, 16, 320, 16, 0)(q, m, c, n)
    with pytest.raises(ValueError):
        ddtree.block_summary(m[0], torch.zeros(1, 20, dtype=torch.int32, device="cuda"), n, 16, from_len=n)
