"""Eviction by weight (ddtree_kv_evict): every output equals a plain ranking's, exactly."""
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


def plain(w, slots, keep, sink, recent):
    n = len(w)
    key = np.where(np.isnan(w), -np.inf, w.astype(np.float64)) + 0.0   # -0 ties with +0
    at = np.arange(n)
    held = (at < sink) | (at >= n - recent)
    order = np.lexsort((at, np.where(held, 0.0, -key), ~held))
    stay = np.sort(order[:max(0, min(keep, n))])
    gone = np.setdiff1d(at, stay)
    return slots[stay], w[stay], slots[gone]


def run(w, lens, keep, sink, recent, slots=None, **kw):
    B, stride = w.shape
    slots = np.arange(B * stride, dtype=np.int32).reshape(B, stride)[:, ::-1].copy() if slots is None else slots
    t = lambda x, dt: torch.tensor(np.asarray(x), dtype=dt, device="cuda")  # noqa: E731
    so = torch.full((B, stride), -5, dtype=torch.int32, device="cuda")
    wo = torch.full((B, stride), -5.0, device="cuda")
    fr = torch.full((B, stride), -5, dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    so, wo, lo, fr = ddtree.kv_evict(t(w, torch.float32), t(slots, torch.int32), t(lens, torch.int32),
                                     t(keep, torch.int32), sink, recent, so, wo, None, fr, workspace=ws, **kw)
    so, wo, lo, fr = (x.cpu().numpy() for x in (so, wo, lo, fr))
    for b in range(B):
        n = min(max(lens[b], 0), stride)
        rs, rw, rf = plain(w[b, :n], slots[b, :n], keep[b], sink, recent)
        m = len(rs)
        assert lo[b] == m, (b, lo[b], m)
        assert np.array_equal(so[b, :m], rs), b
        assert np.array_equal(wo[b, :m].view(np.int32), rw.view(np.int32)), b
        assert np.array_equal(fr[b, :n - m], rf), b
        assert (so[b, m:] == -5).all() and (wo[b, m:] == -5).all() and (fr[b, n - m:] == -5).all()
    return ddtree.read_device_status(ws)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 1023, 1025, 4096, 8191, 32768, 32769, 70001])
@pytest.mark.parametrize("sink,recent", [(0, 0), (4, 16)])
def test_sizes(n, sink, recent):
    rng = np.random.default_rng(n)
    w = rng.random((3, n + 3), dtype=np.float32) ** 8
    assert run(w, [n, n // 2, max(1, n - 1)], [n // 2, n // 4 + 1, n], sink, recent) == 0


def test_large_batches():
    """More requests than the small-batch kernel takes, of very different lengths."""
    rng = np.random.default_rng(7)
    lens = [int(x) for x in rng.integers(0, 9000, 40)] + [9000, 1, 0]
    w = rng.choice(rng.random(300, dtype=np.float32) ** 8, (len(lens), 9000))   # many ties
    run(w, lens, [int(n * f) for n, f in zip(lens, rng.random(len(lens)) * 1.1)], 4, 64)


@pytest.mark.parametrize("batch", [20, 153, 256, 257, 400])
def test_batches_whose_requests_take_turns(batch):
    """More CTAs than SMs: equal, empty, too long and negative lengths in any order."""
    rng = np.random.default_rng(batch)
    w = rng.choice(rng.random(50, dtype=np.float32), (batch, 400))
    lens = [int(x) for x in rng.choice([0, 1, 37, 37, 200, 399, 400], batch)]
    keep = [int(n * f) for n, f in zip(lens, rng.random(batch) * 1.1)]
    assert run(w, lens, keep, 2, 5) == 0
    lens[batch // 2], lens[batch // 3] = -7, 401
    assert run(w, lens, keep, 2, 5) == ddtree.STATUS_BAD_PREFIX


def test_ties_and_special_values():
    rng = np.random.default_rng(1)
    n = 5000
    w = rng.choice(np.array([0.0, -0.0, 1.0, np.nan, np.inf, -np.inf, 1e-42, -1e-42, 2.0 ** -126], np.float32), (6, n))
    run(w, [n] * 6, [0, 1, 700, 2500, 4999, 5000], 0, 0)
    run(w, [n] * 6, [3, 10, 700, 2500, 4999, 9000], 5, 9)
    same = np.full((2, n), 0.25, np.float32)
    run(same, [n, n], [1234, 17], 2, 3)


def test_budget_below_the_protected_positions():
    w = np.random.default_rng(2).random((4, 300), dtype=np.float32)
    run(w, [300, 300, 12, 5], [3, 25, 12, 4], 8, 20)
    run(w, [300, 300, 12, 5], [8, 28, 11, 0], 8, 20)
    run(w, [300, 7, 0, 1], [100, 100, 100, 100], 1000, 1000)


def test_empty_and_out_of_range():
    w = np.random.default_rng(3).random((3, 64), dtype=np.float32)
    assert run(w, [0, 64, 10], [10, -4, 0], 1, 1) == 0
    assert run(w, [-1, 65, 10], [10, 20, 5], 1, 1) == ddtree.STATUS_BAD_PREFIX


def test_long_request_whose_keys_do_not_stay_in_shared_memory():
    n = 8 * 40960 + 77
    w = np.random.default_rng(4).random((1, n), dtype=np.float32) ** 8
    run(w, [n], [n // 3], 4, 512)


def test_graph_replay_on_new_weights():
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.rand(2, 3000, device="cuda", generator=g)
    slots = torch.arange(6000, dtype=torch.int32, device="cuda").reshape(2, 3000)
    lens = torch.tensor([3000, 2100], dtype=torch.int32, device="cuda")
    keep = torch.tensor([1000, 700], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(slots), torch.zeros_like(w), torch.zeros_like(lens), torch.zeros_like(slots)]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    call = lambda o: ddtree.kv_evict(w, slots, lens, keep, 4, 8, o[0], o[1], o[2], o[3], workspace=ws)  # noqa: E731
    call(outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    w.copy_(torch.rand(2, 3000, device="cuda", generator=g))
    graph.replay()
    torch.cuda.synchronize()
    fresh = [torch.zeros_like(x) for x in outs]
    call(fresh)
    for b, n in ((0, 1000), (1, 700)):
        assert torch.equal(outs[0][b, :n], fresh[0][b, :n]) and torch.equal(outs[1][b, :n], fresh[1][b, :n])


def test_refusals():
    w = torch.rand(1, 64, device="cuda")
    s = torch.zeros(1, 64, dtype=torch.int32, device="cuda")
    n = torch.tensor([64], dtype=torch.int32, device="cuda")
    for kw in (dict(slot_idx_out=s), dict(weight_out=w), dict(prefix_len_out=n)):
        with pytest.raises(ddtree.DDTError) as e:
            ddtree.kv_evict(w, s, n, n, **kw)
        assert e.value.code == -7
    with pytest.raises(ddtree.DDTError):
        ddtree.kv_evict(w, s, n, n, sink=-1)
    with pytest.raises(ValueError):
        ddtree.kv_evict(w.double(), s, n, n)
    with pytest.raises(ValueError):
        ddtree.kv_evict(w.cpu(), s, n, n)
