"""The check of drafted tokens (ddtree_accept) against 64-bit arithmetic, token by token.

Outputs are whole numbers and have to be equal.  The kernel's weights are off by 2^-31 of themselves (and by less than
2^-43 of the largest), so a trial or a draw that 64-bit arithmetic decides within 1e-8 of its border is not judged; of the
thousands here that leaves out a handful at most.
"""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import build_and_load, require_cuda

pytestmark = pytest.mark.gpu
NEAR = 1e-8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def make(batch, nodes, vocab, dtype=torch.float32, tree="random", drawn=False, temperature=1.0, seed=0, peak=4.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = np.random.default_rng(seed)
    logits = (peak * torch.randn(batch, nodes, vocab, generator=g, device="cuda")).to(dtype)
    parent = np.full((batch, nodes), -1, np.int32)
    for i in range(1, nodes):
        parent[:, i] = i - 1 if tree == "chain" else 0 if tree == "star" else h.integers(max(0, i - 6), i, batch)
    up = torch.tensor(parent, device="cuda").long().clamp(min=0)
    rows = torch.arange(batch, device="cuda")[:, None]
    at_parent = logits[rows, up].float()
    draft = None
    if drawn:
        draft = torch.softmax(logits.float() + 1.5 * torch.randn(logits.shape, generator=g, device="cuda"), -1)
        tokens = torch.multinomial(draft[rows, up].reshape(-1, vocab), 1, generator=g).reshape(batch, nodes)
    else:
        noisy = at_parent + 2 * torch.randn(at_parent.shape, generator=g, device="cuda")
        tokens = noisy.argmax(-1)
    return dict(logits=logits, draft=draft, tokens=tokens.to(torch.int32), parent=torch.tensor(parent, device="cuda"),
                uniform=torch.rand(batch, nodes, generator=g, device="cuda"), tree_len=None,
                temperature=torch.full((batch,), temperature, device="cuda"))


def call(d, library=None, **kw):
    batch, nodes, vocab = d["logits"].shape
    a = ddtree.TreeAcceptor(batch, nodes, vocab, library=library)
    got = a(d["logits"], d["tokens"], d["parent"], d["uniform"], d["temperature"], draft_prob=d["draft"],
            tree_len=d["tree_len"], **kw)
    return [x.cpu().numpy() for x in got], a.status()


def reference(d, b):
    """(path, next token, nearest border) of request b."""
    logits = d["logits"][b].double().cpu().numpy()
    draft = None if d["draft"] is None else d["draft"][b].double().cpu().numpy()
    tokens, parent = d["tokens"][b].tolist(), d["parent"][b].tolist()
    u = d["uniform"][b].double().cpu().numpy()
    u = np.where(np.isnan(u), 0, np.clip(u, 0, 1 - 2.0 ** -24))
    temperature, vocab = float(d["temperature"][b]), logits.shape[1]
    n = logits.shape[0] if d["tree_len"] is None else min(max(int(d["tree_len"][b]), 0), logits.shape[0])
    if n == 0:
        return [], -1, 1.0
    near, path, v = 1.0, [0], 0
    while True:
        l = np.where(np.isnan(logits[v]), -np.inf, np.minimum(logits[v], 3.4028234663852886e38))
        if not (l > -np.inf).any():
            return path, -1, near
        if temperature > 0:
            with np.errstate(invalid="ignore"):
                y = (l - l.max()) / temperature
            w = np.exp(np.where(np.isnan(y), -np.inf, y))
        else:
            w = np.zeros(vocab)
            w[int(l.argmax())] = 1
        go = None
        for c in [c for c in range(v + 1, n) if parent[c] == v and 0 <= tokens[c] < vocab]:
            x, total = tokens[c], w.sum()
            q = 1.0 if draft is None else float(draft[v, x])
            near = min(near, abs(u[c] * total * q - w[x]) / total)
            if u[c] * total * q < w[x]:
                go = c
                break
            left = w.copy()
            if draft is None:
                left[x] = 0
            else:
                left = np.maximum(w - total * draft[v], 0)
            if left.sum() > 0:
                w = left
        if go is None:
            break
        v = go
        path.append(v)
    sums = np.cumsum(w)
    near = min(near, np.abs(sums[w > 0][:-1] / sums[-1] - u[0]).min(initial=1.0) if sums[-1] > 0 else 1.0)
    return path, int(np.argmax(sums > u[0] * sums[-1])), near


def check(d, got, requests=None):
    path, length, token = got
    judged = 0
    for b in range(path.shape[0]) if requests is None else requests:
        want, want_token, near = reference(d, b)
        if near < NEAR and float(d["temperature"][b]) > 0:
            continue
        judged += 1
        assert length[b] == len(want) and path[b, :len(want)].tolist() == want, (b, want, path[b], near)
        assert (path[b, len(want):] == -1).all()
        assert token[b] == want_token, (b, want_token, token[b], near)
    return judged


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,nodes,vocab,tree", [
    (1, 1, 1, "chain"), (1, 9, 2, "chain"), (64, 9, 33, "random"), (7, 33, 1001, "random"), (40, 9, 5003, "chain"),
    (3, 65, 32768, "random"), (2, 128, 2050, "star"), (1, 5, 131072, "random"), (200, 4, 257, "star"),
    (1, 3, 262144, "chain"), (12, 5, 100003, "random")])
def test_trees(batch, nodes, vocab, tree, dtype, drawn):
    total = judged = 0
    for seed in range(2):
        d = make(batch, nodes, vocab, dtype, tree, drawn, temperature=0.8 if seed else 1.0, seed=seed + nodes)
        got, st = call(d)
        assert st == 0
        total += batch
        judged += check(d, got)
    assert judged >= 0.9 * total - 1


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_temperatures_of_their_own(dtype, drawn):
    d = make(16, 17, 700, dtype, "random", drawn, seed=3)
    d["temperature"] = torch.tensor([0.0, 1.0, -1.0, math.nan, math.inf, 1e-30, 1e-3, 100.0] * 2, device="cuda")
    got, st = call(d)
    assert st == 0
    check(d, got, requests=[b for b in range(16) if b % 8 != 3])
    d["temperature"][3] = d["temperature"][11] = 0     # NaN is greedy too
    again, _ = call(d)
    assert all((x == y).all() for x, y in zip(got, again))


@pytest.mark.parametrize("drawn", [False, True])
def test_logits_whose_difference_is_no_number(drawn):
    """They count as -inf, at any temperature; differences that are numbers do not."""
    d = make(12, 3, 300, torch.float32, "star", drawn, seed=17)
    d["temperature"] = torch.tensor([math.inf, 1e38, 1.0] * 4, device="cuda")
    d["logits"][:] = 2e38
    d["logits"][:, :, 100:] = -2e38
    d["tokens"][:, 1:] = 250
    e = dict(d, logits=d["logits"].clone())
    e["logits"][:, :, 100:] = -math.inf
    got, st = call(d)
    want, _ = call(e)
    assert st == 0 and all((x == y).all() for x, y in zip(got, want))
    assert (got[1] == 1).all() and (got[2] < 100).all() and (got[2] >= 0).all()


def test_greedy_takes_the_lowest_of_equal_logits():
    d = make(4, 3, 5000, torch.bfloat16, "chain", temperature=0.0, seed=4)
    d["logits"][:] = 0
    d["logits"][:, :, 4321] = 7
    d["logits"][:, :, 1234] = 7
    d["tokens"][:, 1] = torch.tensor([1234, 4321, 1234, 0], device="cuda")
    d["tokens"][:, 2] = torch.tensor([1234, 1234, 4321, 1234], device="cuda")
    (path, length, token), st = call(d)
    assert st == 0 and length.tolist() == [3, 1, 2, 1] and token.tolist() == [1234] * 4
    d["logits"][:] = -0.0
    d["logits"][:, :, 17] = 0.0
    (path, length, token), st = call(d)
    assert token.tolist() == [0] * 4


def test_logits_that_are_not_numbers():
    d = make(6, 3, 900, torch.float32, "chain", seed=5)
    d["logits"][0, :, 100:] = -math.inf
    d["logits"][1, :, ::2] = math.nan
    d["logits"][2, 0] = -math.inf
    d["logits"][3, :] = math.nan
    d["logits"][4, 0, 55] = math.inf
    d["logits"][4, 0, 66] = math.inf
    d["logits"][5, 0, 3] = 3.4028234e38
    got, st = call(d)
    assert st == ddtree.STATUS_BAD_LOGITS
    check(d, got)
    assert got[2][3] == -1 and got[1][3] == 1 and got[2][2] == -1


@pytest.mark.parametrize("drawn", [False, True])
def test_bad_tokens_parents_and_tree_lengths(drawn):
    d = make(6, 9, 300, torch.float32, "random", drawn, seed=6)
    d["tokens"][:, 0] = 1 << 30                   # the root's is not looked at
    got, st = call(d)
    assert st == 0
    check(d, got)
    d["tokens"][0, 1:] = 300
    d["tokens"][1, 2], d["tokens"][1, 4] = -1, -2 ** 31
    got, st = call(d)
    assert st == ddtree.STATUS_BAD_TOKEN
    check(d, got)
    d["parent"][2, 3], d["parent"][2, 4], d["parent"][3, 5] = 3, 100, -1
    got, st = call(d)
    assert st == ddtree.STATUS_BAD_TOKEN | ddtree.STATUS_BAD_PARENT
    check(d, got)
    d["tree_len"] = torch.tensor([9, 4, 10, -1, 0, 1], dtype=torch.int32, device="cuda")
    d["tokens"][5, 1:] = -7                       # not active: not looked at
    got, st = call(d)
    assert st & ddtree.STATUS_BAD_TREE_LEN
    check(d, got)
    assert got[1].tolist()[3:] == [0, 0, 1] and got[2][3] == got[2][4] == -1


def test_siblings_with_the_same_token():
    d = make(64, 6, 40, torch.float32, "star", seed=7)
    d["tokens"][:, 1:4] = d["tokens"][:, 1:2]
    got, st = call(d)
    assert st == 0
    check(d, got)
    assert not (got[0][:, 1] == 2).any() and not (got[0][:, 1] == 3).any()   # the second trial cannot succeed


@pytest.mark.parametrize("value", [0.0, 0.99999994, 1.0, 5.0, -3.0, math.nan, 1e-40])
@pytest.mark.parametrize("drawn", [False, True])
def test_uniforms_at_their_ends(value, drawn):
    d = make(8, 9, 500, torch.float32, "random", drawn, seed=8)
    d["uniform"][:4] = value
    d["uniform"][4:, 0] = value
    got, st = call(d)
    assert st == 0
    check(d, got)


def test_draft_equal_to_the_target_accepts_everything():
    d = make(20, 9, 1000, torch.float32, "chain", drawn=True, seed=9)
    d["draft"] = torch.softmax(d["logits"].double(), -1).float() * 0.999
    (path, length, _), st = call(d)
    assert st == 0 and (length == 9).all()


def test_draft_probabilities_out_of_range():
    d = make(4, 3, 300, torch.float32, "chain", drawn=True, seed=10)
    d["draft"][0, 0] = 0
    d["draft"][1, 0] = -1
    d["draft"][2, 0] = math.nan
    d["draft"][3, 0] = 2.0                        # counts as 1: nothing would be left, so a refusal changes nothing
    (path, length, token), st = call(d)
    assert st == 0 and (length[:3] >= 2).all() and ((token >= 0) & (token < 300)).all()


@pytest.mark.parametrize("drawn", [False, True])
def test_the_same_tokens_on_any_cluster(drawn):
    """One request takes eight CTAs a row, a batch of 64 one: sums are exact, so nothing changes."""
    d = make(64, 9, 40001, torch.bfloat16, "random", drawn, seed=11)
    all_of, st = call(d)
    assert st == 0
    for b in (0, 13, 63):
        one = {k: None if v is None else v[b:b + 1].contiguous() for k, v in d.items()}
        got, _ = call(one)
        assert all((x[0] == y[b]).all() for x, y in zip(got, all_of))
    check(d, all_of, requests=range(0, 64, 9))


def test_rows_inside_wider_tensors_at_any_alignment():
    d = make(5, 7, 1003, torch.bfloat16, "random", drawn=True, seed=12)
    want, _ = call(d)
    for pad in (1, 5):
        wide = torch.full((5, 7, 1003 + 2 * pad), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[:, :, pad:pad + 1003] = d["logits"]
        wide_q = torch.full((5, 7, 1003 + pad), math.nan, device="cuda")
        wide_q[:, :, pad:] = d["draft"]
        got, st = call(dict(d, logits=wide[:, :, pad:pad + 1003], draft=wide_q[:, :, pad:]))
        assert st == 0 and all((x == y).all() for x, y in zip(got, want))


def test_frequencies_follow_the_target():
    """The first new token's distribution is the target's, whatever was drafted: 200000 trials, five standard deviations."""
    n, vocab = 1000, 12
    h = torch.Generator(device="cuda").manual_seed(13)
    logits = torch.randn(vocab, generator=h, device="cuda")
    p = torch.softmax(logits.double(), -1).cpu().numpy()
    q = torch.softmax(torch.randn(vocab, generator=h, device="cuda"), -1)
    parent = torch.tensor([[-1, 0, 0, 0]], dtype=torch.int32, device="cuda").expand(n, 4).contiguous()
    for drawn in (False, True):
        count = np.zeros(vocab)
        for _ in range(200):
            tokens = (torch.multinomial(q.expand(n * 4, vocab), 1, generator=h).reshape(n, 4) if drawn else
                      torch.tensor([[0, 3, 7, 1]], device="cuda").expand(n, 4)).to(torch.int32).contiguous()
            d = dict(logits=logits.expand(n, 4, vocab).contiguous(), tokens=tokens, parent=parent, tree_len=None,
                     draft=q.expand(n, 4, vocab).contiguous() if drawn else None,
                     uniform=torch.rand(n, 4, generator=h, device="cuda"), temperature=torch.ones(n, device="cuda"))
            (path, length, token), _ = call(d)
            first = np.where(length > 1, tokens.cpu().numpy()[np.arange(n), np.maximum(path[:, 1], 0)], token)
            count += np.bincount(first, minlength=vocab)
        total = 200 * n
        assert (np.abs(count - total * p) <= 5 * np.sqrt(total * p * (1 - p))).all()


def test_captured_replayed_and_on_another_stream():
    d = make(4, 9, 5000, torch.bfloat16, "random", drawn=True, seed=14)
    want, _ = call(d)
    a = ddtree.TreeAcceptor(4, 9, 5000)
    args = (d["logits"], d["tokens"], d["parent"], d["uniform"], d["temperature"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = a(*args, draft_prob=d["draft"], stream=side)
    side.synchronize()
    assert a.status(side) == 0 and all((x.cpu().numpy() == y).all() for x, y in zip(got, want))
    torch.cuda.synchronize()
    out = [torch.zeros_like(x) for x in got]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a(*args, draft_prob=d["draft"], path=out[0], path_len=out[1], next_token=out[2])
    for seed in (15, 16):
        e = make(4, 9, 5000, torch.bfloat16, "random", drawn=True, seed=seed)
        for k in ("logits", "tokens", "parent", "uniform", "draft"):
            d[k].copy_(e[k])
        graph.replay()
        torch.cuda.synchronize()
        assert a.status() == 0
        check(d, [x.cpu().numpy() for x in out])


@pytest.mark.parametrize("batch,step", [(1, 1), (1, 2), (3, 1), (3, 4)])
def test_a_wait_that_runs_out(batch, step):
    """A test build does not send a warp's part of one reduction: the status word says so, and the next call is right."""
    hooks = build_and_load("testhooks")
    d = make(batch, 9, 40000, torch.bfloat16, "star", drawn=True, seed=17)
    d["uniform"][:, 1:] = 0.9999            # several refusals, a reduction each
    want, _ = call(d)
    hooks.ddtree_test_set_keep_back(step)
    try:
        _, st = call(d, library=hooks)
    finally:
        hooks.ddtree_test_set_keep_back(-1)
    assert st & ddtree.STATUS_TIMEOUT
    got, st = call(d, library=hooks)
    assert st == 0 and all((x == y).all() for x, y in zip(got, want))
