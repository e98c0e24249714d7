"""A decoding step over the 8-bit cache, its operators in order, each fed by the one before."""
import math

import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda
import test_gpu_accept as accept
import test_gpu_kv8_attn as attn

pytestmark = pytest.mark.gpu
B, T, H, V, STRIDE = 3, 9, 16, 4001, 700
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


class Step:
    """What a serving loop keeps: the cache, the slot tables, the free slots, the handles."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(0)
        self.slots = 4096
        self.pool, self.scale = ddtree.kv8_pool(self.slots)
        self.table = torch.zeros(B, STRIDE, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor([600, 33, 250], dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.slots, generator=g, device="cuda").to(torch.int32)
        self.norm = torch.exp(0.3 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
        angle = torch.arange(2048, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
        self.rotation = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        self.head = torch.randn(512, V, generator=g, device="cuda") / 4
        self.verify = ddtree.Kv8Verifier(B, T, H, self.slots, STRIDE)
        self.accept = ddtree.TreeAcceptor(B, T, V)
        self.weigh = ddtree.KeyWeights(B, T, H, self.slots, STRIDE)
        self.g = g
        at = 0
        for b, n in enumerate(self.lens.tolist()):      # the prompts
            self.table[b, :n] = self.free[at:at + n]
            rows = torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16)
            ddtree.kv8_write(rows, self.table[b, :n].contiguous(), self.pool, self.scale, norm_weight=self.norm,
                             rotation=self.rotation, position=torch.arange(n, dtype=torch.int32, device="cuda"))
            at += n
        self.free = self.free[at:].contiguous()

    def draft(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        parent = torch.full((B, T), -1, dtype=torch.int32)
        depth = torch.zeros(B, T, dtype=torch.int32)
        host = torch.Generator().manual_seed(seed)
        for b in range(B):
            for i in range(1, T):
                parent[b, i] = int(torch.randint(0, i, (1,), generator=host))
                depth[b, i] = depth[b, parent[b, i]] + 1
        return dict(parent=parent.cuda(), depth=depth.cuda(), tokens=torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32),
                    rows=torch.randn(B * T, 576, generator=g, device="cuda").to(torch.bfloat16),
                    q=torch.randn(B, T, H, 576, generator=g, device="cuda").to(torch.bfloat16),
                    uniform=torch.rand(B, T, generator=g, device="cuda"))

    def run(self, d, logits_of):
        tree = self.free[:B * T].reshape(B, T).contiguous()
        position = (self.lens[:, None] + d["depth"]).reshape(-1)
        ddtree.kv8_write(d["rows"], tree.reshape(-1), self.pool, self.scale, norm_weight=self.norm, rotation=self.rotation,
                         position=position)
        out, lse = self.verify(d["q"], self.pool, self.scale, self.table, self.lens, d["parent"], tree, SCALE)
        logits = logits_of(out)
        path, length, token = self.accept(logits, d["tokens"], d["parent"], d["uniform"],
                                          torch.full((B,), 0.9, device="cuda"))
        back = ddtree.kv8_read(self.pool, self.scale, torch.arange(self.slots, dtype=torch.int32, device="cuda"))
        weight = self.weigh(d["q"], back, self.table, self.lens, lse, SCALE, node_idx=path)
        return dict(tree=tree, out=out, lse=lse, logits=logits, path=path, length=length, token=token, weight=weight)

    def keep(self, r):
        """The accepted rows join the prefix; the others' slots are free again."""
        for b, n in enumerate(r["length"].tolist()):
            m = int(self.lens[b])
            kept = r["tree"][b][r["path"][b, :n].long()]
            self.table[b, m:m + n] = kept
            self.free = self.free[~torch.isin(self.free, kept)].contiguous()
        self.lens += r["length"]


def checked(step, d, r):
    e = dict(q=d["q"], pool=step.pool, scale=step.scale, slot=step.table, lens=step.lens, parent=d["parent"], tree=r["tree"],
             tree_len=None)
    assert step.verify.status() == 0 and step.accept.status() == 0 and step.weigh.status() == 0
    attn.check(e, r["out"], r["lse"])
    a = dict(logits=r["logits"], draft=None, tokens=d["tokens"], parent=d["parent"], uniform=d["uniform"], tree_len=None,
             temperature=torch.full((B,), 0.9, device="cuda"))
    assert accept.check(a, [r[k].cpu().numpy() for k in ("path", "length", "token")]) >= 2
    # a row's weights and its tree part sum to one: so the sums are below the number of accepted rows
    for b in range(B):
        total = float(r["weight"][b, :int(step.lens[b])].double().sum())
        assert 0 < total < int(r["length"][b]) * H
    assert not bool(r["weight"][1, int(step.lens[1]):].any())


def test_three_steps():
    step = Step()
    for seed in range(1, 4):
        d = step.draft(seed)

        def logits_of(out):   # a head that likes the drafted tokens, so that paths have lengths
            logits = out.float().mean(2) @ step.head
            b = torch.arange(B, device="cuda")[:, None].expand(B, T - 1)
            at = (b, d["parent"][:, 1:].long(), d["tokens"][:, 1:].long())
            return logits.index_put(at, torch.tensor(9.0, device="cuda"), accumulate=True)
        r = step.run(d, logits_of)
        checked(step, d, r)
        before = step.lens.clone()
        step.keep(r)
        assert bool((step.lens > before).all())


def test_captured():
    """The step in a graph, replayed with other drafts, gives what the calls give by themselves."""
    step = Step()
    d = step.draft(11)

    def logits_of(out):
        return out.float().mean(2) @ step.head
    step.run(d, logits_of)                     # (first calls set devices and libraries up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step.run(d, logits_of)
    for seed in (12, 13):
        for k, v in step.draft(seed).items():
            d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in r.items()}
        want = step.run(d, logits_of)
        for k in ("out", "lse", "path", "length", "token", "weight"):
            assert torch.equal(got[k], want[k]), k
        checked(step, d, want)
