"""Kernel variants that only large calls reach: eviction without keys in shared memory, the block choice of many nodes,
lists of more than 4096 blocks, and which bad slots block attention reports."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda
import test_gpu_block_attn as attn
import test_gpu_block_select as select
import test_gpu_kv_evict as evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


@pytest.mark.parametrize("keep", [0.0, 1 / 3, 1.0])
def test_evict_one_request_beyond_shared_memory(keep):
    """A cluster of 16 keeps 16 x 40960 order keys; one request of more."""
    n = 16 * 40960 + 77
    w = np.random.default_rng(4).random((1, n), dtype=np.float32) ** 8
    assert evict.run(w, [n], [int(n * keep)], 4, 512) == 0


def test_evict_one_request_beyond_shared_memory_with_ties():
    n = 16 * 40960 + 1
    rng = np.random.default_rng(5)
    w = rng.choice(np.array([0.0, -0.0, 0.25, 1.0, np.nan, np.inf, -np.inf, 1e-42], np.float32), (1, n))
    assert evict.run(w, [n], [n // 2], 0, 0) == 0
    assert evict.run(w, [n - 3], [n // 5], 3, 9) == 0


@pytest.mark.parametrize("batch", [160, 306])
def test_evict_short_requests_of_a_table_beyond_shared_memory(batch):
    """A batch above 152 takes one CTA a request: a stride above 40960, whatever the lengths."""
    rng = np.random.default_rng(6)
    stride = 41000
    lens = [int(x) for x in rng.choice([0, 1, 31, 33, 500, 1999], batch)]
    lens[7], lens[batch - 6] = stride, 40961
    w = np.zeros((batch, stride), np.float32)
    w[:] = rng.random(stride, dtype=np.float32)[None] ** 8
    keep = [int(n * f) for n, f in zip(lens, rng.random(batch) * 1.1)]
    assert evict.run(w, lens, keep, 2, 17) == 0


@pytest.mark.parametrize("batch,lens,nodes,block,topk,first,last", [
    (8, [16401, 20000, 17000, 16, 0, 19999, 18000, 17], 33, 16, 32, 1, 2),       # 1025 .. 1250 blocks
    (2, [262144, 100000], 80, 16, 128, 1, 4),                                   # 16384: the last in shared memory
    (2, [262145, 262144], 77, 16, 64, 0, 1),                                    # 16385: one node's list is, one's is not
    (3, [280000, 5000, 270001], 65, 16, 300, 2, 2),
])
def test_select_for_more_nodes_than_sms(batch, lens, nodes, block, topk, first, last):
    lens = [max(1, n) for n in lens]
    select.select_case(batch, lens, nodes, 1, block, topk, first, last, seed=batch)


@pytest.mark.parametrize("nb", [1300, 16500])
def test_select_ties_for_more_nodes_than_sms(nb):
    def tweak(q, summary, scale):
        summary[:, 10:] = summary[:, 3:4]
        scale[:, 10:] = scale[:, 3:4]
    select.select_case(2, [nb * 16, nb * 16 - 5], 78, 2, 16, 37, 0, 0, tweak=tweak)


@pytest.mark.parametrize("block,n", [(16, 185000), (16, 65536 + 1), (32, 131072 + 40)])
def test_attention_over_lists_of_more_than_4096_blocks(block, n):
    """The union of lists is made 4096 blocks at a time: blocks on both sides of each border, and the last one."""
    d = attn.make([n, 300], 5, 16, block, 64, seed=block)
    nb = -(-n // block)
    edge = [x for c in range(4096, nb, 4096) for x in (c - 1, c)] + [0, nb - 1]
    idx = d["idx"][0].cpu().numpy()
    for t in range(5):
        take = edge if t % 2 == 0 else edge[::2]
        idx[t, :len(take)] = take[::-1]
    d["idx"][0] = torch.tensor(idx, device="cuda")
    out, lse, st = attn.call(d)
    assert st == 0
    attn.check(d, out, lse)
    d["idx"][0, 3, 60] = nb
    out, lse, st = attn.call(d)
    assert st == ddtree.STATUS_BAD_BLOCK
    attn.check(d, out, lse)


def test_bad_slots_are_reported_where_they_are_read():
    d = attn.make([500], 5, 16, 32, 8, seed=9, lists="all")
    d["idx"][:] = torch.tensor([0, 2, 3, 5, 7, 9, 11, 15], dtype=torch.int32, device="cuda")
    d["slot"][0, 32 * 4 + 1] = -1                       # block 4: nobody lists it
    out, lse, st = attn.call(d)
    assert st == 0
    attn.check(d, out, lse)
    for pos, bad in ((5, -1), (77, 1 << 30), (499, d["kv"].shape[0])):
        e = dict(d, slot=d["slot"].clone())
        e["slot"][0, pos] = bad
        out, lse, st = attn.call(e)
        assert st == ddtree.STATUS_BAD_SLOT, pos
        attn.check(e, out, lse)
    d["idx"][0, :4] = -1                                # one node lists it
    d["idx"][0, 4, 0] = 4
    out, lse, st = attn.call(d)
    assert st == ddtree.STATUS_BAD_SLOT
    attn.check(d, out, lse)
