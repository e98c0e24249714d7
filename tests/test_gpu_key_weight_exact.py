"""Key weights where the products add up exactly: the score is sm_scale q.k and nothing is added to it.

sm_scale = fp32(ln 2) / 8, so that scores in log2 units are q.k / 8 (the library's constant is off by 2^-26 at most:
2.7e-9 for fp32(ln 2), and the product rounds to 2^-3).  q and k are small integers, q.k < 2^24 in size, so no
accumulation rounds.  The exponent is q.k / 8 - lse log2(e): one product of lse (2^-24) with an fp32 constant
(2^-26), and the result rounds once (2^-24); 2^x adds 2^-22.  With a score and lse of at most M log2 units the weight is
off by at most ln 2 (M (2^-24 + 2^-26 + 2^-26) + 2^-24 |exponent|) + 2^-22, relative to it, and a sum of n of
them by n 2^-24 more.
"""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
SCALE = float(np.float32(math.log(2.0))) / 8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def check(q, kv, lse):
    """q [T, H, 576], kv [n, 576], lse [T, H] fp32."""
    n, (nodes, heads) = kv.shape[0], q.shape[:2]
    w = ddtree.KeyWeights(1, nodes, heads, n, n)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = w(q[None].contiguous(), kv, torch.arange(n, **i32)[None].contiguous(), torch.tensor([n], **i32),
            lse[None].contiguous(), SCALE)[0]
    assert w.status() == 0
    dot = kv.double() @ q.double().reshape(-1, 576).T                # [n, T * H], exact
    l = lse.double().reshape(-1) / math.log(2.0)
    x = dot / 8 - l
    big = torch.maximum((dot / 8).abs(), l.abs().expand_as(dot))
    rel = math.log(2.0) * (big * (2.0 ** -24 + 2.0 ** -25) + 2.0 ** -24 * x.abs()) + 2.0 ** -22 + q.shape[0] * heads * 2.0 ** -24
    p = torch.exp2(x)
    err = (out.double() - p.sum(1)).abs()
    tol = (p * rel).sum(1)
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dim", [0, 15, 191, 287, 288, 511, 575])
@pytest.mark.parametrize("a,b", [(64, 32), (-64, -32), (32, 16), (1, 0)])
def test_one_product(dim, a, b):
    """Scores of 256, 64 and 0 log2 units from one product, and an lse beside them: weights near 1."""
    q = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(130, 576, dtype=torch.bfloat16, device="cuda")
    q[..., dim], kv[:, dim] = a, b
    lse = torch.full((2, 16), a * b / 8 * math.log(2.0), device="cuda")
    check(q, kv, lse)


@pytest.mark.parametrize("nodes,heads,n", [(1, 1, 5), (9, 16, 300), (3, 128, 513)])
def test_integers(nodes, heads, n):
    g = torch.Generator(device="cuda").manual_seed(nodes)
    draw = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kv = draw(nodes, heads, 576), draw(n, 576)
    top = (kv.float() @ q.float().reshape(-1, 576).T).amax(0) / 8 * math.log(2.0)
    check(q, kv, top.reshape(nodes, heads).float())


def test_large_scores_of_both_halves():
    """Every dim the same: 576 products of 8 x 8, 4608 log2 units."""
    q = torch.full((1, 16, 576), 8.0, dtype=torch.bfloat16, device="cuda")
    kv = torch.full((64, 576), 8.0, dtype=torch.bfloat16, device="cuda")
    check(q, kv, torch.full((1, 16), 576 * 64 / 8 * math.log(2.0), device="cuda"))
