"""Scales at the ends of what attention over the 8-bit cache takes, and beyond, against fp64.

Scales from 2^-60 to 2^40 are used; a key with another one gives NaN to the nodes that see it and to no others. The
comparison allows a weight's 2^-12 and a score's error (below 2^-12) twice, the result's rounding to bf16 (2^-8) and what
the sums lose: 2^-9 of the weighted size in all. A weight times scale below the parts' last step, 2^-16 where the row's
largest is at least 2^7, is off by up to half of that step, 2^-24 of the largest, whatever its own size: with w s that
largest and v the stored values, 2^-24 w s times the sum of all |v| of a dim. (It shows where the keys that weigh most have
a value of next to nothing.)
"""
import math

import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def make(keys, nodes, heads, exponents, seed=0, latent=0.0, rope=1.0):
    """A star tree over one prefix; key i has scale 2^exponents[i % len], values of its own, and rope values of size `rope`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = keys + nodes
    pool, scale = ddtree.kv8_pool(n)
    scale[:] = torch.exp2(torch.tensor(exponents, device="cuda", dtype=torch.float64))[torch.arange(n, device="cuda") % len(exponents)].float()
    pool[:, :512] = torch.randn(n, 512, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    turned = rope * torch.randn(n, 64, generator=g, device="cuda")
    pool[:, 512:] = (turned.double() / scale.double()[:, None]).float().to(torch.bfloat16).view(torch.uint8)
    q = torch.randn(1, nodes, heads, 576, generator=g, device="cuda")
    q[..., :512] *= latent
    parent = torch.full((1, nodes), 0, dtype=torch.int32, device="cuda")
    parent[0, 0] = -1
    return dict(q=q.to(torch.bfloat16), pool=pool, scale=scale, slot=torch.arange(keys, dtype=torch.int32, device="cuda")[None].contiguous(),
                lens=torch.tensor([keys], dtype=torch.int32, device="cuda"), parent=parent,
                tree=torch.arange(keys, n, dtype=torch.int32, device="cuda")[None].contiguous())


def call(d):
    _, nodes, heads, _ = d["q"].shape
    v = ddtree.Kv8Verifier(1, nodes, heads, d["pool"].shape[0], d["slot"].shape[1])
    out, lse = v(d["q"], d["pool"], d["scale"], d["slot"], d["lens"], d["parent"], d["tree"], SCALE)
    assert v.status() == 0
    return out, lse


def check(d, out, lse, nodes):
    keys = d["slot"].shape[1]
    row = torch.cat([d["pool"][:, :512].view(torch.float8_e4m3fn).double(), d["pool"][:, 512:].contiguous().view(torch.bfloat16).double()], 1)
    row = row * d["scale"].double()[:, None]
    for t in nodes:
        k = row[list(range(keys)) + sorted({keys, keys + t})]
        s = SCALE * (d["q"][0, t].double() @ k.T)
        w = torch.softmax(s, -1)
        by = d["scale"].double()[list(range(keys)) + sorted({keys, keys + t})]
        last = 2.0 ** -24 * (w * by).amax(1)[:, None] * (k[:, :512].abs() / by[:, None]).sum(0)
        ref, size = w @ k[:, :512], w @ k[:, :512].abs()
        assert bool(((lse[0, t].double() - torch.logsumexp(s, -1)).abs() <= 2.0 ** -11).all()), t
        assert bool(((out[0, t].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -9 * size + last).all()), t


@pytest.mark.parametrize("exponents", [[-60], [40], [-60, -7], [-7, 40], [-60, 40, 0], [-60, -60, -60, -60, -60, -60, 40]])
def test_scales_at_the_ends(exponents):
    d = make(500, 5, 16, exponents, seed=len(exponents))
    out, lse = call(d)
    check(d, out, lse, range(5))


@pytest.mark.parametrize("bad", [2.0 ** -149, 2.0 ** -140, 2.0 ** -128, 2.0 ** -126, 2.0 ** -61, 2.0 ** 40 * 1.001, 2.0 ** 64, 3e38, 0.0, -0.0,
                                 -1.0, math.inf, math.nan])
def test_a_scale_that_is_not_usable(bad):
    """In the tree's third node: it alone sees the key. In the prefix: every node does."""
    d = make(300, 5, 16, [-7], seed=3, latent=1.0)
    d["scale"][302] = bad
    out, lse = call(d)
    assert bool(torch.isnan(out[0, 2]).all()) and bool(torch.isnan(lse[0, 2]).all())
    check(d, out, lse, [0, 1, 3, 4])
    d["scale"][302], d["scale"][17] = 2.0 ** -7, bad
    out, lse = call(d)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("exponents,rope", [([-60], 16.0), ([-60], 200.0), ([-60, -7], 30.0), ([-7], 1000.0)])
def test_rope_values_alone(exponents, rope):
    """No latent value in the queries, and (where the scale is the least one) none in the keys to speak of."""
    d = make(500, 5, 16, exponents, seed=7, rope=rope)
    d["q"][..., 512:] *= 64.0 / rope
    out, lse = call(d)
    check(d, out, lse, range(5))


def test_rows_without_latent_values():
    """As ddtree_kv8_write stores them; a query with large rope values beside small latent ones."""
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.zeros(405, 576, device="cuda")
    rows[:, 512:] = 20 * torch.randn(405, 64, generator=g, device="cuda")
    rows[::3, :512] = torch.randn(135, 512, generator=g, device="cuda")
    d = make(400, 5, 16, [0], seed=8, latent=1.0)
    ddtree.kv8_write(rows.to(torch.bfloat16), torch.arange(405, dtype=torch.int32, device="cuda"), d["pool"], d["scale"])
    d["q"][..., 512:] *= 2
    d["q"][0, 1, :, :512] = 0
    d["q"][0, 2, :, :512] *= 2.0 ** -30
    d["q"][0, 3, :, :512] *= 2.0 ** -55
    out, lse = call(d)
    check(d, out, lse, range(5))
