"""Rows into the 8-bit cache: each value is the formula's, rounded once.

The formula in 64 bits (its own error is far below) is rounded to the stored types. A value whose quotient lies within
2^-21 of itself of a border between two stored values may go to either side: the kernel's chain from the row to the
quotient, in fp32, is a reciprocal root with one step of refinement (2^-23 of it), a product that is exact and two
roundings (2^-24 each), so 2^-22 in all; the rotation rounds once but for the last sum. Of normal values 2^-21 of the value
on either side of a border, of which there are 8 to an octave, are 1 in 60000; the test allows 1 in 10000 of them.
"""
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


def e4m3(x):
    """Nearest e4m3 value (ties to even), and the distance of |x| to the nearest border between two, relative to |x|."""
    a = x.abs()
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(a.clamp(min=2.0 ** -20))), min=-6) - 3)
    at = a / step
    return torch.sign(x) * torch.round(at) * step, (at - torch.floor(at) - 0.5).abs() * step / a.clamp(min=2.0 ** -20)


def bf16(x):
    """The same for bf16, of normal values."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -100))) - 7)
    at = a / step
    return torch.sign(x) * torch.round(at) * step, (at - torch.floor(at) - 0.5).abs() * step / a.clamp(min=2.0 ** -100)


@pytest.mark.parametrize("amp,eps", [(1.0, 1e-6), (300.0, 1e-5), (0.01, 1e-6), (1e-3, 1e-5)])
@pytest.mark.parametrize("pairs", [False, True])
def test_values_rounded_once(amp, eps, pairs):
    n = 4000
    g = torch.Generator(device="cuda").manual_seed(int(amp * 1000) + pairs)
    rows = (amp * torch.randn(n, 576, generator=g, device="cuda")).to(torch.bfloat16)
    w = torch.exp(0.5 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
    a = 100 * torch.rand(50, 32, generator=g, device="cuda")
    table = torch.cat([a.cos(), a.sin()], 1).contiguous()
    position = torch.randint(0, 50, (n,), generator=g, device="cuda", dtype=torch.int32)
    pool, scale = ddtree.kv8_pool(n)
    ddtree.kv8_write(rows, torch.arange(n, dtype=torch.int32, device="cuda"), pool, scale, norm_weight=w, eps=eps,
                     rotation=table, position=position, interleaved=pairs)
    x = rows.double()
    c = x[:, :512] / torch.sqrt((x[:, :512] ** 2).mean(1, keepdim=True) + eps) * w.double()
    r = x[:, 512:].clone()
    i = torch.arange(32, device="cuda")
    i, j = (2 * i, 2 * i + 1) if pairs else (i, i + 32)
    cos, sin = table[position.long()].double().split(32, 1)
    r[:, i], r[:, j] = r[:, i] * cos - r[:, j] * sin, r[:, j] * cos + r[:, i] * sin
    want = torch.exp2(torch.ceil(torch.log2(c.abs().amax(1) / 448)))
    edge = (c.abs().amax(1) / 448 / want - 0.5).abs() < 2.0 ** -21   # (a maximum of 448 scales, to the last bits)
    edge |= (c.abs().amax(1) / 448 / want - 1.0).abs() < 2.0 ** -21
    assert torch.equal(scale.double()[~edge], want[~edge]) and int(edge.sum()) <= 2
    got = pool[:, :512].view(torch.float8_e4m3fn).double(), pool[:, 512:].contiguous().view(torch.bfloat16).double()
    for value, have, form in ((c, got[0], e4m3), (r, got[1], bf16)):
        ref, near = form(value / want[:, None])
        if form is bf16:   # where the two products cancel, what is left of their roundings counts for more
            size = torch.zeros_like(r)
            size[:, i] = size[:, j] = x[:, 512:][:, i].abs() + x[:, 512:][:, j].abs()
            near = near * value.abs() / size
        off = (have != ref) & ~edge[:, None]
        assert not bool((off & (near > 2.0 ** -21)).any()), int(off.sum())
        assert int(off.sum()) <= off.numel() // 10000
