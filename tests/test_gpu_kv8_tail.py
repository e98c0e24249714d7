"""Attention over the 8-bit cache with one dominant key before a flat tail, against fp64.

A key far above the others is the ordinary state of a language model; what the many small weights add up to has to reach
the output. Tolerance, from the arithmetic and the same for any number of keys: a weight enters the second product as the
nearest f16 (2^-12 of it), a score's error (up to 2^-13 here: 40 partial sums of two units of 2^-24 of sum |q k| < 200,
and three roundings of 2^-23 of values below 32) counts twice, a sum over 32768 keys is cut to fp32 for every 32 of them and
each part (2^-23 each, 2^-11.4 in all): together within 2^-9 of the values' weighted size. What falls below the parts' last
step is at most 2^-24 of the largest weight a key, 2^-9 of it over 32768 keys of one sign. Rounding out to bf16: 2^-8 of it.
"""
import ctypes
import math

import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
HEADS = 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def make(keys, batch, gaps, spread, at, nodes=1, seed=0):
    """Requests that share one prefix of alike latent values but one; head h has that key gaps[h] nats above the others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    slots = keys + nodes
    pool, scale = ddtree.kv8_pool(slots)
    latent = torch.randn(2, 512, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    pool[:, :512] = latent[0]
    pool[at, :512] = latent[1]
    rope = torch.zeros(slots, 64, device="cuda")
    rope[:, 1] = 2 * torch.rand(slots, generator=g, device="cuda") - 1
    rope[at, 0], rope[at, 1] = 4.0, 0.0
    pool[:, 512:] = rope.to(torch.bfloat16).view(torch.uint8)
    scale[:] = 0.5
    q = torch.zeros(batch, nodes, HEADS, 576, device="cuda")
    q[..., :512] = 0.05 * torch.randn(HEADS, 512, generator=g, device="cuda")
    lift = torch.tensor(gaps, device="cuda").float()[torch.arange(HEADS, device="cuda") % len(gaps)]
    # (the latent values' share of the score is taken out of the gap)
    share = SCALE * 0.5 * (q[0, 0, :, :512].to(torch.bfloat16).float() @ (latent[1].view(torch.float8_e4m3fn).float()
                                                                          - latent[0].view(torch.float8_e4m3fn).float()))
    q[..., 512] = (lift - share) / (SCALE * 0.5 * 4.0)
    q[..., 513] = spread / (SCALE * 0.5)
    order = torch.arange(keys, dtype=torch.int32, device="cuda").expand(batch, keys).contiguous()
    return dict(q=q.to(torch.bfloat16), pool=pool, scale=scale, slot=order,
                lens=torch.full((batch,), keys, dtype=torch.int32, device="cuda"),
                parent=torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda").expand(batch, nodes).contiguous(),
                tree=torch.arange(keys, slots, dtype=torch.int32, device="cuda").expand(batch, nodes).contiguous())


def units(d, hint):
    """Units of the work, as the library plans them here."""
    batch, nodes, heads, _ = d["q"].shape
    out, size = (ctypes.c_int32 * 3)(), ctypes.c_int64()
    keys = d["slot"].shape[1]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert ddtree.lib().ddtree_internal_kv8_plan(
        ctypes.byref(ddtree.make_dims(batch, nodes, heads, d["pool"].shape[0], keys, keys, hint)), sms, out, ctypes.byref(size)) == 0
    return out[2]


def run(d):
    batch, nodes, heads, _ = d["q"].shape
    keys = d["slot"].shape[1]
    v = ddtree.Kv8Verifier(batch, nodes, heads, d["pool"].shape[0], keys, prefix_len_sum=min(batch * keys, 2 ** 31 - 1))
    out, lse = v(d["q"], d["pool"], d["scale"], d["slot"], d["lens"], d["parent"], d["tree"], SCALE)
    assert v.status() == 0
    return out, lse


def check(d, out, lse, node=0):
    keys = d["slot"].shape[1]
    rows = torch.cat([d["pool"][:, :512].view(torch.float8_e4m3fn).float(),
                      d["pool"][:, 512:].contiguous().view(torch.bfloat16).float()], 1)
    k = rows[:keys + node + 1].double() * d["scale"][0].double()
    s = SCALE * (d["q"][0, node].double() @ k.T)
    ref_l = torch.logsumexp(s, -1)
    w = torch.softmax(s, -1)
    ref = w @ k[:, :512]
    size, most = w @ k[:, :512].abs(), k[:, :512].abs().amax(0)
    for b in {0, out.shape[0] // 2, out.shape[0] - 1}:
        assert bool(((lse[b, node].double() - ref_l).abs() <= 2.0 ** -10).all())
        e = (out[b, node].double() - ref).abs()
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -9 * size + 2.0 ** -9 * w.amax(1)[:, None] * most
        assert bool((e <= tol).all()), (b, [round(float(x), 3) for x in (e / tol).amax(1)])


GAPS = [6.0, 8.0, 9.0, 10.0, 11.0, 12.0, 13.0, 14.0]


@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("keys,batch", [(8192, 256), (32768, 152)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_one_unit_a_request(keys, batch, where, spread):
    at = dict(first=0, middle=keys // 2 + 5, last=keys - 1)[where]
    d = make(keys, batch, GAPS, spread, at, seed=keys)
    assert units(d, batch * keys) == batch
    out, lse = run(d)
    check(d, out, lse)


@pytest.mark.parametrize("keys", [700, 8192, 131072, 600000])
def test_split_requests(keys):
    d = make(keys, 1, GAPS, 0.5, 3, seed=2)
    out, lse = run(d)
    check(d, out, lse)


@pytest.mark.parametrize("batch,nodes,keys", [(64, 33, 8192), (4, 128, 32768)])
def test_trees(batch, nodes, keys):
    """Groups of 64 rows, whose references are raised together."""
    d = make(keys, batch, GAPS, 0.5, 0, nodes=nodes, seed=3)
    out, lse = run(d)
    for node in (0, nodes // 2, nodes - 1):
        check(d, out, lse, node)


def test_scores_that_climb():
    """The largest key comes again and again: references are raised all along, and the tail before them keeps its share."""
    d = make(20000, 256, [0.0], 6.0, 0, seed=4)
    rope = torch.linspace(-1, 1, 20001, device="cuda")
    view = d["pool"][:, 512:].contiguous().view(torch.bfloat16)
    view[:, 1] = rope.to(torch.bfloat16)
    d["pool"][:, 512:] = view.view(torch.uint8)
    out, lse = run(d)
    check(d, out, lse)
