"""Attention over the 8-bit cache where one unit of the work has very many keys, against fp64.

Sums of the second product are cut to fp32, always towards zero, and what falls below a weight's parts is left out; a
unit starts its sums anew every 32768 keys and joins them in fp32, so neither grows with the prefix. Tolerances as for
shorter units (test_gpu_kv8_tail.py).
"""
import ctypes
import math

import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from test_gpu_kv8_tail import GAPS, HEADS, SCALE, _cuda, check, make, run, units  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("where", ["first", "second segment", "last"])
@pytest.mark.parametrize("keys,batch,spread", [(32769, 152, 0.5), (40000, 256, 0.5), (131072, 152, 0.0), (131072, 152, 0.5),
                                               (600000, 152, 0.5)])
def test_a_tail_behind_one_key(keys, batch, where, spread):
    at = {"first": 0, "second segment": 32768, "last": keys - 1}[where]
    d = make(keys, batch, GAPS if keys < 600000 else [9.0, 11.0, 12.0, 13.0, 14.0, 15.0, 16.0], spread, at, seed=keys)
    assert units(d, min(batch * keys, 2 ** 31 - 1)) == batch
    out, lse = run(d)
    check(d, out, lse)
    again, lse2 = run(d)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_sums_of_one_sign_over_two_million_keys():
    """All weights but a few are alike, all values positive: every cut of a sum has one sign."""
    keys, batch = 2_000_003, 152
    pool, scale = ddtree.kv8_pool(2)
    latent = (1 + torch.arange(512, device="cuda") % 8 / 8).to(torch.float8_e4m3fn)
    pool[:, :512] = latent.view(torch.uint8)
    rope = torch.zeros(2, 64, device="cuda")
    rope[1, 0] = 1.0
    pool[:, 512:] = rope.to(torch.bfloat16).view(torch.uint8)
    slot = torch.zeros(batch, keys, dtype=torch.int32, device="cuda")
    slot[:, ::64] = 1
    q = torch.zeros(batch, 1, HEADS, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 512] = 0.25
    v = ddtree.Kv8Verifier(batch, 1, HEADS, 2, keys, prefix_len_sum=batch * keys)
    d = dict(q=q, pool=pool, slot=slot)
    assert units(d, batch * keys) == batch
    out, lse = v(q, pool, scale, slot, torch.full((batch,), keys, dtype=torch.int32, device="cuda"),
                 torch.full((batch, 1), -1, dtype=torch.int32, device="cuda"),
                 torch.zeros(batch, 1, dtype=torch.int32, device="cuda"), 1.0)
    assert v.status() == 0
    k = latent.double()
    assert bool(((out.double() - k).abs() <= (2.0 ** -8 + 2.0 ** -10) * k).all())
    high = -(-keys // 64)
    assert bool(((lse.double() - math.log(keys + 1 - high + high * math.exp(0.25))).abs() <= 2.0 ** -13).all())


def test_units_of_split_requests():
    """One request, 65 nodes of 128 heads: seven units a group, of 85715 keys each, that are merged."""
    keys, nodes, heads = 600000, 65, 128
    d = make(keys, 1, GAPS, 0.5, 7, nodes=nodes, seed=5)
    d["q"] = d["q"].repeat(1, 1, heads // HEADS, 1).contiguous()
    out, lse = run(d)
    for node in (0, 32, 64):
        check(d, out, lse, node)


def test_one_long_request_among_very_many():
    """More than 1024 requests have a unit each, however long they are."""
    keys, batch = 200000, 1100
    d = make(keys, 1, GAPS, 0.5, 3, seed=6)
    slot = torch.zeros(batch, keys, dtype=torch.int32, device="cuda")
    slot[70] = d["slot"][0]
    slot[:70, :50] = slot[71:141, :50] = 9
    lens = torch.full((batch,), 50, dtype=torch.int32, device="cuda")
    lens[70] = keys
    q = d["q"].expand(batch, 1, HEADS, 576).contiguous()
    v = ddtree.Kv8Verifier(batch, 1, HEADS, d["pool"].shape[0], keys)
    out, lse = v(q, d["pool"], d["scale"], slot, lens, torch.full((batch, 1), -1, dtype=torch.int32, device="cuda"),
                 d["tree"].expand(batch, 1).contiguous(), SCALE)
    assert v.status() == 0
    check(dict(d, q=q[70:71], slot=slot[70:71]), out[70:71], lse[70:71])
    assert torch.equal(out[0], out[100]) and torch.equal(lse[0], lse[100])


@pytest.mark.parametrize("levels", [(0.0, -140.0, -2.0, -1.0), (-140.0, 0.0, -140.0, -3.0), (-60.0, -40.0, -20.0, 0.0),
                                    (0.0, -20.0, -40.0, -150.0)])
def test_segments_of_very_different_scores(levels):
    """Every 32768 keys another level of the scores and other values; in one of them a tile without a key."""
    keys, batch = 4 * 32768 + 77, 152
    d = make(keys, batch, [0.0], 75.0, 0, seed=8)
    g = torch.Generator(device="cuda").manual_seed(9)
    part = (torch.arange(d["pool"].shape[0], device="cuda") // 32768).clamp(max=3)
    d["pool"][:, :512] = torch.randn(4, 512, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)[part]
    rope = torch.zeros(d["pool"].shape[0], 64, device="cuda")
    rope[:, 1] = (torch.tensor(levels, device="cuda") / 75.0)[part] + 0.01 * torch.rand(len(part), generator=g, device="cuda")
    d["pool"][:, 512:] = rope.to(torch.bfloat16).view(torch.uint8)
    d["q"][..., :512] = 0
    out, lse = run(d)
    check(d, out, lse)
    # a segment's first tiles without a key (of the even and of the odd set), and a whole segment
    for lo, hi in ((32768, 32768 + 64), (65536, 65536 + 200), (32768, 65536)):
        e = dict(d, slot=d["slot"].clone())
        e["slot"][:, lo:hi] = -1
        v = ddtree.Kv8Verifier(batch, 1, HEADS, d["pool"].shape[0], keys, prefix_len_sum=batch * keys)
        got, got_l = v(e["q"], e["pool"], e["scale"], e["slot"], e["lens"], e["parent"], e["tree"], SCALE)
        assert v.status() == ddtree.STATUS_BAD_SLOT
        order = torch.cat([torch.arange(lo), torch.arange(hi, keys + 1)]).cuda()
        f = dict(d, pool=d["pool"][order], slot=d["slot"][:, :keys - (hi - lo)])
        check(f, got, got_l)


def test_a_key_that_is_not_finite_in_an_early_segment():
    d = make(70000, 152, GAPS, 0.5, 3, seed=10)
    d["slot"][5, 100], d["slot"][6, 40000] = 70001, 70001
    pool, scale = ddtree.kv8_pool(70002)
    pool[:70001], scale[:70001] = d["pool"], d["scale"]
    scale[70001] = math.nan
    d["pool"], d["scale"] = pool, scale
    out, lse = run(d)
    bad = torch.zeros(152, dtype=torch.bool, device="cuda")
    bad[5:7] = True
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    assert torch.equal(out[~bad], out[:1].expand_as(out[~bad])) and bool(torch.isfinite(out[0]).all())


def test_workspace_holds_the_segments():
    """Where units may have more than one segment, the workspace has room for their sums."""
    def size(batch, keys):
        n, plan = ctypes.c_int64(), (ctypes.c_int32 * 3)()
        d = ddtree.make_dims(batch, 1, HEADS, 1, keys, keys, min(batch * keys, 2 ** 31 - 1))
        assert ddtree.lib().ddtree_internal_kv8_plan(ctypes.byref(d), 152, plan, ctypes.byref(n)) == 0
        assert plan[2] == batch
        return n.value
    short, long = size(304, 32767), size(304, 32768)
    assert 304 * HEADS * 513 * 4 <= long - short <= 304 * HEADS * 513 * 4 + 512
