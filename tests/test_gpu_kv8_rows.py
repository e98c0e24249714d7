"""Rows into the 8-bit latent cache and back (ddtree_kv8_write, ddtree_kv8_read) against 64-bit arithmetic.

Tolerances, from the arithmetic.  A latent value is rounded once to 4 significant bits (half a step: 2^-4 of it), below
2^-6 scales to half of 2^-9 scales; a rope value once to bf16 (2^-8 of it).  Before that, fp32: the norm is a sum of 512
squares (a lane adds 16, five levels of pairs: at most 21 roundings), a division, a square root and two products, within
32 units of 2^-24 (16 of the sum through the square root, and the rest); a rotation two products and a sum.
Rows without norm and rotation are powers of two times their bf16 values up to the rounding, so they are compared bit
for bit.
"""
import math

import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def make(n, slots, seed=0, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = (amp * torch.randn(n, 576, generator=g, device="cuda")).to(torch.bfloat16)
    where = torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32)
    pool = torch.randint(0, 120, (slots, 640), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand(slots, generator=g, device="cuda")
    return rows, where, pool, scale


def rounded(x, bits, lowest):
    step = torch.exp2(torch.clamp(torch.frexp(x).exponent.double() - bits, min=lowest))
    return torch.round(x / step) * step


def stored(pool, scale, slots):
    """The values of listed slots in 64 bits, decoded from the bytes."""
    raw = pool[slots]
    byte = raw[:, :512].int()
    power, frac = (byte >> 3) & 15, (byte & 7).double()
    size = torch.where(power > 0, (1 + frac / 8) * torch.exp2((power - 7).double()), frac * 2.0 ** -9)
    rope = raw[:, 512:].contiguous().view(torch.bfloat16).double()
    return torch.cat([torch.where(byte >= 128, -size, size), rope], 1) * scale[slots].double()[:, None]


@pytest.mark.parametrize("n,slots,amp", [(1, 1, 1.0), (7, 9, 1e-3), (8, 4096, 300.0), (1000, 1000, 1e30),
                                         (4099, 70000, 1e-20)])
def test_plain_rows_bit_for_bit(n, slots, amp):
    rows, where, pool, scale = make(n, slots, seed=n, amp=amp)
    before, before_scale = pool.clone(), scale.clone()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ddtree.kv8_write(rows, where, pool, scale, workspace=ws)
    assert ddtree.read_device_status(ws) == 0
    x, at = rows.double(), where.long()
    top = x[:, :512].abs().amax(1)
    want = torch.exp2(torch.clamp(torch.ceil(torch.log2(top / 448)), min=-60))
    assert torch.equal(scale[at].double(), want)
    ref = torch.cat([rounded(x[:, :512] / want[:, None], 4, -9), x[:, 512:] / want[:, None]], 1) * want[:, None]
    assert torch.equal(stored(pool, scale, at), ref)
    rest = torch.ones(slots, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(pool[rest], before[rest]) and torch.equal(scale[rest], before_scale[rest])
    assert torch.equal(ddtree.kv8_read(pool, scale, where).double(), ref)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("turn", ["none", "halves", "pairs"])
@pytest.mark.parametrize("n,amp,eps", [(1, 1.0, 1e-6), (333, 5.0, 1e-5), (64, 1e-4, 1e-6), (64, 1e25, 1e-6), (33, 1e-16, 1e-12)])
def test_norm_and_rotation(norm, turn, n, amp, eps):
    rows, where, pool, scale = make(n, n + 100, seed=n + 7 * norm, amp=amp)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.exp(torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16) if norm else None
    table = position = None
    if turn != "none":
        a = 100 * torch.rand(50, 32, generator=g, device="cuda")
        table = torch.cat([a.cos(), a.sin()], 1).contiguous()
        position = torch.randint(0, 50, (n,), generator=g, device="cuda", dtype=torch.int32)
    ddtree.kv8_write(rows, where, pool, scale, norm_weight=w, eps=eps, rotation=table, position=position,
                     interleaved=turn == "pairs")
    x = rows.double()
    c, r = x[:, :512], x[:, 512:].clone()
    if norm:
        c = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * w.double()
    size = r.abs()
    if turn != "none":
        i = torch.arange(32, device="cuda")
        i, j = (2 * i, 2 * i + 1) if turn == "pairs" else (i, i + 32)
        cos, sin = table[position.long()].double().split(32, 1)
        px, py = r[:, i].clone(), r[:, j].clone()
        r[:, i], r[:, j] = px * cos - py * sin, py * cos + px * sin
        size[:, i] = size[:, j] = px.abs() + py.abs()
    s = scale[where.long()].double()
    top = c.abs().amax(1)
    assert bool((torch.frexp(s).mantissa == 0.5).all())
    off = 32 * U if norm else 0.0
    low = torch.maximum(top * (1 - off) / 448, torch.tensor(2.0 ** -60, device="cuda", dtype=torch.float64))
    assert bool((s >= low).all()) and bool((s <= torch.maximum(2 * top * (1 + off) / 448, torch.full_like(s, 2.0 ** -60))).all())
    got = stored(pool, scale, where.long())
    s = s[:, None]
    assert bool(((got[:, :512] - c).abs() <= c.abs() * (2.0 ** -4 + 2 * off) + 2.0 ** -10 * s).all())
    assert bool(((got[:, 512:] - r).abs() <= r.abs() * 2.0 ** -8 + 4 * U * size + 2.0 ** -133 * s).all())
    back = ddtree.kv8_read(pool, scale, where).double()
    assert torch.equal(back, got)


def test_rows_and_results_inside_wider_tensors():
    rows, where, pool, scale = make(37, 64, seed=1)
    wide = torch.full((37, 600 + 8), 1e30, device="cuda", dtype=torch.bfloat16)
    wide[:, 16:592] = rows
    other, other_scale = pool.clone(), scale.clone()
    ddtree.kv8_write(rows, where, pool, scale)
    ddtree.kv8_write(wide[:, 16:592], where, other, other_scale)
    assert torch.equal(pool, other) and torch.equal(scale, other_scale)
    out = torch.full((37, 640), 7.0, device="cuda", dtype=torch.bfloat16)
    ddtree.kv8_read(pool, scale, where, out=out[:, 32:608])
    assert torch.equal(out[:, 32:608], ddtree.kv8_read(pool, scale, where))
    assert bool((out[:, :32] == 7).all()) and bool((out[:, 608:] == 7).all())


def test_skipped_and_bad_rows_leave_the_cache():
    rows, where, pool, scale = make(40, 100, seed=2)
    table = torch.ones(10, 64, device="cuda")
    position = torch.zeros(40, dtype=torch.int32, device="cuda")
    bad = where.clone()
    for i, v in ((0, -1), (5, 100), (6, -2), (7, 2 ** 31 - 1), (8, -2 ** 31)):
        bad[i] = v
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ref_pool, ref_scale = pool.clone(), scale.clone()
    keep = [i for i in range(40) if i not in (0, 5, 6, 7, 8, 20, 21)]
    ddtree.kv8_write(rows[keep].contiguous(), where[keep], ref_pool, ref_scale, rotation=table, position=position[keep])
    only = bad.clone()
    only[5:9] = -1
    position[20], position[21] = 10, -1
    ddtree.kv8_write(rows, only, pool, scale, rotation=table, position=position, workspace=ws)
    assert ddtree.read_device_status(ws) == ddtree.STATUS_BAD_POSITION
    ddtree.kv8_write(rows, bad, pool, scale, rotation=table, position=position, workspace=ws)
    assert ddtree.read_device_status(ws) == ddtree.STATUS_BAD_POSITION | ddtree.STATUS_BAD_SLOT
    assert torch.equal(pool, ref_pool) and torch.equal(scale, ref_scale)
    got = ddtree.kv8_read(pool, scale, bad, workspace=ws)
    assert ddtree.read_device_status(ws) == ddtree.STATUS_BAD_SLOT
    assert not bool(got[[0, 5, 6, 7, 8]].any()) and torch.equal(got[9:], ddtree.kv8_read(pool, scale, where[9:]))
    quiet_pool, quiet_scale = pool.clone(), scale.clone()      # without a workspace nothing is reported
    ddtree.kv8_write(rows, bad, quiet_pool, quiet_scale, rotation=table, position=position)
    assert torch.equal(quiet_pool, pool) and torch.equal(ddtree.kv8_read(quiet_pool, quiet_scale, bad), got)
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    got = ddtree.kv8_read(pool, scale, none, workspace=ws)
    assert ddtree.read_device_status(ws) == 0 and not bool(got.any())


def test_rows_that_are_not_finite_zero_or_uneven():
    rows, where, pool, scale = make(8, 8, seed=3)
    rows[0, 3], rows[1, 500], rows[2, 575] = math.nan, math.inf, -math.inf
    rows[3] = 0
    rows[4, :512] = 0                       # rope values alone
    rows[5, :512] = 1e-38                   # far below the smallest scale
    rows[6, 512:] = 3e38                    # rope values that the latent scale cannot hold
    rows[6, :512] = 1e-10
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    ddtree.kv8_write(rows, where, pool, scale)
    at = where.long()
    assert bool(torch.isnan(scale[at[:3]]).all()) and not bool(pool[at[:3]].any())
    back = ddtree.kv8_read(pool, scale, where)
    assert bool(torch.isnan(back[:3]).all()) and not bool(back[3].any())
    assert torch.equal(back[4, 512:], rows[4, 512:]) and not bool(back[5, :512].any())
    assert torch.equal(back[6, 512:], rows[6, 512:]) and bool(torch.isfinite(back[3:]).all())
    ddtree.kv8_write(rows, where, pool, scale, norm_weight=w)    # the norm does not hide them
    assert bool(torch.isnan(scale[at[:3]]).all()) and bool(torch.isfinite(ddtree.kv8_read(pool, scale, where[3:])).all())


def test_the_same_slot_read_often_and_an_empty_list():
    rows, where, pool, scale = make(5, 9, seed=4)
    ddtree.kv8_write(rows, where, pool, scale)
    often = where[2:3].expand(1000).contiguous()
    got = ddtree.kv8_read(pool, scale, often)
    assert torch.equal(got, got[:1].expand(1000, 576))
    before = pool.clone()
    ddtree.kv8_write(rows[:0], where[:0], pool, scale)
    assert ddtree.kv8_read(pool, scale, where[:0]).shape == (0, 576) and torch.equal(pool, before)


def test_slots_beyond_31_bits_of_bytes():
    slots = (1 << 31) // 640 + 1000
    rows, _, _, _ = make(100, 100, seed=5)
    pool, scale = ddtree.kv8_pool(slots)
    where = torch.arange(slots - 100, slots, dtype=torch.int32, device="cuda")
    ddtree.kv8_write(rows, where, pool, scale)
    small, small_scale = ddtree.kv8_pool(100)
    here = torch.arange(100, dtype=torch.int32, device="cuda")
    ddtree.kv8_write(rows, here, small, small_scale)
    assert torch.equal(ddtree.kv8_read(pool, scale, where), ddtree.kv8_read(small, small_scale, here))
    assert not bool(pool[:slots - 100].any())


def test_captured_and_on_another_stream():
    rows, where, pool, scale = make(64, 200, seed=6)
    ref_pool, ref_scale = pool.clone(), scale.clone()
    ddtree.kv8_write(rows, where, ref_pool, ref_scale)
    want = ddtree.kv8_read(ref_pool, ref_scale, where)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p2, s2 = pool.clone(), scale.clone()
    torch.cuda.synchronize()
    ddtree.kv8_write(rows, where, p2, s2, stream=side)
    got = ddtree.kv8_read(p2, s2, where, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.zeros_like(rows)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ddtree.kv8_write(rows, where, pool, scale, workspace=ws)
        ddtree.kv8_read(pool, scale, where, out=out, workspace=ws)
    rows.copy_(2 * rows)
    graph.replay()
    assert torch.equal(out, (2 * want.float()).to(torch.bfloat16))
