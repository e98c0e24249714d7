"""The division of attention over the 8-bit cache into units: what the host plans, and what the kernels make of it."""
import ctypes
import random

import pytest

from speculative_decoding_tree_05_gb300 import ddtree


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_tree_05_gb300 import build
    build.build()
    return ddtree.lib()


def plan(lib, sms=152, **kw):
    d = dict(batch=1, nodes=9, heads=16, pool_slots=1 << 20, slot_stride=4096, max_prefix_len=4096)
    d.update(kw)
    out, size = (ctypes.c_int32 * 3)(), ctypes.c_int64()
    rc = lib.ddtree_internal_kv8_plan(ctypes.byref(ddtree.make_dims(**d)), sms, out, ctypes.byref(size))
    assert rc == 0
    return out[0], out[1], out[2], size.value


def units_of(tiles, shares):
    """Units of each request, as the kernels count them: a share is ceil(all / shares) tiles."""
    share = max(1, -(-sum(tiles) // shares))
    return [-(-n // share) for n in tiles]


def test_units_fit_the_grid_whatever_the_lengths(lib):
    r = random.Random(5)
    for _ in range(300):
        batch, most = r.choice([1, 2, 3, 8, 64, 500, 1024]), r.choice([0, 1, 64, 5000, 200000])
        hint = r.choice([0, 1, most * batch // 2])
        groups, shares, units, _ = plan(lib, batch=batch, slot_stride=most, max_prefix_len=most, heads=r.choice([1, 16, 128]),
                                        prefix_len_sum=min(hint, 2 ** 31 - 1))
        assert shares >= 1 and units == shares + batch - 1
        lens = [r.choice([0, most, r.randint(0, most)]) for _ in range(batch)]
        tree = [r.choice([0, 9, r.randint(0, 9)]) for _ in range(batch)]
        tiles = [0 if t == 0 else -(-(n + t) // 64) for n, t in zip(lens, tree)]
        counts = units_of(tiles, shares)
        assert sum(counts) <= units
        for n, c in zip(tiles, counts):
            cuts = [n * k // c for k in range(c + 1)] if c else []
            assert (c == 0) == (n == 0) and all(b > a for a, b in zip(cuts, cuts[1:]))   # no unit is empty


def test_groups(lib):
    for nodes, heads, want in ((1, 1, 1), (9, 16, 3), (65, 128, 130), (128, 1024, 2048), (64, 1, 1), (65, 1, 2), (5, 100, 10)):
        assert plan(lib, nodes=nodes, heads=heads)[0] == want


def test_large_batches_have_a_unit_a_request(lib):
    assert plan(lib, batch=1025)[1:3] == (0, 1025)
    assert plan(lib, batch=65535, nodes=128, heads=1024)[1:3] == (0, 65535)


def test_a_long_request_fills_the_device_and_a_short_one_does_not_split_far(lib):
    groups, shares, units, _ = plan(lib, slot_stride=185000, max_prefix_len=185000)
    assert groups * units <= 152 and groups * (units + 1) > 152
    assert plan(lib, slot_stride=40, max_prefix_len=40)[1] == 1
    groups, shares, _, _ = plan(lib, nodes=65, heads=128, slot_stride=65536, max_prefix_len=65536)
    waves = -(-groups * shares // 152)
    assert groups * shares > 0.9 * waves * 152   # whole waves


def test_no_partials_without_a_split(lib):
    image = 128 * 512 + 64 * 128 + 256            # a group's query rows
    assert plan(lib, slot_stride=40, max_prefix_len=40)[3] == 512 + 3 * image
    # more groups than SMs: their units cut the query rows themselves
    assert plan(lib, batch=51, slot_stride=40, max_prefix_len=40)[1] == 1
    assert plan(lib, batch=50, slot_stride=40, max_prefix_len=40)[3] == 768 + 150 * image
    assert plan(lib, batch=51, slot_stride=40, max_prefix_len=40)[3] == 768
    groups, shares, units, size = plan(lib, slot_stride=185000, max_prefix_len=185000)
    assert size == 512 + 3 * image + -(-units * 144 * 4 // 256) * 256 + units * 144 * 512 * 4
