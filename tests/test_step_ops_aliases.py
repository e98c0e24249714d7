"""Inputs of ddtree_kv8_write that lie inside the cache it writes are refused (no GPU work is reached here)."""
import pytest

from test_step_ops_refusals import A, WRITE, call, lib  # noqa: F401

POOL, SCALES = 4096 * 640, 4096 * 4
BYTES = dict(norm=512 * 2, rotation=64 * 64 * 4, position=100 * 4)


@pytest.mark.parametrize("name", ["norm", "rotation", "position"])
@pytest.mark.parametrize("buffer,size", [("pool", POOL), ("scale", SCALES)])
def test_norm_and_rotation_inside_the_cache(lib, name, buffer, size):  # noqa: F811
    at = WRITE[buffer]
    for where in (at, at + size - 16, at - BYTES[name] + 16):
        assert call(lib, "ddtree_kv8_write", WRITE, **{name: where}) == -7, (name, buffer, where - at)

