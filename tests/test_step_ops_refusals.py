"""Host-side checks of the 8-bit cache's entry points and of the check of drafted tokens (no GPU work is reached here)."""
import ctypes

import pytest

from speculative_decoding_tree_05_gb300 import ddtree

A = lambda k: 0x10000000 * k  # noqa: E731  aligned addresses, far apart, that no check may follow


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_tree_05_gb300 import build
    build.build()
    return ddtree.lib()


def dims(**kw):
    d = dict(batch=2, nodes=9, heads=16, pool_slots=4096, slot_stride=256, max_prefix_len=256)
    d.update(kw)
    return ddtree.make_dims(**d)


WRITE = dict(rows=A(1), row_stride=576, slots=A(2), n=100, norm=A(3), eps=1e-6, rotation=A(4), position=A(5), positions=64,
             interleaved=0, pool=A(6), scale=A(7), pool_slots=4096, workspace=A(8), stream=None)
READ = dict(pool=A(1), scale=A(2), slots=A(3), n=100, rows=A(4), row_stride=576, pool_slots=4096, workspace=A(5), stream=None)
ATTN = dict(q=A(1), pool=A(2), scale=A(3), slot_idx=A(4), prefix_len=A(5), parent=A(6), tree=A(7), tree_len=A(8), sm=0.1,
            out=A(9), lse=A(10), dims="dims", workspace=A(11), bytes=1 << 30, stream=None)
ACCEPT = dict(logits=A(1), fp32=0, stride=1000, vocab=1000, draft=A(2), draft_stride=1000, tokens=A(3), parent=A(4),
              tree_len=A(5), uniform=A(6), temperature=A(7), path=A(8), path_len=A(9), next_token=A(10), dims="dims",
              workspace=A(11), bytes=1 << 20, stream=None)


def call(lib, fn, args, d=None, **change):
    assert set(change) <= set(args)
    full = {**args, **change}
    return getattr(lib, fn)(*[ctypes.byref(d) if v == "dims" else v for v in full.values()])


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=(1 << 31) + 1), dict(row_stride=575), dict(row_stride=577),
                                 dict(row_stride=0), dict(pool_slots=0), dict(pool_slots=(1 << 31) + 1)])
def test_row_sizes(lib, bad):
    assert call(lib, "ddtree_kv8_write", WRITE, **bad) == -2
    assert call(lib, "ddtree_kv8_read", READ, **bad) == -2


@pytest.mark.parametrize("bad", [dict(eps=0.0), dict(eps=-1.0), dict(eps=2.0), dict(eps=float("nan")), dict(positions=0)])
def test_norm_and_rotation_arguments(lib, bad):
    assert call(lib, "ddtree_kv8_write", WRITE, **bad) == -2


def test_no_rows_is_ok(lib):
    assert call(lib, "ddtree_kv8_write", WRITE, **{k: None for k, v in WRITE.items() if k != "n" and isinstance(v, int) and v >= A(1)}, n=0) == 0
    assert call(lib, "ddtree_kv8_read", READ, **{k: None for k, v in READ.items() if k != "n" and isinstance(v, int) and v >= A(1)}, n=0) == 0


@pytest.mark.parametrize("name", ["rows", "slots", "position", "pool", "scale", "workspace"])
def test_write_null_and_misaligned(lib, name):
    if name != "workspace":
        assert call(lib, "ddtree_kv8_write", WRITE, **{name: None}) == -1
    assert call(lib, "ddtree_kv8_write", WRITE, **{name: WRITE[name] + 2}) == -4


@pytest.mark.parametrize("name", ["rows", "slots", "pool", "scale", "workspace"])
def test_read_null_and_misaligned(lib, name):
    if name != "workspace":
        assert call(lib, "ddtree_kv8_read", READ, **{name: None}) == -1
    assert call(lib, "ddtree_kv8_read", READ, **{name: READ[name] + 2}) == -4


def test_row_overlaps(lib):
    pool, rows = 4096 * 640, 100 * 1152
    for change in (dict(rows=A(6) + pool - 16), dict(rows=A(6) - rows + 16), dict(rows=A(7)), dict(scale=A(6) + 64),
                   dict(slots=A(6)), dict(slots=A(7) + 16)):
        assert call(lib, "ddtree_kv8_write", WRITE, **change) == -7, change
    for change in (dict(rows=A(1) + pool - 16), dict(rows=A(2)), dict(rows=A(3) - rows + 16)):
        assert call(lib, "ddtree_kv8_read", READ, **change) == -7, change


@pytest.mark.parametrize("bad", [dict(nodes=0), dict(nodes=129), dict(heads=0), dict(heads=1025), dict(batch=-1),
                                 dict(batch=65536), dict(max_prefix_len=-1), dict(slot_stride=100, max_prefix_len=256),
                                 dict(pool_slots=0), dict(slot_stride=(1 << 30) + 1, max_prefix_len=(1 << 30) + 1)])
def test_attention_sizes(lib, bad):
    assert call(lib, "ddtree_verify_attn_kv8", ATTN, dims(**bad)) == -2


def test_attention_pointers(lib):
    assert call(lib, "ddtree_verify_attn_kv8", {**ATTN, "dims": None}) == -1
    assert call(lib, "ddtree_verify_attn_kv8", {k: None if isinstance(v, int) and v >= A(1) and k != "bytes" else v
                                                for k, v in ATTN.items()}, dims(batch=0)) == 0
    for name in ("q", "pool", "scale", "slot_idx", "prefix_len", "parent", "tree", "out", "lse", "workspace"):
        assert call(lib, "ddtree_verify_attn_kv8", ATTN, dims(), **{name: None}) == -1, name
        assert call(lib, "ddtree_verify_attn_kv8", ATTN, dims(), **{name: ATTN[name] + 2}) == -4, name
    assert call(lib, "ddtree_verify_attn_kv8", ATTN, dims(), tree_len=A(8) + 1) == -4


@pytest.mark.parametrize("bad", [dict(nodes=0), dict(nodes=129), dict(batch=-1), dict(batch=65536)])
def test_accept_sizes(lib, bad):
    assert call(lib, "ddtree_accept", ACCEPT, dims(**bad)) == -2
    assert lib.ddtree_accept_workspace_bytes(ctypes.byref(dims(**bad)), 1000) == 0


@pytest.mark.parametrize("bad", [dict(vocab=0), dict(vocab=(1 << 18) + 1, stride=1 << 19), dict(stride=999),
                                 dict(draft_stride=999)])
def test_accept_vocab(lib, bad):
    assert call(lib, "ddtree_accept", ACCEPT, dims(), **bad) == -2


def test_accept_pointers(lib):
    assert call(lib, "ddtree_accept", {**ACCEPT, "dims": None}) == -1
    assert call(lib, "ddtree_accept", {k: None if isinstance(v, int) and v >= A(1) and k != "bytes" else v
                                       for k, v in ACCEPT.items()}, dims(batch=0)) == 0
    for name in ("logits", "tokens", "parent", "uniform", "temperature", "path", "path_len", "next_token", "workspace"):
        assert call(lib, "ddtree_accept", ACCEPT, dims(), **{name: None}) == -1, name
        assert call(lib, "ddtree_accept", ACCEPT, dims(), **{name: ACCEPT[name] + 1}) == -4, name
    assert call(lib, "ddtree_accept", ACCEPT, dims(), fp32=1, logits=A(1) + 2) == -4
    assert call(lib, "ddtree_accept", ACCEPT, dims(), bytes=255) == -3


def test_accept_overlaps(lib):
    n = 2 * 9 * 4
    for change in (dict(path=A(3)), dict(path=A(4) + n - 4), dict(path_len=A(5)), dict(next_token=A(6) + 68),
                   dict(path=A(1) + 18 * 2000 - 4), dict(path_len=A(8) + 68), dict(next_token=A(9) + 4), dict(path=A(2) + 400)):
        assert call(lib, "ddtree_accept", ACCEPT, dims(), **change) == -7, change


def test_binding_refuses_tensors_of_the_host():
    import torch
    pool, scale = torch.zeros(4, 640, dtype=torch.uint8), torch.ones(4)
    slots = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ddtree.kv8_write(torch.zeros(2, 576, dtype=torch.bfloat16), slots, pool, scale)
    with pytest.raises(ValueError, match="CUDA"):
        ddtree.kv8_read(pool, scale, slots)
    with pytest.raises(ValueError, match="CUDA"):
        ddtree.kv8_pool(4, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ddtree.Kv8Verifier(1, 1, 1, 4, 4, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ddtree.TreeAcceptor(1, 1, 4, device="cpu")
