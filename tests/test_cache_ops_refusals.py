"""Host-side checks of the cache-size and block-sparse entry points (no GPU work is reached here)."""
import ctypes

import pytest

from speculative_decoding_tree_05_gb300 import ddtree

P = 0x10000  # an aligned address that no check may follow


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_tree_05_gb300 import build
    build.build()
    return ddtree.lib()


def dims(**kw):
    d = dict(batch=2, nodes=9, heads=16, pool_slots=4096, slot_stride=256, max_prefix_len=256)
    d.update(kw)
    return ddtree.make_dims(**d)


def call(lib, fn, args, d):
    """args: a list, ints as they are; the dims go where the word "dims" stands."""
    full = [ctypes.byref(d) if a == "dims" and d is not None else (None if a == "dims" else a) for a in args]
    return getattr(lib, fn)(*full)


WEIGHT = [P, P, P, P, P, None, 0, 0.1, 0.0, None, P, "dims", P, 1 << 30, None]
EVICT = [0x100000, 0x200000, 0x300000, 0x310000, 4, 8, 0x400000, 0x500000, 0x600000, 0x700000, "dims", P, None]
SUMMARY = [P, P, P, None, 64, P, P, "dims", P, None]
SELECT = [P, P, P, P, 64, 4, 0, 1, P, "dims", P, 1 << 30, None]
BLOCKS = [P, P, P, P, P, P, P, 64, 4, 0.1, P, P, "dims", P, 1 << 30, None]
ALL = [("ddtree_kv_weight", WEIGHT), ("ddtree_kv_evict", EVICT), ("ddtree_block_summary", SUMMARY),
       ("ddtree_block_select", SELECT), ("ddtree_verify_attn_blocks", BLOCKS)]


def change(args, at, value):
    out = list(args)
    out[at] = value
    return out


@pytest.mark.parametrize("fn,args", ALL)
def test_sizes_and_empty_batches(lib, fn, args):
    assert call(lib, fn, args, None) == -1
    for bad in (dict(nodes=0), dict(nodes=129), dict(heads=0), dict(batch=-1), dict(max_prefix_len=-1),
                dict(slot_stride=100, max_prefix_len=256), dict(pool_slots=0)):
        assert call(lib, fn, args, dims(**bad)) == -2
    empty = [0 if a == P or (isinstance(a, int) and a >= 0x100000 and a != 1 << 30) else a for a in args]
    assert call(lib, fn, empty, dims(batch=0)) == 0


@pytest.mark.parametrize("fn,args,at", [
    ("ddtree_kv_weight", WEIGHT, 0), ("ddtree_kv_weight", WEIGHT, 1), ("ddtree_kv_weight", WEIGHT, 2),
    ("ddtree_kv_weight", WEIGHT, 4), ("ddtree_kv_weight", WEIGHT, 10), ("ddtree_kv_weight", WEIGHT, 12),
    ("ddtree_kv_evict", EVICT, 0), ("ddtree_kv_evict", EVICT, 3), ("ddtree_kv_evict", EVICT, 8),
    ("ddtree_kv_evict", EVICT, 9), ("ddtree_block_summary", SUMMARY, 0), ("ddtree_block_summary", SUMMARY, 5),
    ("ddtree_block_select", SELECT, 0), ("ddtree_block_select", SELECT, 8), ("ddtree_verify_attn_blocks", BLOCKS, 6),
    ("ddtree_verify_attn_blocks", BLOCKS, 10), ("ddtree_verify_attn_blocks", BLOCKS, 13)])
def test_null_pointers(lib, fn, args, at):
    assert call(lib, fn, change(args, at, None), dims()) == -1


@pytest.mark.parametrize("fn,args,at,value", [
    ("ddtree_kv_weight", WEIGHT, 0, P + 8), ("ddtree_kv_weight", WEIGHT, 12, P + 16), ("ddtree_kv_weight", WEIGHT, 10, P + 2),
    ("ddtree_kv_evict", EVICT, 0, 0x100002), ("ddtree_kv_evict", EVICT, 11, P + 4), ("ddtree_block_summary", SUMMARY, 5, P + 4),
    ("ddtree_block_select", SELECT, 1, P + 2), ("ddtree_verify_attn_blocks", BLOCKS, 10, P + 8),
    ("ddtree_verify_attn_blocks", BLOCKS, 6, P + 1)])
def test_alignment(lib, fn, args, at, value):
    assert call(lib, fn, change(args, at, value), dims()) == -4


def test_arguments(lib):
    d = dims()
    assert call(lib, "ddtree_kv_weight", change(change(WEIGHT, 6, -1), 5, P), d) == -2
    assert call(lib, "ddtree_kv_weight", change(WEIGHT, 6, 3), d) == -1             # nodes chosen, no list
    assert call(lib, "ddtree_kv_weight", change(WEIGHT, 8, 0.5), d) == -1           # decay without old weights
    assert call(lib, "ddtree_kv_weight", change(change(WEIGHT, 6, 65536), 5, P), d) == -2
    assert call(lib, "ddtree_kv_evict", change(EVICT, 4, -1), d) == -2
    assert call(lib, "ddtree_kv_evict", change(EVICT, 5, -1), d) == -2
    for block in (0, 8, 24, 256, -64):
        assert call(lib, "ddtree_block_summary", change(SUMMARY, 4, block), d) == -2
        assert call(lib, "ddtree_block_select", change(SELECT, 4, block), d) == -2
        assert call(lib, "ddtree_verify_attn_blocks", change(BLOCKS, 7, block), d) == -2
    for topk in (0, -1, (1 << 20) + 1):
        assert call(lib, "ddtree_block_select", change(SELECT, 5, topk), d) == -2
        assert call(lib, "ddtree_verify_attn_blocks", change(BLOCKS, 8, topk), d) == -2
    assert call(lib, "ddtree_block_select", change(SELECT, 6, -1), d) == -2
    assert call(lib, "ddtree_block_select", change(SELECT, 7, -1), d) == -2


@pytest.mark.parametrize("fn,args", ALL)
def test_longest_prefix(lib, fn, args):
    far = dims(batch=1, slot_stride=(1 << 30) + 1, max_prefix_len=(1 << 30) + 1)
    assert call(lib, fn, args, far) == -2


def test_sizes_past_the_counters(lib):
    # 2^31 query rows and more, and more key tiles than the kernels count
    big = dims(batch=65535, nodes=128, heads=1024)
    assert call(lib, "ddtree_kv_weight", WEIGHT, big) == -2
    long = dims(batch=65535, slot_stride=1 << 30, max_prefix_len=1 << 30)
    assert call(lib, "ddtree_kv_weight", WEIGHT, long) == -2


@pytest.mark.parametrize("out", [6, 7, 8, 9])
def test_evict_overlap(lib, out):
    d = dims()
    for src in (0, 1, 2, 3):
        assert call(lib, "ddtree_kv_evict", change(EVICT, out, EVICT[src]), d) == -7
    other = 6 if out != 6 else 7
    assert call(lib, "ddtree_kv_evict", change(EVICT, out, EVICT[other] + 4), d) == -7
    assert call(lib, "ddtree_kv_evict", change(EVICT, 6, EVICT[0] + 2 * 256 * 4 - 4), d) == -7   # the last entry


def test_without_a_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for fn, args in ALL:
        assert call(lib, fn, args, dims()) == -6
    assert lib.ddtree_kv_weight_workspace_bytes(ctypes.byref(dims()), 0) == 0
    assert lib.ddtree_verify_blocks_workspace_bytes(ctypes.byref(dims()), 64, 4) == 0


def test_select_workspace_needs_no_gpu(lib):
    n = lib.ddtree_block_select_workspace_bytes(ctypes.byref(dims()), 64)
    assert n >= 2 * 9 * 16 * (576 * 2 + 4) + 2 * 9 * 4 * 4
    assert lib.ddtree_block_select_workspace_bytes(ctypes.byref(dims()), 48) == 0
