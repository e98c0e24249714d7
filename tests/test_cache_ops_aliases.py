"""Host-side checks of buffers that overlap (no GPU work is reached here)."""
import pytest

from speculative_decoding_tree_05_gb300 import ddtree
from test_cache_ops_refusals import WEIGHT, call, change, dims, lib  # noqa: F401

TABLE = 2 * 256 * 4    # bytes of the table of dims()
OLD = 0x400000


def weigh(lib, old, out, decay):  # noqa: F811
    args = change(change(change(WEIGHT, 8, decay), 9, old), 10, out)
    return call(lib, "ddtree_kv_weight", args, dims())


@pytest.mark.parametrize("shift", [4, TABLE // 2, TABLE - 4, -4, 4 - TABLE])
def test_weights_that_overlap_in_part(lib, shift):  # noqa: F811
    assert weigh(lib, OLD, OLD + shift, 0.5) == -7


@pytest.mark.parametrize("shift,decay", [(0, 0.5), (TABLE, 0.5), (-TABLE, 1.0), (4, 0.0)])
def test_weights_in_place_apart_or_not_read(lib, shift, decay):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would run on these addresses")
    assert weigh(lib, OLD, OLD + shift, decay) == -6


def test_the_message_names_no_other_call(lib):  # noqa: F811
    """The code is eviction's and key weights' too, not kv_compact's alone."""
    text = ddtree.status_string(-7)
    assert text.startswith("an output overlaps an input or another output")
