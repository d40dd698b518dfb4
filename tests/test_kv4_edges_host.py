"""Refusals of tensors whose elements overlap where they are written, by the C entry points (every
call here fails its host checks, so no pointer is followed), and of views of a pool that do not
hold its pages, by the binding."""
import pytest

from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from test_kv4_host import CALLS, FAKE, INVALID, STRIDE, U8, _z

FAR = FAKE << 16
ATTENTION = [FAKE, 8192, 128, FAKE, STRIDE, 10, 64, FAKE, FAKE, 90000, 4, 64, 8, 128, 0.1, FAR, 8192, 128, FAKE, 64, FAKE,
             1 << 40, None]
PAGED = [FAKE, 8192, 128, FAKE, STRIDE, 10, 64, FAKE, 1600, FAKE, 0, 2, 2, 100000, 64, 8, 128, 0.1, FAR, 8192, 128, None, 0,
         FAKE, 1 << 40, None]
PREFILL = [FAKE, 8192, 128, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, FAKE, 2, 100, 1000, 64, 8, 128, 0.1, 1, FAR, 8192, 128,
           FAKE, 64, FAKE, 1 << 30, None]
GATHER = [FAKE, STRIDE, 10, 64, 8, 128, FAKE, 8, 8, FAKE, None, 2, 100, FAR, 1024, 128, 2 * FAR, 1024, 128, None]
WEIGHTS = [FAKE, 8192, 128, FAKE, STRIDE, 10, 64, FAKE, 16, FAKE, 0, 2, 2, 1000, 64, 8, 128, 0.1, FAKE, 64, 1, FAR, 9000,
           1000, 1000, 2 * FAR, 9000, 1000, None]
EVICT = [FAR, 9000, 1000, 1000, 2 * FAR, 2, 8, 128, 100, 10, 0, FAKE, STRIDE, 10, 64, 3 * FAR, 16, 16, 4 * FAR, 2, 2, 5 * FAR,
         6 * FAR, 7 * FAR, FAKE, 1 << 30, None]


@pytest.mark.parametrize("name,args,changes", [
    # rows, or heads, on top of one another; heads within a row's reach; the same with heads outermost
    ("idx_kv4_attention", ATTENTION, {16: 0}), ("idx_kv4_attention", ATTENTION, {16: 8184}),
    ("idx_kv4_attention", ATTENTION, {16: 128, 17: 504}), ("idx_kv4_attention", ATTENTION, {16: 64, 17: 8192}),
    ("idx_paged_kv4_attention", PAGED, {19: 0}), ("idx_paged_kv4_attention", PAGED, {19: 8184}),
    ("idx_grouped_prefill", PREFILL, {20: 0}), ("idx_grouped_prefill", PREFILL, {20: 128, 21: 128 * 99}),
    ("idx_kv4_gather", GATHER, {14: 0}), ("idx_kv4_gather", GATHER, {17: 1016}),
    # keys and values of one place, a row apart, and beside one another by a part
    ("idx_kv4_gather", GATHER, {16: FAR}), ("idx_kv4_gather", GATHER, {16: FAR + 2048}),
    ("idx_kv4_gather", GATHER, {14: 2048, 17: 2048, 16: FAR + 2048 - 16}), ("idx_kv4_gather", GATHER, {16: FAR + 32, 17: 2048}),
    # sums shared by sequences, by heads, by a column
    ("idx_paged_kv4_weights", WEIGHTS, {26: 0}), ("idx_paged_kv4_weights", WEIGHTS, {27: 0}),
    ("idx_paged_kv4_weights", WEIGHTS, {27: 999}), ("idx_paged_kv4_weights", WEIGHTS, {26: 7999}),
    ("idx_paged_kv4_weights", WEIGHTS, {26: 1000, 27: 1999}),
    # in place under strides that overlap, and sums that are another view of what they add to
    ("idx_paged_kv4_weights", WEIGHTS, {21: 2 * FAR, 22: 0, 26: 0}), ("idx_paged_kv4_weights", WEIGHTS, {21: 2 * FAR + 4}),
    ("idx_paged_kv4_weights", WEIGHTS, {21: 2 * FAR - 4 * 999}), ("idx_paged_kv4_weights", WEIGHTS, {21: 2 * FAR + 4 * 1000}),
    ("idx_paged_kv4_weights", WEIGHTS, {21: 2 * FAR + 4 * 9000}), ("idx_paged_kv4_weights", WEIGHTS, {21: 2 * FAR + 4, 23: 0}),
    # an eviction's outputs among its inputs and one another
    ("idx_kv4_evict", EVICT, {22: 2 * FAR}), ("idx_kv4_evict", EVICT, {23: FAR}), ("idx_kv4_evict", EVICT, {23: FAR + 4 * 16999}),
    ("idx_kv4_evict", EVICT, {21: 3 * FAR + 4 * 31}), ("idx_kv4_evict", EVICT, {22: 4 * FAR + 12}),
    ("idx_kv4_evict", EVICT, {21: 7 * FAR}), ("idx_kv4_evict", EVICT, {22: 5 * FAR + 4 * 1599})])
def test_written_elements_overlap(name, args, changes):
    a = list(args)
    for at, value in changes.items():
        a[at] = value
    assert getattr(B.lib(), name)(*a) == INVALID


@pytest.mark.parametrize("name,at", [("store", 2), ("gather", 0), ("attention", 1), ("paged", 1), ("weights", 1), ("evict", 4)])
def test_rows_narrower_than_a_page(name, at):
    """The stride of such a view is a page's, its rows are not: bytes outside it were touched."""
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        args = good()
        args[at] = _z(4, B.kv4_page_bytes(64, 2), d=U8)[:, :64 * 2 * 136 - 1]
        with pytest.raises(ValueError, match="bytes a page"):
            f(*args)
        args[at] = _z(4, B.kv4_page_bytes(64, 2) + 48, d=U8)[:, :64 * 2 * 136]
        with pytest.raises(ValueError, match="CUDA"):  # wide enough: the next check
            f(*args)
