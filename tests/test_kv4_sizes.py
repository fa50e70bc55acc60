"""Workspace sizes of the 4-bit cache's attention, on any host: for every batch that the checks let
through, also an empty one, and never less than the joins of the parts need."""
import ctypes
import itertools

import pytest

from trellis_coded_bit_amd import binding as tb


@pytest.mark.parametrize("head_dim", [128, 256])
@pytest.mark.parametrize("page_size", [16, 256])
def test_attn_workspace_sizes(head_dim, page_size):
    p = 0x1000000
    for heads, group, n_seq, rows, max_pages in itertools.product(
            (1, 8, 1024), (1, 4, 64), (0, 1, 2, 300), (0, 1, 15, 4096, 100000), (1, 7, 4096)):
        if rows and not n_seq:
            continue
        c = tb.CKV4Cache(p, 1, 10, page_size, heads, head_dim)
        b = tb.CKV4Batch()
        b.table = b.lens = b.cu = p
        b.slots = None
        b.n_slots = max(n_seq, 1)
        b.n_seq, b.rows, b.max_pages = n_seq, rows, max_pages
        nb = tb.lib().trellis_kv4_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads * group)
        assert nb >= 65536, (heads, group, n_seq, rows, max_pages, tb.lib().trellis_last_error())
        # a sum of the parts of every column at most 64 times, and of a full grid of narrow tiles twice
        cols = rows * group * heads + 64 * heads * max(n_seq, 1)
        assert nb <= 65536 + 256 + (64 * cols + 2 * 16 * 4096) * (head_dim + 8) * 4
