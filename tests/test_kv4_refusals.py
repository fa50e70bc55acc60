"""Arguments of the key/value cache's calls that the host has to refuse, or has not to, on any host: sizes
that no launch could have."""
import ctypes

import pytest

from trellis_coded_bit_amd import binding as tb

P = 0x1000000  # (never read: the calls end before anything is enqueued)


@pytest.mark.parametrize("n_keep", [(1 << 27) + 1, 1 << 28, 1 << 30, -1])
def test_compaction_of_more_than_a_grid_holds(n_keep):
    """The copy takes 16 threads a kept token: from 2^28 tokens on their number leaves 32 bits."""
    c = tb.CKV4Cache(P, 1, 10, 16, 1, 128)
    st = tb.lib().trellis_kv4_compact(ctypes.byref(c), P, P, 4, 10, P, P, P, 1, P, P, n_keep, P, 1 << 30, None)
    assert st == -1 and b"n_keep" in tb.lib().trellis_last_error()
