"""Arguments of the key/value cache's calls that the host has to refuse, or has not to, on any host: sizes
that no launch could have, strides that nothing uses."""
import ctypes
import types

import pytest
import torch

from trellis_coded_bit_amd import binding as tb

P = 0x1000000  # (not memory: the calls end before anything is enqueued)


@pytest.mark.parametrize("n_keep", [(1 << 27) + 1, 1 << 28, 1 << 30, -1])
def test_compaction_of_more_than_a_grid_holds(n_keep):
    """The copy takes 16 threads a kept token: from 2^28 tokens on their number leaves 32 bits."""
    c = tb.CKV4Cache(P, 1, 10, 16, 1, 128)
    # (without a workspace: a count that passed would be refused for that, not launched on these pointers)
    st = tb.lib().trellis_kv4_compact(ctypes.byref(c), P, P, 4, 10, P, P, P, 1, P, P, n_keep, None, 0, None)
    assert st == -1 and b"n_keep" in tb.lib().trellis_last_error()


def test_strides_that_nothing_uses():
    """One row, or one head, of a buffer whose rows are not multiples of 8 elements apart."""
    cache = types.SimpleNamespace(device=torch.device("cpu"), head_dim=128)
    odd = torch.zeros((3, 5 * 128 + 4), dtype=torch.float16)
    assert tb._kv4_rows(cache, odd[:1, :384].view(1, 3, 128), 3, "k") == (0, 128)
    assert tb._kv4_rows(cache, odd[:1, :128].as_strided((1, 1, 128), (7, 9, 1)), 1, "k") == (0, 0)
    wide = torch.zeros((3, 5, 128), dtype=torch.float16)
    assert tb._kv4_rows(cache, wide[:, 1:2], 1, "k") == (640, 0)
    assert tb._kv4_rows(cache, wide[:, 1:3], 2, "k") == (640, 128)
    assert tb._kv4_rows(cache, odd.as_strided((3, 2, 128), (644, 128, 1)), 2, "k") == (644, 128)  # (the library refuses)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 2])
def test_one_row_of_an_odd_buffer(heads):
    from gpu_util import log_case
    from test_gpu_kv4 import Setup, ints
    log_case(f"kv4 one row of an odd buffer heads={heads}")
    st = Setup([50], T=16, Hk=heads)
    n = heads * 128
    x = torch.randn((4, 6 * n + 4), device="cuda").half()
    k, v, q = (x[2:3].narrow(1, at * n, m * n).view(1, m * heads, 128) for at, m in ((0, 1), (1, 1), (2, 4)))
    cu = ints([0, 1])
    got = []
    for t in ((k, v, q), tuple(y.contiguous() for y in (k, v, q))):
        tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, cu, t[0], t[1])
        got.append((st.cache.pool.clone(), tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, t[2])))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert tb.error_word() == 0
