"""The error word of the library-held workspace: it is sticky, also where a larger call replaces the
buffer.  On any host, with a stand-in for the stream, and on the GPU as it comes about."""
import pytest
import torch

from trellis_coded_bit_amd import binding as tb


@pytest.mark.parametrize("capturing", [False, True])
def test_growing_keeps_the_error_word(monkeypatch, capturing):
    cpu = torch.device("cpu", 0)
    monkeypatch.setattr(tb, "_ws", {})
    monkeypatch.setattr(tb, "_stream", lambda: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    assert tb.error_word() == 0
    a = tb.workspace(1000, cpu)
    a[:4].view(torch.int32)[0] = 8
    b = tb.workspace(2000, cpu)
    assert b.numel() >= 2000 and tb.error_word() == 8
    b[:4].view(torch.int32)[0] |= 1
    assert tb.workspace(1500, cpu) is b
    c = tb.workspace(5000, cpu)
    assert c is not b and tb.error_word() == 9 and bool((c[4:] == 0).all())
    tb.clear_error_word()
    assert tb.error_word() == 0 and tb.error_word(c) == 0
    monkeypatch.setattr(tb, "_stream", lambda: 9)  # another stream's is its own
    assert tb.workspace(300, cpu) is not c and tb.error_word() == 0


@pytest.mark.gpu
def test_refused_reserve_before_a_larger_call():
    """A reserve that was refused is still known after an attention call whose workspace is larger."""
    from gpu_util import log_case
    from test_gpu_kv4 import Setup, ints
    log_case("error word over growth")
    with torch.cuda.stream(torch.cuda.Stream()):
        tb._ws.pop((0, tb._stream()), None)  # (its number may be one that was used before)
        st = Setup([5000, 40], T=64, Hk=1, spare=1)
        tb.trellis_kv4_reserve(st.cache, st.table, st.lens, st.ref, ints([128, 0]))
        before = tb._ws[(0, tb._stream())]
        q = torch.ones((2, 4, 128), dtype=torch.float16, device="cuda")
        tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, 1, 2]), q)
        assert tb._ws[(0, tb._stream())] is not before  # it has grown
        assert tb.error_word() == 8
        tb.clear_error_word()
        assert tb.error_word() == 0
