"""What include/trellis_kv4.h promises of calls whose arguments are not as they should be, or far from
usual, on the GPU: a bound on the rows that is too small, lists to release with a bad entry, and
sequences' bounds out of order."""
import pytest
import torch

from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case
from test_gpu_kv4 import Setup, both, ints, random_pool

pytestmark = pytest.mark.gpu


def test_many_rows_under_too_small_a_bound():
    """max_rows chooses kernels and nothing else: a long prompt called with a bound of one row leaves no
    row unwritten, of itself or of the sequence behind it.  Its 8 heads have 8 x 16300 column tiles of 4
    over 128 tiles of keys: their count is below 2^24 and, with what a segment costs, above."""
    log_case("attn bound too small")
    length, Hk, heads = 16384, 8, 32
    st = Setup([length, 300], T=256, Hk=Hk, seed=40)
    new = [16300, 1]
    g = torch.Generator(device="cuda").manual_seed(41)
    q = torch.randn((sum(new), heads, 128), generator=g, device="cuda").half()
    cu = ints([0, new[0], sum(new)])
    want = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((sum(new), heads), float("nan"), device="cuda")
    ws = torch.zeros(tb.trellis_kv4_attn_workspace_bytes(st.cache, st.table, st.lens, cu, sum(new), heads), dtype=torch.uint8,
                     device="cuda")
    y = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, max_q=1, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert not bool(torch.isnan(y).any()) and not bool(torch.isnan(lse).any())
    assert bool((ws[:256 + 65536] == 0).all())  # no join is left waiting
    # both are within the formats' bound (2e-3 of the result, over a tensor) of the exact one
    for at in (0, 1, 8000, new[0] - 1, new[0]):
        assert (y[at].double() - want[at].double()).norm() <= 4e-3 * want[at].double().norm(), at
    assert (y.float() - want.float()).norm() <= 4e-3 * want.float().norm()


@pytest.mark.parametrize("length", [None, -1, -(1 << 31), 16 * 5 + 1, 1 << 30])
@pytest.mark.parametrize("n", [2, 4, 300, 1500])
def test_free_refuses_as_a_whole(n, length):
    """A list with a slot out of range, or a slot whose length is, releases none of the others."""
    log_case(f"free refuses n={n} length={length}")
    lens = [1 + (11 * i) % 48 for i in range(n)]
    st = Setup(lens, T=16, Hk=1, spare=3, fill=False)  # (tables of five pages)
    random_pool(st)
    args = (st.cache, st.table, st.lens, st.ref)
    slots = list(range(n))
    bad = n // 2
    if length is None:
        slots[bad] = n
    else:
        st.lens[bad] = length
    o, same = both(st)
    tb.clear_error_word()
    tb.trellis_kv4_free(*args, ints(slots))
    same()
    assert tb.error_word() == 4
    tb.clear_error_word()
    tb.trellis_kv4_free(*args, ints([i for i in range(n) if i != bad]))
    o.free([i for i in range(n) if i != bad])
    same()
    assert tb.error_word() == 0


@pytest.mark.parametrize("max_q", [0, 1])
@pytest.mark.parametrize("each", [1, 30])
@pytest.mark.parametrize("n", [1, 3, 64, 65, 300, 700])
@pytest.mark.parametrize("how", ["past the rows", "descending", "negative", "late start", "short"])
def test_bounds_out_of_order(how, n, each, max_q):
    """The sequences before the first bad bound are as ever; every row behind them is zero and says that
    it saw nothing."""
    log_case(f"attn bounds {how} n={n} each={each} max_q={max_q}")
    st = Setup([40 + i % 50 for i in range(n)], T=16, Hk=1, seed=42)
    rows = n * each
    g = torch.Generator().manual_seed(43)
    q = torch.randn((rows, 4, 128), generator=g).half().cuda()
    cu = [i * each for i in range(n + 1)]
    want = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints(cu), q, max_q=max_q)
    lse = torch.empty((rows, 4), device="cuda")
    tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints(cu), q, lse=lse, max_q=max_q)
    assert tb.error_word() == 0
    at = 2 * n // 3  # the first sequence that is bad; its rows are from at * each on
    if how == "past the rows":
        cu[at + 1] = rows + 1
    elif how == "descending":
        if at == 0:
            cu[1] = -1
        else:
            cu[at + 1] = cu[at] - 1
    elif how == "negative":
        cu[at + 1] = -(1 << 31)
    elif how == "late start":
        cu[0], at = 1, 0
    else:
        cu[n], at = rows - each, n - 1
    y = torch.full_like(q, float("nan"))
    got = torch.full_like(lse, float("nan"))
    tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints(cu), q, max_q=max_q, out=y, lse=got)
    assert tb.error_word() == 4
    tb.clear_error_word()
    good = at * each
    assert torch.equal(y[good:], torch.zeros_like(y[good:])) and bool((got[good:] == -torch.inf).all())
    # (the work may be split at other places: both are within the formats' bound of the exact result)
    assert (y[:good].float() - want[:good].float()).norm() <= 4e-3 * want[:good].float().norm()
    assert bool(((got[:good] - lse[:good]).abs() <= 1e-3 * (1 + lse[:good].abs())).all())
