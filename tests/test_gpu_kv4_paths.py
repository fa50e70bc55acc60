"""The paged 4-bit key/value cache on the GPU, where its attention takes one path or another:
sequences on both sides of the bound between the kernels for few and for many columns in one
call, keys split over workgroups, many sequences, bad pages among many rows, extreme values, and
the serving loop of the benchmark.  Helpers and tolerances are test_gpu_kv4's: their bounds
follow from the formats, and what is held in more bits than they allow for is within them too."""
import argparse

import numpy as np
import pytest
import torch

from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case
from test_gpu_kv4 import DT, Setup, check_attn, host, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,group,new", [
    (128, 4, [1, 24, 25, 40, 3]),       # columns 4, 96, 100, 160, 12
    (128, 1, [95, 96, 97, 1, 200]),
    (256, 6, [16, 17, 1, 0, 30]),
    (128, 64, [1, 2, 1]),
    (128, 7, [13, 14, 2]),
])
def test_few_and_many_columns_in_one_call(dtype, D, group, new):
    """Sequences of at most 96 columns and of more in one call, known and unknown bounds."""
    log_case(f"attn both kernels {dtype} D={D} group={group} new={new}")
    lens = [n + 150 * (b % 3) + 1 for b, n in enumerate(new)]
    st = Setup(lens, T=32, Hk=2, D=D, dtype=dtype, seed=20)
    check_attn(st, new, 2 * group, max_q=max(new))
    check_attn(st, new, 2 * group)
    check_attn(st, new, 2 * group, window=90, sinks=5)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("T,length,new,window,sinks", [
    (64, 6001, 40, 0, 0),
    (16, 6001, 25, 3000, 0),
    (256, 3333, 130, 0, 0),
    (32, 9000, 33, 4096, 700),
])
def test_many_columns_over_a_split_context(D, T, length, new, window, sinks):
    """Few column tiles and a long context: several workgroups share a column tile's keys.  The
    same bits every time."""
    log_case(f"attn split D={D} T={T} length={length} new={new} window={window} sinks={sinks}")
    st = Setup([length], T=T, Hk=1, D=D, dtype="bf16", seed=21)
    a = check_attn(st, [new], 4, window=window, sinks=sinks)
    for _ in range(3):
        assert torch.equal(a, check_attn(st, [new], 4, window=window, sinks=sinks))


@pytest.mark.parametrize("n", [63, 64, 65, 130, 300])
def test_many_sequences(n):
    """More sequences than one round of a workgroup's search takes, some empty, some without rows."""
    log_case(f"attn sequences {n}")
    g = np.random.default_rng(n)
    lens = [int(x) for x in g.integers(0, 300, n)]
    lens[0], lens[-1] = 0, 257
    st = Setup(lens, T=16, Hk=1, seed=22)
    new = [int(x) for x in g.integers(0, 3, n)]
    new[-1] = 1
    check_attn(st, new, 4, max_q=2)
    new[n // 2] = 60  # (more rows than tokens, perhaps)
    check_attn(st, new, 4)
    check_attn(st, new, 4, window=33, sinks=2)


@pytest.mark.parametrize("new", [2, 70])
def test_pages_missing_under_many_rows(new):
    """A page number out of range hides its tokens and is reported, unless no row can see them."""
    log_case(f"attn missing pages new={new}")
    length, T = 400, 16
    st = Setup([length], T=T, Hk=1, seed=23)
    q = torch.randn((new, 4, 128)).half().cuda()
    cu = ints([0, new])
    whole = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, window=100, max_q=new)
    assert tb.error_word() == 0
    # pages 0 .. of tokens that no row sees
    hidden = (length - new - 100 + 1) // T
    bad = st.table.clone()
    bad[0, :hidden] = 1 << 30
    y = tb.trellis_kv4_attn(st.cache, 0, bad, st.lens, cu, q, window=100, max_q=new)
    assert torch.equal(y, whole) and tb.error_word() == 0
    # a page that rows do see: as if its tokens were masked
    bad = st.table.clone()
    page = (length - new - 20) // T
    bad[0, page] = st.cache.n_pages
    y = tb.trellis_kv4_attn(st.cache, 0, bad, st.lens, cu, q, max_q=new)
    torch.cuda.synchronize()
    assert tb.error_word() == 4
    tb.clear_error_word()
    k, v = (t.double() for t in tb.trellis_kv4_read(st.cache, 0, st.table, st.lens, ints([0, length]), length))
    i = torch.arange(length, device="cuda")
    for r in range(new):
        seen = (i <= length - new + r) & ((i // T) != page)
        w = torch.softmax((k[:, 0] @ q[r].double().T).T * 128 ** -0.5 + torch.where(seen, 0.0, -torch.inf), -1)
        want = w @ v[:, 0]
        # the cache's own rounding to fp16 on reading back, beside the attention's bound
        assert (y[r].double() - want).norm() <= 4e-3 * want.norm()


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 2.0 ** 60, 2.0 ** 100])
def test_values_of_any_size(new, size):
    """The weights' powers of two follow the values': results scale with them exactly enough."""
    log_case(f"attn value size {size} new={new}")
    length = 300
    st = Setup([length], T=16, Hk=1, dtype="bf16", seed=24, fill=False)
    g = torch.Generator().manual_seed(25)
    k, v = (torch.randn((length, 1, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn((new, 4, 128), generator=g).to(torch.bfloat16).cuda()
    cu = ints([0, length])
    out = []
    for f in (1.0, size):
        tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, cu, k, (v.float() * f).to(torch.bfloat16))
        out.append(tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, new]), q, max_q=new).double() / f)
    # scales and codes are the same but for the power of two, and so are the sums but where they are
    # split against it: both within the format's bound of the exact result
    assert (out[0] - out[1]).norm() <= 2 * 4e-3 * out[0].norm()
    assert tb.error_word() == 0


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -14, 2.0 ** 12])
def test_queries_of_any_size(new, size):
    """Queries that vanish (every key weighs the same) and ones that leave one key."""
    log_case(f"attn query size {size} new={new}")
    st = Setup([500], T=64, Hk=2, seed=26)
    q = (torch.randn((new, 8, 128)) * size).half().cuda()
    if size > 1:
        # (the tolerance of a weight grows with the spread of scores: only its largest key matters here)
        y = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, new]), q, max_q=new)
        assert bool(torch.isfinite(y).all()) and tb.error_word() == 0
    else:
        check_attn(st, [new], 8, q=q, max_q=new)


@pytest.mark.parametrize("new", [1, 64])
def test_queries_that_are_not_finite(new):
    """A NaN or an infinity in a query makes that row and head NaN, and no other."""
    log_case(f"attn query NaN new={new}")
    st = Setup([200], T=16, Hk=2, seed=27)
    q = torch.randn((new, 8, 128)).half().cuda()
    cu = ints([0, new])
    clean = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, max_q=new)
    bad = q.clone()
    bad[0, 3, 5] = float("nan")
    bad[new - 1, 6, 127] = float("inf")
    y = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, bad, max_q=new)
    hit = torch.zeros((new, 8), dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[new - 1, 6] = True
    assert bool(torch.isnan(y[hit]).all())
    assert torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,Hk,D", [(16400, 4, 128), (1100, 32, 256), (4099, 8, 128)])
def test_append_and_read_long_calls(dtype, rows, Hk, D):
    """Calls long enough for several blocks a workgroup give the bits of short calls."""
    log_case(f"append long {dtype} rows={rows} Hk={Hk} D={D}")
    st = Setup([rows], T=64, Hk=Hk, D=D, dtype=dtype, seed=28, fill=False)
    g = torch.Generator().manual_seed(29)
    k, v = (torch.randn((rows, Hk, D), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, ints([0, rows]), k, v)
    whole = st.cache.pool.clone()
    rk, rv = tb.trellis_kv4_read(st.cache, 0, st.table, st.lens, ints([0, rows]), rows, DT[dtype])
    st.cache.pool.fill_(0xFF)
    step = 64
    for at in range(0, rows, step):
        n = min(step, rows - at)
        tb.trellis_kv4_append(st.cache, 0, st.table, ints([at + n]), ints([0, n]), k[at:at + n], v[at:at + n])
    assert torch.equal(st.cache.pool, whole)
    for at in (0, rows // 2, rows - 7):
        n = min(step, rows - at)
        sk, sv = tb.trellis_kv4_read(st.cache, 0, st.table, ints([at + n]), ints([0, n]), n, DT[dtype])
        assert torch.equal(sk, rk[at:at + n]) and torch.equal(sv, rv[at:at + n])
    assert tb.error_word() == 0


@pytest.mark.parametrize("new", [1, 64])
def test_attn_on_another_stream(new):
    """Called on a stream of the program's own, with tensors of it, beside work on the default one."""
    log_case(f"attn stream new={new}")
    st = Setup([900, 300], T=16, Hk=2, seed=30)
    q = torch.randn((2 * new, 8, 128)).half().cuda()
    cu = ints([0, new, 2 * new])
    want = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, max_q=new)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q2 = q.clone()
        got = [tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q2, max_q=new) for _ in range(3)]
    for _ in range(3):
        assert torch.equal(tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, max_q=new), want)
    s.synchronize()
    for y in got:
        assert torch.equal(y, want)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_serving_loop(window, sinks):
    """The benchmark's serving loop, small: it checks its attention and its pages itself."""
    log_case(f"serving loop window={window}")
    import bench
    from trellis_coded_bit_amd import synth
    args = argparse.Namespace(seed=0, warmup=3, steps=8)
    out = bench.run_serve(args, torch, tb, synth, n_layers=2, prompt=192, chunk=96, samples=3, page=16, window=window,
                          sinks=sinks, keep_first=5, keep_last=50)
    assert out["tokens_kept"] == 55 and out["rel_err_decode"] < 2e-3
