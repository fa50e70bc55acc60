"""The paged 4-bit key/value cache on the GPU against the 64-bit oracle: append and read back,
attention (heads, types, page sizes, lengths from nothing to long, masks, strides), and the
page operations.

Tolerances of attention, from the formats alone.  A weight p is held in two E4M3 parts, each
rounded within 2^-4 of what it holds, so within 2^-8; a query element within 2^-12 (three
parts, or the 16-bit input itself), which moves a score by at most 2^-12 * spread
(spread = scale * sum |q_d k_d|) and so a weight by twice that at most; the output is rounded to
its type.  Per (row, head), in the 2-norm over its elements (the rotation keeps it):
    |y - ref| <= (2^-8 + 2 * 2^-12 * spread) * |sum p |v|| + u * |ref|,   u = 2^-11 or 2^-8.
Over a whole tensor the roundings are independent, and the library's relative L2 bound holds:
2e-3 in fp16, 4e-3 in bf16 (whose own rounding is up to 2^-9).
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv4 as KO
from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
REL = {"fp16": 2e-3, "bf16": 4e-3}
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """Sequences of the given lengths over pages in no order, the cache filled by append."""

    def __init__(self, lens, T=16, Hk=2, D=128, layers=1, dtype="fp16", seed=0, spare=4, extra_slots=0, layer=None, fill=True):
        g = torch.Generator().manual_seed(seed)
        need = [-(-l // T) for l in lens]
        n_pages = sum(need) + spare
        perm = torch.randperm(n_pages, generator=g).tolist()
        slots = len(lens) + extra_slots
        table = np.full((slots, max(need + [1]) + 2), -7, np.int32)
        ref = np.zeros(n_pages, np.int32)
        for b, n in enumerate(need):
            table[b, :n] = [perm.pop() for _ in range(n)]
            ref[table[b, :n]] = 1
        self.T, self.Hk, self.D, self.dtype = T, Hk, D, dtype
        self.host_lens = list(lens)
        self.table, self.ref = torch.from_numpy(table).cuda(), torch.from_numpy(ref).cuda()
        self.lens = ints(list(lens) + [0] * extra_slots)
        self.cache = tb.KV4Cache.allocate(layers, n_pages, T, Hk, D)
        # what no token wrote holds codes and NaN scales
        self.cache.pool.fill_(0xFF)
        self.layer = layers - 1 if layer is None else layer
        self.g = g
        if fill and sum(lens):
            self.k, self.v = (torch.randn((sum(lens), Hk, D), generator=g).to(DT[dtype]).cuda() for _ in range(2))
            self.cu = ints(np.concatenate([[0], np.cumsum(lens)]))
            tb.trellis_kv4_append(self.cache, self.layer, self.table, self.lens, self.cu, self.k, self.v,
                                  slots=ints(range(len(lens))))

    def oracle(self):
        return KO.Cache(self.cache.n_layers, self.cache.n_pages, self.T, self.Hk, self.D, self.cache.pool.cpu().numpy().copy())


def check_attn(st, new, heads, window=0, sinks=0, scale=None, max_q=0, q=None, seed=1, q_size=1.5, slots=None):
    g = torch.Generator().manual_seed(seed)
    rows = sum(new)
    if q is None:
        q = (q_size * torch.randn((rows, heads, st.D), generator=g)).to(DT[st.dtype]).cuda()
    cu = ints(np.concatenate([[0], np.cumsum(new)]))
    lse = torch.full((rows, heads), 9.0, device="cuda")
    out = torch.full((rows, heads, st.D), 9.0, dtype=DT[st.dtype], device="cuda")
    y = tb.trellis_kv4_attn(st.cache, st.layer, st.table, st.lens, cu, q, window=window, sinks=sinks, scale=scale,
                            max_q=max_q, out=out, lse=lse, slots=slots)
    assert y.data_ptr() == out.data_ptr()
    torch.cuda.synchronize()
    oc = st.oracle()
    table = st.table.cpu().numpy()
    sc = st.D ** -0.5 if scale is None else scale
    at, refs, got = 0, [], host(y)
    names = slots.tolist() if slots is not None else list(range(len(new)))
    for b, n in enumerate(new):
        if n == 0:
            continue
        length = st.host_lens[names[b]]
        k, v = (oc.rows(st.layer, table[names[b]], length, w) for w in (0, 1))
        ry, rl, mass, spread = KO.attention(host(q[at:at + n]), k, v, sc, window, sinks)
        refs.append(ry)
        err = np.linalg.norm(got[at:at + n] - ry, axis=-1)
        bound = (2.0 ** -8 + 2 * 2.0 ** -12 * spread) * np.linalg.norm(mass, axis=-1) + \
            UNIT[st.dtype] * np.linalg.norm(ry, axis=-1) + 1e-6
        assert (err <= bound).all(), (b, float((err / bound).max()))
        gl = host(lse[at:at + n])
        empty = np.isinf(rl)
        assert (gl[empty] == -np.inf).all() and (got[at:at + n][empty] == 0).all()
        assert (np.abs(gl[~empty] - rl[~empty]) <= 2.0 ** -11 * (1 + spread[~empty])).all()
        at += n
    ref = np.concatenate(refs)
    norm = np.linalg.norm(ref)
    if norm:
        assert np.linalg.norm(got - ref) / norm < REL[st.dtype]
    assert tb.error_word() == 0
    return y


# ---------------------------------------------------------------------------------------
# Append and read
# ---------------------------------------------------------------------------------------

def check_codes(st, x, which, positions):
    """Codes and scales of the appended rows against the oracle's; a code may differ where the
    64-bit value lies within 2^-17 of a midpoint (relative to the block's largest, 6: the
    butterflies' and the division's roundings are 9 * 2^-24 of it at most, doubled), a scale
    where the largest value lies that near a rounding boundary."""
    oc = st.oracle()
    table = st.table.cpu().numpy()
    for row, (slot, p) in enumerate(positions):
        page, t = int(table[slot, p // st.T]), p % st.T
        codes, s = oc.parts(st.layer, page, t, which)
        xr = host(x[row]).reshape(st.Hk, -1, 128)
        rc, rs = KO.quantize(xr)
        r = xr @ KO.H
        same = rs == s
        if not same.all():
            exact = np.abs(r).max(-1) / 6
            near = np.abs(KO.bf16_bits(exact * (1 + 2.0 ** -20)).astype(int) - KO.bf16_bits(exact * (1 - 2.0 ** -20)).astype(int))
            assert (near[~same] == 1).all()
        y = r / np.where(KO.bf16_value(s) == 0, 1, KO.bf16_value(s))[..., None]
        gap = np.abs(np.abs(y)[..., None] - KO.MIDPOINTS).min(-1)
        ok = (rc == codes) | (gap < 6 * 2.0 ** -17) | ((np.abs(y) < 2.0 ** -17) & ((rc ^ codes) == 8)) | ~same[..., None]
        assert ok.all(), (row, which)
        assert np.abs(KO.e2m1_values(codes) - KO.e2m1_values(rc))[same].max(initial=0) <= 2


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hk,D,lens,new", [
    (16, 1, 128, [1], [1]),
    (16, 2, 128, [17, 33, 5], [1, 1, 1]),
    (32, 3, 256, [70, 9, 40], [23, 0, 40]),
    (64, 8, 128, [130, 65], [130, 2]),
    (256, 2, 128, [300], [45]),
])
def test_append_codes_and_read(dtype, T, Hk, D, lens, new):
    log_case(f"append {dtype} T={T} Hk={Hk} D={D} lens={lens} new={new}")
    st = Setup(lens, T=T, Hk=Hk, D=D, layers=2, dtype=dtype, seed=3, fill=False)
    rows = sum(new)
    g = torch.Generator().manual_seed(4)
    x = torch.randn((rows, 2 * Hk + 1, D), generator=g)
    x[..., ::19] *= 9
    x = x.to(DT[dtype]).cuda()
    k, v = x[:, :Hk], x[:, Hk + 1:]  # slices of a wider buffer
    cu = ints(np.concatenate([[0], np.cumsum(new)]))
    before = st.cache.pool.clone()
    tb.trellis_kv4_append(st.cache, st.layer, st.table, st.lens, cu, k, v)
    positions = [(b, l - n + i) for b, (l, n) in enumerate(zip(lens, new)) for i in range(n)]
    check_codes(st, k, 0, positions)
    check_codes(st, v, 1, positions)
    # nothing else changed: as many bytes as the rows have, in this layer alone
    assert torch.equal(st.cache.pool[0], before[0])
    changed = (st.cache.pool != before).sum().item()
    assert changed <= rows * 132 * (D // 128) * Hk
    rk, rv = tb.trellis_kv4_read(st.cache, st.layer, st.table, st.lens, cu, rows, DT[dtype])
    oc, table = st.oracle(), st.table.cpu().numpy()
    at = 0
    for b, n in enumerate(new):
        for which, got in ((0, rk), (1, rv)) if n else ():
            ref = oc.rows(st.layer, table[b], lens[b], which)[lens[b] - n:]
            top = np.abs(ref).reshape(n, Hk, -1, 128).max(-1, keepdims=True) * np.ones(128)
            err = np.abs(host(got[at:at + n]) - ref)
            assert (err <= UNIT[dtype] * np.abs(ref) + 2.0 ** -18 * top.reshape(ref.shape)).all()
        at += n
    assert tb.error_word() == 0


def test_append_special_values():
    log_case("append special values")
    st = Setup([6], Hk=1, dtype="bf16", fill=False)
    x = torch.randn((6, 1, 128), dtype=torch.float32)
    x[0] = 0
    x[1, 0, 5] = float("nan")
    x[2, 0, 7] = float("-inf")
    x[3] = 1e-41       # below what a normal bf16 scale can hold
    x[4, 0] = 0
    x[4, 0, 0] = 3.0   # every rotated element at the largest magnitude
    x[5] *= 1e30
    k = x.to(torch.bfloat16).cuda()
    v = torch.ones_like(k)
    cu = ints([0, 6])
    tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, cu, k, v)
    rk, rv = tb.trellis_kv4_read(st.cache, 0, st.table, st.lens, cu, 6, torch.bfloat16)
    rk, rv = host(rk), host(rv)
    assert (rk[0] == 0).all() and (rk[3] == 0).all()
    assert np.isnan(rk[1]).all() and np.isnan(rk[2]).all()
    assert abs(rk[4, 0, 0] - 3.0) <= 3 * 2.0 ** -8 and np.abs(rk[4, 0, 1:]).max() <= 3 * 2.0 ** -8
    assert np.isfinite(rk[5]).all() and np.linalg.norm(rk[5] - host(k[5])) / np.linalg.norm(host(k[5])) < 0.2
    assert np.isfinite(rv).all()
    check_codes(st, k[4:5], 0, [(0, 4)])


def test_bad_places_are_skipped_and_flagged():
    """Page numbers, slots and lengths that are out of range: the rows are skipped (append) or
    zero (read, attention), and the error word says so."""
    log_case("bad places")
    st = Setup([40, 40, 40], T=16, Hk=2)
    tb.clear_error_word()
    good = st.cache.pool.clone()
    table = st.table.clone()
    table[0, 2] = st.cache.n_pages          # one past the last page
    table[1, 2] = -1
    lens = st.lens.clone()
    lens[2] = 1 << 29                       # far over the table
    cu = ints([0, 1, 2, 3])
    k = torch.ones((3, 2, 128), dtype=torch.float16, device="cuda")
    tb.trellis_kv4_append(st.cache, 0, table, lens, cu, k, k)
    assert tb.error_word() == 4
    assert torch.equal(st.cache.pool, good)
    tb.clear_error_word()
    rk, rv = tb.trellis_kv4_read(st.cache, 0, table, lens, cu, 3, torch.float16)
    assert (rk == 0).all() and (rv == 0).all() and tb.error_word() == 4
    tb.clear_error_word()
    # slots out of range, and rows past cu's end
    tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, ints([0, 1, 2]), k, k, slots=ints([3, -1]))
    assert torch.equal(st.cache.pool, good) and tb.error_word() == 4
    tb.clear_error_word()
    q = torch.ones((3, 2, 128), dtype=torch.float16, device="cuda")
    y = tb.trellis_kv4_attn(st.cache, 0, st.table, lens, ints([0, 1, 2]), q, slots=ints([2, 7]))
    assert (y == 0).all() and tb.error_word() == 4
    tb.clear_error_word()
    # a bad page inside a context: its keys are left out
    y = tb.trellis_kv4_attn(st.cache, 0, table, st.lens, cu, q)
    assert torch.isfinite(y).all() and tb.error_word() == 4
    tb.clear_error_word()


# ---------------------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hk,group,D,lens,new", [
    (16, 1, 1, 128, [1], [1]),
    (16, 2, 4, 128, [1, 2, 15, 16, 17, 31], [1] * 6),
    (16, 8, 4, 128, [777], [1]),
    (32, 2, 8, 128, [127, 128, 129, 500, 3], [1, 1, 1, 1, 1]),
    (64, 1, 16, 128, [900, 64], [1, 1]),
    (128, 2, 3, 128, [333, 0, 1000], [1, 0, 1]),
    (256, 1, 5, 128, [700], [3]),
    (16, 2, 6, 256, [130, 90, 1], [5, 3, 1]),
    (32, 1, 1, 256, [260], [1]),
    (64, 1, 64, 128, [150], [1]),
])
def test_attn_few_rows(dtype, T, Hk, group, D, lens, new):
    log_case(f"attn few rows {dtype} T={T} Hk={Hk} group={group} D={D} lens={lens} new={new}")
    st = Setup(lens, T=T, Hk=Hk, D=D, layers=2, dtype=dtype, seed=5)
    check_attn(st, new, Hk * group)
    check_attn(st, new, Hk * group, max_q=max(new))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hk,group,D,lens,new", [
    (16, 1, 1, 128, [65], [65]),
    (16, 2, 4, 128, [200, 150], [130, 150]),
    (64, 1, 8, 128, [300, 5, 77], [100, 5, 1]),
    (32, 2, 3, 256, [140, 260], [140, 61]),
    (128, 1, 5, 128, [400], [257]),
])
def test_attn_many_rows(dtype, T, Hk, group, D, lens, new):
    log_case(f"attn many rows {dtype} T={T} Hk={Hk} group={group} D={D} lens={lens} new={new}")
    st = Setup(lens, T=T, Hk=Hk, D=D, dtype=dtype, seed=6)
    check_attn(st, new, Hk * group, max_q=max(new))
    check_attn(st, new, Hk * group)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (100, 130), (128, 4), (129, 17), (5000, 4), (0, 50)])
@pytest.mark.parametrize("new", [1, 4, 90])
def test_attn_window_and_sinks(window, sinks, new):
    log_case(f"attn window={window} sinks={sinks} new={new}")
    lens = [700, 130, 90]
    st = Setup(lens, T=32, Hk=2, dtype="bf16" if sinks % 2 else "fp16", seed=7)
    check_attn(st, [min(new, l) for l in lens], 8, window=window, sinks=sinks, max_q=new)


def test_attn_rows_that_see_nothing():
    """More new rows than the sequence has tokens: the first ones stand before it and see nothing."""
    log_case("attn empty rows")
    st = Setup([3, 0, 40], T=16, Hk=2)
    for new in ([5, 2, 1], [70, 80, 64]):
        y = check_attn(st, new, 4)
        assert (y[:new[0] - 3] == 0).all()


def test_attn_slots_and_scales():
    log_case("attn slots")
    st = Setup([50, 300, 129, 20], T=16, Hk=1, layers=3, seed=8, layer=1)
    check_attn(st, [1, 2, 1], 4, slots=ints([3, 1, 0]))
    check_attn(st, [1, 40], 4, slots=ints([2, 1]), scale=0.3)
    check_attn(st, [1, 40], 4, slots=ints([2, 1]), scale=0.0)
    check_attn(st, [1, 1], 4, slots=ints([1, 1]), scale=-0.2)  # one sequence twice


@pytest.mark.parametrize("new", [1, 48])
def test_attn_sharp_and_flat(new):
    """Scores that leave one key, and scores that are all the same."""
    log_case(f"attn sharp and flat new={new}")
    st = Setup([1500], T=64, Hk=1, seed=9)
    check_attn(st, [new], 4, q_size=12.0)
    check_attn(st, [new], 4, q=torch.zeros((new, 4, 128), dtype=torch.float16, device="cuda"))


@pytest.mark.parametrize("new", [1, 80])
def test_attn_strided_queries(new):
    log_case(f"attn strided queries new={new}")
    st = Setup([260], T=16, Hk=2, dtype="bf16", seed=10)
    wide = torch.randn((new, 12, 128), dtype=torch.float32).to(torch.bfloat16).cuda()
    check_attn(st, [new], 8, q=wide[:, 2:10])
    swapped = torch.randn((8, new, 128), dtype=torch.float32).to(torch.bfloat16).cuda()
    check_attn(st, [new], 8, q=swapped.transpose(0, 1))


@pytest.mark.parametrize("new", [1, 64])
def test_attn_masked_places_may_hold_anything(new):
    """NaN scales past the length, outside the window and in other layers never reach a result;
    a visible NaN does, and only in its head."""
    log_case(f"attn masked NaN new={new}")
    st = Setup([200], T=16, Hk=2, seed=11)
    base = check_attn(st, [new], 4, window=64 + new, sinks=2)
    oc = st.oracle()
    table = st.table.cpu().numpy()
    for p in range(2, 200 - 64 - 2 * new):  # between the sinks and the first row's window
        for which in (0, 1):
            a = oc.at(which, 0, p % 16)[1]
            oc.pool[0, table[0, p // 16], :, a:a + 2] = 0xFF
    st.cache.pool.copy_(torch.from_numpy(oc.pool.reshape(st.cache.pool.shape)))
    again = check_attn(st, [new], 4, window=64 + new, sinks=2)
    assert torch.equal(base, again)
    # the last token's value of head 0 becomes NaN: its rows that see it are NaN, head 1's are not
    a = oc.at(1, 0, 199 % 16)[1]
    oc.pool[0, table[0, 199 // 16], 0, a:a + 2] = 0xFF
    st.cache.pool.copy_(torch.from_numpy(oc.pool.reshape(st.cache.pool.shape)))
    g = torch.Generator().manual_seed(1)
    q = (1.5 * torch.randn((new, 4, 128), generator=g)).half().cuda()
    y = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, new]), q, window=64 + new, sinks=2)
    assert torch.isnan(y[-1, :2]).all() and torch.equal(y[:, 2:], base[:, 2:]) and torch.equal(y[:-1], base[:-1])


def test_attn_long_and_repeatable():
    """A long context (split over the GPU and joined): right, and the same bits every time, on
    another stream too."""
    log_case("attn long")
    st = Setup([20011, 37], T=64, Hk=1, seed=12)
    q = torch.randn((2, 4, 128)).half().cuda()
    y = check_attn(st, [1, 1], 4, q=q)
    for _ in range(5):
        assert torch.equal(y, tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, 1, 2]), q))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, 1, 2]), q)
    torch.cuda.synchronize()
    assert torch.equal(y, z)


def test_attn_parts_join_by_lse():
    """A context attended in two halves and joined by the returned logarithms is the whole."""
    log_case("attn join by lse")
    st = Setup([512, 256, 256], T=64, Hk=1, seed=13)
    st.table[1, :4] = st.table[0, :4]
    st.table[2, :4] = st.table[0, 4:8]
    q = torch.randn((1, 4, 128)).half().cuda()
    lse = [torch.empty((1, 4), device="cuda") for _ in range(3)]
    y = [tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, 1]), q, slots=ints([s]), lse=lse[s]).float() for s in range(3)]
    w = torch.softmax(torch.stack(lse[1:]), 0)[..., None]
    joined = w[0] * y[1] + w[1] * y[2]
    assert (joined - y[0]).norm() / y[0].norm() < 2e-3
    assert (torch.logaddexp(lse[1], lse[2]) - lse[0]).abs().max() < 1e-3


def test_attn_offsets_past_32_bits():
    """Pages on both sides of 4 GiB from the pool's start, read and written there."""
    log_case("attn offsets past 4 GiB")
    T, Hk, D = 256, 8, 256
    nb = tb.trellis_kv4_page_bytes(T, Hk, D)
    n_pages = (5 << 30) // nb
    cache = tb.KV4Cache.allocate(1, n_pages, T, Hk, D)
    lens = [3 * T - 5]
    table = ints([n_pages - 1, 1, (4 << 30) // nb]).reshape(1, 3)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((lens[0], Hk, D), generator=g).half().cuda() for _ in range(2))
    cu = ints([0, lens[0]])
    tb.trellis_kv4_append(cache, 0, table, ints(lens), cu, k, v)
    rk, rv = tb.trellis_kv4_read(cache, 0, table, ints(lens), cu, lens[0])
    for x, r in ((k, rk), (v, rv)):
        assert (x.float() - r.float()).norm() / x.float().norm() < 0.2
    q = torch.randn((1, Hk, D), generator=g).half().cuda()
    y = tb.trellis_kv4_attn(cache, 0, table, ints(lens), ints([0, 1]), q)
    ry, _, _, _ = KO.attention(host(q), host(rk), host(rv), D ** -0.5)
    assert np.linalg.norm(host(y) - ry) / np.linalg.norm(ry) < REL["fp16"] + 2.0 ** -11


# ---------------------------------------------------------------------------------------
# Page operations
# ---------------------------------------------------------------------------------------

def both(st):
    """The GPU's state and the oracle's copy of it."""
    o = KO.Pages(st.oracle(), st.table.cpu().numpy().copy(), st.lens.cpu().numpy().copy(), st.ref.cpu().numpy().copy())

    def same():
        torch.cuda.synchronize()
        assert np.array_equal(st.lens.cpu().numpy(), o.lens)
        assert np.array_equal(st.ref.cpu().numpy(), o.ref)
        assert np.array_equal(st.table.cpu().numpy(), o.table)
        assert np.array_equal(st.cache.pool.cpu().numpy().reshape(o.c.pool.shape), o.c.pool)

    return o, same


def random_pool(st, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st.cache.pool.random_(0, 256, generator=g)


@pytest.mark.parametrize("T,Hk,D,layers", [(16, 2, 128, 3), (64, 1, 256, 2), (256, 1, 128, 1)])
def test_page_operations_follow_the_oracle(T, Hk, D, layers):
    log_case(f"pages T={T} Hk={Hk} D={D} layers={layers}")
    st = Setup([3 * T + 5, 2 * T, 7, 0], T=T, Hk=Hk, D=D, layers=layers, spare=30, extra_slots=6, fill=False)
    random_pool(st)
    o, same = both(st)
    args = (st.cache, st.table, st.lens, st.ref)
    tb.trellis_kv4_fork(*args, ints([0, 1, 2, 3, 0]), ints([4, 5, 6, 7, 8]))
    assert o.fork([0, 1, 2, 3, 0], [4, 5, 6, 7, 8])
    same()
    tb.trellis_kv4_reserve(*args, ints([1, T, 0, 2 * T - 5]), slots=ints([4, 1, 9, 8]))
    assert o.reserve([4, 1, 9, 8], [1, T, 0, 2 * T - 5])
    same()
    keeps = [list(range(0, 3 * T + 5, 2)), [6, 0, 3], []]
    cu = np.concatenate([[0], np.cumsum([len(k) for k in keeps])])
    tb.trellis_kv4_compact(*args, ints([0, 2, 5]), ints([0, 9, 5]), ints(sum(keeps, [])), ints(cu))  # in place and not
    assert o.compact([0, 2, 5], [0, 9, 5], keeps)
    same()
    tb.trellis_kv4_free(*args, ints([4, 1, 3]))
    o.free([4, 1, 3])
    same()
    tb.trellis_kv4_fork(*args, ints([0, 8]), ints([6, 4]))  # over a slot that holds pages
    assert o.fork([0, 8], [6, 4])
    same()
    tb.trellis_kv4_reserve(*args, ints([1] * 10))
    assert o.reserve(range(10), [1] * 10)
    same()
    tb.trellis_kv4_free(*args, ints(range(10)))
    o.free(range(10))
    same()
    assert (st.ref == 0).all() and tb.error_word() == 0


def test_page_operations_refuse_as_a_whole():
    log_case("pages refusals")
    T = 16
    st = Setup([20, 33, 16], T=T, spare=2, extra_slots=3, fill=False)
    random_pool(st)
    o, same = both(st)
    args = (st.cache, st.table, st.lens, st.ref)

    def refused(bit):
        same()
        assert tb.error_word() == bit
        tb.clear_error_word()

    tb.clear_error_word()
    tb.trellis_kv4_reserve(*args, ints([48, 1]), slots=ints([5, 2]))           # three and one pages: two are free
    refused(8)
    tb.trellis_kv4_fork(*args, ints([0, 1, 0]), ints([3, 4, 5]))
    refused(8)
    tb.trellis_kv4_compact(*args, ints([1]), ints([3]), ints(range(33)), ints([0, 33]))
    refused(8)
    tb.trellis_kv4_reserve(*args, ints([-1]))                                  # a negative length
    refused(4)
    tb.trellis_kv4_reserve(*args, ints([1 << 30]))                             # over the table
    refused(4)
    tb.trellis_kv4_reserve(*args, ints([1, 1]), slots=ints([2, 2]))            # a slot twice
    refused(4)
    tb.trellis_kv4_fork(*args, ints([0]), ints([6]))
    refused(4)
    tb.trellis_kv4_fork(*args, ints([-1]), ints([3]))
    refused(4)
    tb.trellis_kv4_fork(*args, ints([0, 3]), ints([3, 4]))                     # a dst that is a src
    refused(4)
    tb.trellis_kv4_fork(*args, ints([0, 1]), ints([3, 3]))
    refused(4)
    tb.trellis_kv4_compact(*args, ints([0, 0]), ints([0, 3]), ints([1, 2]), ints([0, 1, 2]))
    refused(4)
    tb.trellis_kv4_compact(*args, ints([0]), ints([3]), ints([1, 2]), ints([0, 3]))  # keep_cu past keep
    refused(4)
    tb.trellis_kv4_free(*args, ints([6, -1]))
    refused(4)
    tb.trellis_kv4_free(*args, ints([1, 1, 1]))                                # released once
    o.free([1])
    refused(0)


def test_compact_skips_bad_positions():
    log_case("compact bad positions")
    st = Setup([20], T=16, spare=4, extra_slots=1, fill=False)
    random_pool(st)
    tb.clear_error_word()
    tb.trellis_kv4_compact(st.cache, st.table, st.lens, st.ref, ints([0]), ints([1]), ints([3, 20, -1, 19]), ints([0, 4]))
    assert tb.error_word() == 4 and st.lens.tolist() == [20, 4]
    tb.clear_error_word()
    oc, table = st.oracle(), st.table.cpu().numpy()
    for u, pos in ((0, 3), (3, 19)):
        for which in (0, 1):
            a, b = oc.parts(0, table[0, pos // 16], pos % 16, which), oc.parts(0, table[1, 0], u, which)
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_many_items_and_pages():
    """More items and pages than one round of the plan takes."""
    log_case("pages many")
    n = 1500
    T = 16
    lens = [1 + (7 * i) % 20 for i in range(n)]
    st = Setup(lens, T=T, Hk=1, spare=9000, extra_slots=n, fill=False)
    random_pool(st)
    o, same = both(st)
    args = (st.cache, st.table, st.lens, st.ref)
    src, dst = list(range(n)), list(range(2 * n - 1, n - 1, -1))
    tb.trellis_kv4_fork(*args, ints(src), ints(dst))
    assert o.fork(src, dst)
    same()
    tb.trellis_kv4_reserve(*args, ints([T] * (2 * n)))
    assert o.reserve(range(2 * n), [T] * (2 * n))
    same()


# ---------------------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------------------

def test_decode_step_in_a_graph():
    """reserve, append, attention captured once and replayed: each replay is the next token, and
    the same as eager calls on a second cache."""
    log_case("kv4 graph")
    lens = [30, 64, 100]
    a = Setup(lens, T=16, Hk=2, spare=20, seed=14)
    b = Setup(lens, T=16, Hk=2, spare=20, seed=14)
    for st in (a, b):
        st.table = torch.cat((st.table, torch.full((3, 4), -1, dtype=torch.int32, device="cuda")), 1)
    x = torch.zeros((3, 12, 128), dtype=torch.float16, device="cuda")
    one, cu = ints([1, 1, 1]), ints([0, 1, 2, 3])
    y = torch.zeros((3, 8, 128), dtype=torch.float16, device="cuda")
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")

    def step(st, out, w):
        tb.trellis_kv4_reserve(st.cache, st.table, st.lens, st.ref, one, ws=w)
        tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, cu, x[:, 8:10], x[:, 10:], ws=w)
        tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, x[:, :8], window=50, sinks=4, max_q=1, out=out, ws=w)

    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step(a, y, ws)
    torch.cuda.current_stream().wait_stream(s)
    gen = torch.Generator().manual_seed(15)
    z = torch.zeros_like(y)
    w2 = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for t in range(20):
        x.copy_(torch.randn(x.shape, generator=gen).half())
        g.replay()
        torch.cuda.synchronize()
        step(b, z, w2)
        torch.cuda.synchronize()
        assert torch.equal(y, z), t
        assert torch.equal(a.cache.pool, b.cache.pool) and torch.equal(a.table, b.table) and torch.equal(a.ref, b.ref)
    assert a.lens.tolist() == [l + 20 for l in lens]
    assert tb.error_word(ws) == 0


def test_workspace_shared_with_the_products():
    """Attention's joining leaves the reserved region as it found it: a product on the same
    workspace before and after gives the same bits."""
    log_case("kv4 shared workspace")
    from trellis_coded_bit_amd import synth
    L = tb.TrellisLinear.from_host(synth.make_linear(np.random.SeedSequence(21), 3, 1024, 768))
    x = torch.randn((2, 1024)).half().cuda()
    st = Setup([9000, 300, 5000], T=64, Hk=2, seed=16)
    q = torch.randn((3, 8, 128)).half().cuda()
    cu = ints([0, 1, 2, 3])
    nb = max(tb.trellis_kv4_attn_workspace_bytes(st.cache, st.table, st.lens, cu, 3, 8),
             L.workspace_bytes(tb.TRELLIS_OP_GEMV, 2))
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    y0 = tb.trellis_gemv(L, x, ws=ws)
    a0 = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, ws=ws)
    for _ in range(3):
        assert torch.equal(tb.trellis_gemv(L, x, ws=ws), y0)
        assert torch.equal(tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, cu, q, ws=ws), a0)
    assert (ws[:256 + 65536] == 0).all()
