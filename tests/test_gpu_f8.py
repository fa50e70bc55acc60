"""The block-scaled FP8 operators on the GPU against the 64-bit oracle: the norm, the gated
activation, and products, at the sizes, types, strides and values where they can go wrong.

Tolerances, from the roundings alone (u = 2^-24, one f32 rounding):
  codes   : v / scale is formed with at most 8 roundings (h, h gamma, its largest, 448 / a, the
            product; for the activation expf's 2 u, 1 + e, the division, the product), so a code is
            one that some value within 2^-20 of the exact quotient rounds to.
  scales  : the square sum of at most 32768 channels takes at most 8 + 4 + 6 + 16 additions in a
            chain beside the squares' roundings, halved by the root; with the rest below 2^-19.
  products: a matrix instruction adds the products of eight neighbouring channels in steps of 2^-13
            of the power of two that the largest one's operands have, cutting each term off towards
            zero (measured: 256 * 256 beside 7 gives 65536, beside 14 gives 65544, wherever the two
            lie among eight channels; in different eights nothing is lost up to 2^-23).  That power
            is at most the largest product, so eight channels lose less than 7 * 2^-13 of it.  The
            sixteen sums of eight, the blocks (one fma each), the shares of split sums and the
            factor take (16 + blocks + 32) roundings of at most 2 u sum |terms|.  The result is
            rounded to its type.  Over a whole result the cuts are independent of the rounding and
            far below it, and its relative 2-norm stays within half a step.
"""
import numpy as np
import pytest
import torch

from oracle import f8 as FO
from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the smallest numbers
U = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_rounded(got, ref, dtype, rel=0.0, extra=0.0):
    """Within half a step of `dtype` beside a relative and an absolute error before it."""
    err = np.abs(got - ref)
    bound = np.abs(ref) * (HALF[dtype] * (1 + rel) + rel) + extra * (1 + HALF[dtype]) + TINY[dtype]
    assert (err <= bound).all(), float((err / bound).max())


def check_quantized(q, s, v, rel_code, rel_scale):
    """Codes' values and scales of rows v (64 bits)."""
    rq, rs = FO.quantize(v)
    nan = np.isnan(rs)
    assert np.array_equal(np.isnan(s), nan)
    assert (np.abs(s - rs)[~nan] <= rel_scale * rs[~nan]).all()
    # the quotient from the exact scale: the scale's own error does not reach the codes
    full = np.repeat(FO.block_top(v) / 448.0, 128, 1)[:, :v.shape[1]]
    zero = np.repeat(nan | (rs == 0), 128, 1)[:, :v.shape[1]]
    with np.errstate(all="ignore"):
        t = np.where(zero, 0.0, v / full)
    a, b = FO.e4m3_round(t * (1 - rel_code)), FO.e4m3_round(t * (1 + rel_code))
    ok = (q >= np.minimum(a, b)) & (q <= np.maximum(a, b))
    assert ok.all(), (int((~ok).sum()), q[~ok][:4], t[~ok][:4])
    assert (q != rq).mean() < 1e-3
    return rq, rs


# ---------------------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,n,residual,gamma,stride", [
    (1, 16, False, True, 0), (1, 5120, True, True, 0), (3, 128, True, False, 8), (5, 144, True, True, 0),
    (7, 2032, False, True, 24), (33, 1024, True, True, 0), (2, 8192, True, True, 0), (3, 8208, True, True, 0),
    (2, 17408, True, True, 0), (2, 32768, True, True, 0), (700, 6144, True, True, 0), (4100, 256, False, False, 0),
])
def test_norm(dtype, rows, n, residual, gamma, stride):
    log_case(f"f8 norm {dtype} rows={rows} n={n} residual={residual} gamma={gamma} stride=+{stride}")
    g = torch.Generator().manual_seed(rows * 7 + n)
    x = torch.randn((rows, n + stride), generator=g)
    x[:, ::37] *= 9
    x = x.to(DT[dtype]).cuda()[:, :n]
    res = (3 * torch.randn((rows, n), generator=g)).to(DT[dtype]).cuda() if residual else None
    gam = (1 + 0.3 * torch.randn((n,), generator=g)).to(DT[dtype]).cuda() if gamma else None
    y = torch.empty((rows, n), dtype=DT[dtype], device="cuda")
    q, s, h = tb.trellis_f8_norm(x, gam, 1e-5, residual=res, y=y)
    v, rh = FO.norm(host(x), float(np.float32(1e-5)), host(gam) if gamma else None, host(res) if residual else None)
    assert q.dtype == torch.float8_e4m3fn and s.shape == (rows, -(-n // 128))
    check_quantized(host(q), host(s), v, 2.0 ** -20, 2.0 ** -19)
    check_rounded(host(y), v, dtype, 2.0 ** -19)
    if residual:
        check_rounded(host(h), rh, dtype, U)
    else:
        assert h is None
    # the norm alone, and the residual in place, give the same bits
    y2, h2 = tb.trellis_f8_norm(x, gam, 1e-5, residual=res, quantize=False)
    assert torch.equal(y, y2)
    if residual:
        assert torch.equal(h, h2)
        r2 = res.clone()
        q3, s3, h3 = tb.trellis_f8_norm(x, gam, 1e-5, residual=r2, h=r2)
        assert h3 is r2 and torch.equal(r2, h) and torch.equal(q3.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s3, s)


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_norm_of_special_rows(dtype, rows):
    """Zeros, one channel alone, the type's largest, numbers whose squares leave f32, NaN and
    infinities: rows beside them are not touched."""
    log_case(f"f8 norm special {dtype} rows={rows}")
    n = 400
    g = torch.Generator().manual_seed(3)
    kinds = [torch.randn(n, generator=g), torch.zeros(n), torch.zeros(n), torch.full((n,), torch.finfo(DT[dtype]).max),
             torch.randn(n, generator=g), torch.randn(n, generator=g), torch.randn(n, generator=g) * 1e-6]
    kinds[2][131] = 5.0
    kinds[4][200] = float("nan")
    kinds[5][399] = float("-inf")
    if dtype == "bf16":
        kinds += [torch.randn(n, generator=g) * 1e30, torch.randn(n, generator=g) * 1e-30]
    x = torch.stack(kinds).repeat(rows, 1)
    gam = 1 + 0.3 * torch.randn(n, generator=g)
    gam[300:310] = 0
    x, gam = x.to(DT[dtype]).cuda(), gam.to(DT[dtype]).cuda()
    y = torch.empty_like(x)
    q, s, _ = tb.trellis_f8_norm(x, gam, 1e-12, y=y)
    v, _ = FO.norm(host(x), float(np.float32(1e-12)), host(gam))
    q, s, y = host(q), host(s), host(y)
    assert np.isnan(s).any() and (s[1] == 0).all() and s[2, 1] > 0 and s[2, 0] == 0
    nan = np.isnan(v)
    assert np.array_equal(np.isnan(y), nan)
    assert not np.isnan(s[0]).any() and np.isnan(s[4]).all() and np.isnan(s[5]).tolist() == [False, False, False, True]
    check_quantized(np.where(nan, 0, q), s, v, 2.0 ** -20, 2.0 ** -19)
    check_rounded(np.where(nan, 0, y), np.where(nan, 0, v), dtype, 2.0 ** -19)
    assert (q[np.repeat(np.isnan(s), 128, 1)[:, :n]] == 0).all()


# ---------------------------------------------------------------------------------------
# Gated activation
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,n,stride", [(1, 16, 0), (1, 2048, 0), (5, 144, 8), (264, 2048, 0), (3, 17408, 0), (1000, 112, 32)])
def test_silu_mul(dtype, rows, n, stride):
    log_case(f"f8 silu_mul {dtype} rows={rows} n={n} stride=+{stride}")
    g = torch.Generator().manual_seed(rows + n)
    x = (2 * torch.randn((rows, 2 * n + stride), generator=g)).to(DT[dtype]).cuda()[:, :2 * n]
    y = torch.empty((rows, n), dtype=DT[dtype], device="cuda")
    q, s = tb.trellis_f8_silu_mul(x, y=y)
    v = FO.silu_mul(host(x))
    check_quantized(host(q), host(s), v, 2.0 ** -20, 2.0 ** -20)
    check_rounded(host(y), v, dtype, 2.0 ** -20)
    assert torch.equal(tb.trellis_f8_silu_mul(x, quantize=False), y)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_silu_mul_of_special_values(dtype):
    log_case(f"f8 silu_mul special {dtype}")
    big = torch.finfo(DT[dtype]).max
    x = torch.zeros((4, 2 * 256))
    x[0, :256] = torch.linspace(-80, 80, 256)
    x[0, 256:] = 1.0
    x[1, 3], x[1, 256 + 3] = float("nan"), 1.0
    x[1, 200], x[1, 256 + 200] = 2.0, 3.0
    x[2, 0], x[2, 256] = big, 1.0
    x[2, 128], x[2, 256 + 128] = -big, big      # silu is 0 from below, times the largest
    x[3, 7], x[3, 256 + 7] = float("inf"), 2.0
    x = x.to(DT[dtype]).cuda()
    q, s = tb.trellis_f8_silu_mul(x)
    v = FO.silu_mul(host(x))
    q, s = host(q), host(s)
    assert np.isnan(s).tolist() == [[False, False], [True, False], [False, False], [True, False]]
    assert s[2, 1] == 0 and (q[2, 128:] == 0).all() and (q[1, :128] == 0).all() and (q[3, :128] == 0).all()
    check_quantized(q[:1], s[:1], v[:1], 2.0 ** -20, 2.0 ** -20)
    assert abs(s[2, 0] * 448 / v[2, 0] - 1) < 2.0 ** -20 and abs(s[1, 1] * 448 / v[1, 200] - 1) < 2.0 ** -20


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_silu_mul_of_far_gates(dtype):
    """Gates whose sigmoid is below f32's normal numbers, times numbers that are not small: a row is one
    block of gates within 1 of each other.  Every result and scale that 16 bits and f32 hold is there."""
    log_case(f"f8 silu_mul far gates {dtype}")
    g = torch.Generator().manual_seed(11)
    top = torch.arange(-60.0, -192.0, -0.75)[:, None]
    gates = top - torch.rand((len(top), 128), generator=g)
    big = torch.finfo(DT[dtype]).max
    for size in (big, big ** 0.75, 1.0):
        u = (torch.rand((len(top), 128), generator=g) - 0.5) * 2 * size
        u[:, 5] = size
        x = torch.cat((gates, u), 1).to(DT[dtype]).cuda()
        y = torch.empty((len(top), 128), dtype=DT[dtype], device="cuda")
        q, s = tb.trellis_f8_silu_mul(x, y=y)
        v = FO.silu_mul(host(x))
        _, rs = FO.quantize(v)
        assert dtype == "fp16" or size < big or (rs > 0).sum() > 80
        check_quantized(host(q), host(s), v, 2.0 ** -20, 2.0 ** -20)
        check_rounded(host(y), v, dtype, 2.0 ** -20)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_silu_mul_of_far_gates_and_special_values(dtype):
    log_case(f"f8 silu_mul far gates, special {dtype}")
    inf, nan = float("inf"), float("nan")
    gates = torch.tensor([-79.5, -80.5, -100, -186, -190, -300, -6e4, -inf, -100, nan, -100, -300, -85, 3.0, -inf, -100])
    ups = torch.tensor([inf, inf, inf, -inf, inf, -inf, inf, 1.0, nan, 1.0, 0.0, 0.0, 1.0, 2.0, 0.0, -6e4])
    x = torch.cat((gates.repeat_interleave(128), ups.repeat_interleave(128)))[None].to(DT[dtype]).cuda()
    y = torch.empty((1, 16 * 128), dtype=DT[dtype], device="cuda")
    q, s = tb.trellis_f8_silu_mul(x, y=y)
    y, q, s = host(y).reshape(16, 128), host(q).reshape(16, 128), host(s)[0]
    want = [-inf, -inf, -inf, inf, -inf, inf, -inf, nan, nan, nan, 0, 0, None, None, nan, None]
    for i, w in enumerate(want):
        if w is not None:
            assert (np.isnan(y[i]) if w is nan else y[i] == w).all(), (i, y[i, 0])
            assert (np.isnan(s[i]) if w else s[i] == 0) and (q[i] == 0).all(), (i, s[i])
    v = FO.silu_mul(host(x)).reshape(16, 128)
    live = [12, 13, 15]
    check_rounded(y[live], v[live], dtype, 2.0 ** -20)
    check_quantized(q[live], s[live, None], v[live], 2.0 ** -20, 2.0 ** -20)


def test_values_above_f32_are_infinite():
    """Their blocks stand for NaN; the blocks beside them are as they are."""
    log_case("f8 values above f32")
    x = torch.zeros((2, 512))
    x[:, :256], x[:, 256:] = 1e30, 1.0
    x[0, 256:384], x[1, 256:384] = 1e30, -1e30
    x = x.bfloat16().cuda()
    y = torch.empty((2, 256), dtype=torch.bfloat16, device="cuda")
    q, s = tb.trellis_f8_silu_mul(x, y=y)
    inf = float("inf")
    assert (y[0, :128] == inf).all() and (y[1, :128] == -inf).all() and torch.equal(y[:, 128:], x[:, :128])
    assert torch.isnan(s[:, 0]).all() and (host(q)[:, :128] == 0).all() and torch.isfinite(s[:, 1]).all()
    g = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    g[:128] = torch.finfo(torch.bfloat16).max
    x = torch.zeros((1, 256), dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[0, 200] = 4.0, 1.0  # 4 / sqrt(17 / 256) times the largest number
    y = torch.empty_like(x)
    q, s, _ = tb.trellis_f8_norm(x, g, 1e-6, y=y)
    assert y[0, 5] == inf and torch.isnan(s[0, 0]) and (host(q)[0, :128] == 0).all()
    v, _ = FO.norm(host(x), float(np.float32(1e-6)), host(g))
    check_rounded(host(y)[:, 128:], v[:, 128:], "bf16", 2.0 ** -19)
    check_quantized(host(q)[:, 128:], host(s)[:, 1:], v[:, 128:], 2.0 ** -20, 2.0 ** -19)


# ---------------------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------------------

def codes(shape, g, spread=1.0):
    return (spread * 60 * torch.randn(shape, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)


def make_matrix(n, k, g, experts=None, gain=1.0):
    lead = () if experts is None else (experts,)
    s = gain * torch.exp(torch.randn((*lead, -(-n // 128), -(-k // 128)), generator=g)) / (60 * 60 * k ** 0.5)
    return tb.F8Linear(codes((*lead, n, k), g).cuda(), s.cuda())


def make_rows(m, k, g, q_stride=0, s_stride=0):
    kb = -(-k // 128)
    q = codes((m, k + q_stride), g).cuda()[:, :k]
    s = torch.exp(torch.randn((m, kb + s_stride), generator=g)).cuda()[:, :kb]
    return q, s


def largest_of_eights(q, s, w, sw):
    """Sum over the eights of neighbouring channels of their largest product's magnitude."""
    pad = lambda t: torch.nn.functional.pad(t.float().abs(), (0, -t.shape[1] % 8)).unflatten(1, (-1, 8))  # noqa: E731
    x, m, cols = pad(q), pad(w), torch.arange(w.shape[0], device=w.device) // 128
    total = torch.zeros((q.shape[0], w.shape[0]), device="cuda")
    for i in range(x.shape[1]):
        top = (x[:, None, i] * m[None, :, i]).amax(-1)
        total += top * s[:, None, i // 16] * sw[cols, i // 16]
    return host(total)


def check_product(y, q, s, w, sw, dtype):
    ref, mass = FO.product(host(q), host(s), host(w), host(sw))
    kb = s.shape[1]
    extra = 7 * 2.0 ** -13 * (1 + 2.0 ** -10) * largest_of_eights(q, s, w, sw) + 2 * (16 + kb + 32) * U * mass
    check_rounded(host(y), ref, dtype, 0.0, extra)
    # (results below the type's smallest normal number are rounded to its absolute step)
    assert np.linalg.norm(host(y) - ref) <= HALF[dtype] * np.linalg.norm(ref) + TINY[dtype] * ref.size ** 0.5


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 16, 128), (1, 130, 144), (1, 5120, 6144), (1, 1000, 17408), (2, 257, 272), (3, 640, 2048), (8, 129, 1040),
    (15, 512, 512), (16, 136, 640), (17, 1000, 400), (31, 384, 1024), (33, 264, 2048), (64, 2048, 1024), (65, 300, 784),
    (100, 1032, 1296), (127, 128, 128), (128, 640, 128), (129, 257, 16), (200, 1288, 2064), (255, 768, 640), (256, 1024, 1152),
    (257, 513, 1024), (300, 256, 4096), (513, 2050, 528), (1000, 264, 272), (2048, 384, 512),
    # eights of tokens in odd numbers; blocks shared among workgroups
    (9, 48, 144), (18, 264, 640), (24, 300, 1040), (37, 520, 400), (40, 136, 2048), (50, 257, 656), (56, 640, 272),
    (70, 4104, 6160), (130, 1544, 16400), (70, 2050, 16400), (300, 1032, 4112),
])
def test_gemm(dtype, m, n, k):
    log_case(f"f8 gemm {dtype} m={m} n={n} k={k}")
    g = torch.Generator().manual_seed(m * 131 + n * 7 + k)
    L = make_matrix(n, k, g)
    q, s = make_rows(m, k, g)
    out = torch.full((m, n), 7.0, dtype=DT[dtype], device="cuda")
    y = tb.trellis_f8_gemm(L, q, s, out=out)
    assert y is out
    check_product(y, q, s, L.w, L.scale, dtype)
    # again, into a new tensor: the same bits, whatever shares the sums
    assert torch.equal(tb.trellis_f8_gemm(L, q, s, dtype=DT[dtype]), y)
    assert tb.error_word() == 0


@pytest.mark.parametrize("m", [1, 5, 40, 200])
def test_gemm_of_slices(m):
    """Rows of q, scales and results inside wider buffers; what is between them stays."""
    log_case(f"f8 gemm slices m={m}")
    g = torch.Generator().manual_seed(m)
    n, k = 392, 656
    L = make_matrix(n, k, g)
    q, s = make_rows(m, k, g, 48, 3)
    for width, first in ((n + 8, 0), (n + 13, 5), (n + 16, 8)):
        wide = torch.full((m, width), 3.0, dtype=torch.float16, device="cuda")
        y = wide[:, first:first + n]
        tb.trellis_f8_gemm(L, q, s, out=y)
        check_product(y, q, s, L.w, L.scale, "fp16")
        wide[:, first:first + n] = 3.0
        assert (wide == 3.0).all()
        assert torch.equal(tb.trellis_f8_gemm(L, q.contiguous(), s.contiguous()), tb.trellis_f8_gemm(L, q, s))


@pytest.mark.parametrize("m", [1, 20, 150])
def test_gemm_of_special_values(m):
    """A NaN code or scale reaches its row's or its columns' results and no others; zeros of rows
    behind the last and channels behind the last block's end are no part of the sums."""
    log_case(f"f8 gemm special m={m}")
    g = torch.Generator().manual_seed(m)
    n, k = 300, 400
    L = make_matrix(n, k, g)
    wide = torch.full((m + 4, 512), float("nan")).to(torch.float8_e4m3fn).cuda()  # what lies around q
    scales = torch.full((m + 4, 8), float("nan"), device="cuda")
    q, s = wide[:m, :k], scales[:m, :4]
    q0, s0 = make_rows(m, k, g)
    q.copy_(q0)
    s.copy_(s0)
    y = tb.trellis_f8_gemm(L, q, s)
    check_product(y, q0, s0, L.w, L.scale, "fp16")
    q.view(torch.uint8)[m - 1, 399] = 0x7F
    w = L.w.clone()
    w.view(torch.uint8)[299, 0] = 0xFF
    sw = L.scale.clone()
    sw[1, 2] = float("inf")
    z = tb.trellis_f8_gemm(tb.F8Linear(w, sw), q, s)
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    bad[m - 1], bad[:, 299], bad[:, 128:256] = True, True, True
    assert torch.isfinite(z[~bad]).all() and torch.equal(z[~bad], y[~bad])
    assert torch.isnan(z[m - 1]).all() and torch.isnan(z[:, 299]).all() and not torch.isfinite(z[:, 128:256]).any()


@pytest.mark.parametrize("m,n,k", [(70, 4099, 6160), (200, 2051, 8208)])
def test_gemm_of_shared_blocks(m, n, k):
    """Sums joined from several workgroups: into a slice, of rows inside wider ones, with infinities
    and NaN, by two graphs that share a workspace with each other and with eager calls."""
    log_case(f"f8 gemm shared blocks m={m} n={n} k={k}")
    g = torch.Generator().manual_seed(m)
    L = make_matrix(n, k, g)
    q, s = make_rows(m, k, g, 48, 3)
    ws = torch.zeros(tb.trellis_f8_workspace_bytes(L, m), dtype=torch.uint8, device="cuda")
    assert ws.numel() > tb.trellis_f8_workspace_bytes(L, 1)
    wide = torch.full((m, n + 9), 3.0, dtype=torch.float16, device="cuda")
    y = wide[:, 5:5 + n]
    tb.trellis_f8_gemm(L, q, s, out=y, ws=ws)
    check_product(y, q, s, L.w, L.scale, "fp16")
    want = y.clone()
    y.fill_(3.0)
    assert (wide == 3.0).all()
    outs, graphs = [torch.empty((m, n), dtype=torch.float16, device="cuda") for _ in range(2)], []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tb.trellis_f8_gemm(L, q, s, out=o, ws=ws)
    for _ in range(3):
        for o, graph in zip(outs, graphs):
            o.fill_(9.0)
            graph.replay()
        tb.trellis_f8_gemm(L, q, s, out=y, ws=ws)
        assert all(torch.equal(o, want) for o in outs) and torch.equal(y, want)
    s[m - 1, k // 256] = float("nan")
    w = L.w.clone()
    w.view(torch.uint8)[n - 1, k - 1] = 0x7F
    z = tb.trellis_f8_gemm(tb.F8Linear(w, L.scale), q, s, ws=ws)
    assert torch.isnan(z[m - 1]).all() and torch.isnan(z[:, n - 1]).all() and torch.equal(z[:-1, :-1], want[:-1, :-1])
    assert tb.error_word(ws) == 0


def scaled_far(m, n, k, g):
    """Rows, a matrix and scales whose products leave f32: rows of zeros (0, 4, ..), of one smallest code
    where the product is 1e39 (1, 5, ..), of ordinary codes that stay off those blocks (2, 6, ..), of
    codes that carry the result out of every type (3, 7, ..)."""
    q, s = make_rows(m, k, g)
    L = make_matrix(n, k, g)
    w, sw, block = L.w, L.scale, slice(128, min(k, 256))
    q = q.float()
    s[:, 1] = 1e20
    sw[:, 1] = 1e19
    for kind in (0, 1, 2):
        q[kind::4, block] = 0
    q[0::4] = 0
    q[1::4] = 0
    q[1::4, 130] = 2.0 ** -9
    q[3::4, block] = 300
    w.view(torch.uint8)[:, 130] = torch.arange(n, device="cuda", dtype=torch.int64).remainder(7).to(torch.uint8)  # 0 .. 7 * 2^-9
    w.view(torch.uint8)[:, 131] = 0x70  # (128: the rows of 300 overflow)
    return L, q.to(torch.float8_e4m3fn), s


def check_far(y, q, s, w, sw, dtype):
    """A block's sum is off by up to 7 * 2^-13 of the eights' largest products (see above), whatever its
    scales: where these carry that much out of the type, a sum that nearly cancels may leave the type on
    either side, and only sums that are further from zero say on which."""
    ref, _ = FO.product(host(q), host(s), host(w), host(sw))
    y, kb, big = host(y), s.shape[1], torch.finfo(DT[dtype]).max
    eights = 2.0 ** 80 * largest_of_eights(q, s * 2.0 ** -40, w, sw * 2.0 ** -40)  # (within f32)
    extra = 7 * 2.0 ** -13 * (1 + 2.0 ** -10) * eights + 2 * (16 + kb + 32) * U * np.abs(ref)
    over, within = np.abs(ref) - extra > 1.01 * big, np.abs(ref) + extra < big
    assert over.any() and (y[over] == np.copysign(np.inf, ref[over])).all()
    assert over[3::4].mean() > 0.5 and within[0::4].all() and within[2::4].all() and (dtype == "fp16" or within[1::4].all())
    check_rounded(np.where(within, y, 0.0), np.where(within, ref, 0.0), dtype, 0.0, np.where(within, extra, 0.0))
    assert (y[0::4] == 0).all() and np.isfinite(y[2::4]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 256), (4, 300, 272), (37, 257, 400), (64, 160, 1040), (100, 1032, 1296), (300, 513, 400), (300, 1032, 4112),
                                   (1000, 300, 272)])
def test_gemm_of_scales_whose_product_leaves_f32(dtype, m, n, k):
    log_case(f"f8 gemm far scales {dtype} m={m} n={n} k={k}")
    L, q, s = scaled_far(max(m, 4), n, k, torch.Generator().manual_seed(m + n))
    y = tb.trellis_f8_gemm(L, q, s, dtype=DT[dtype])
    check_far(y, q, s, L.w, L.scale, dtype)
    if m == 1:  # a row of zeros alone, and the one of one code
        assert (tb.trellis_f8_gemm(L, q[:1], s[:1], dtype=DT[dtype]) == 0).all()
        assert torch.equal(tb.trellis_f8_gemm(L, q[1:2], s[1:2], dtype=DT[dtype]), y[1:2])
    # results that need no second look have the bits that they have without one
    s2 = s.clone()
    s2[:, 1] = 1.0
    z = tb.trellis_f8_gemm(tb.F8Linear(L.w, torch.ones_like(L.scale).where(torch.arange(L.scale.shape[1], device="cuda") == 1, L.scale)), q, s2,
                           dtype=DT[dtype])
    assert torch.equal(z[2::4], y[2::4])


@pytest.mark.parametrize("each", [3, 40, 170])
def test_moe_gemm_of_scales_whose_product_leaves_f32(each):
    log_case(f"f8 moe_gemm far scales each={each}")
    g = torch.Generator().manual_seed(each)
    n, k = 264, 400
    parts = [scaled_far(4 * each, n, k, g) for _ in range(3)]
    E = tb.F8Linear(torch.stack([p[0].w.view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn), torch.stack([p[0].scale for p in parts]))
    q, s = torch.cat([p[1].view(torch.uint8) for p in parts]), torch.cat([p[2] for p in parts])
    back = torch.randperm(len(q), generator=g).cuda()  # the rows of q in another order
    at = torch.empty_like(back)
    at[back] = torch.arange(len(q), device="cuda")
    off = ints([0, 4 * each, 8 * each, 12 * each])
    y = tb.trellis_f8_moe_gemm(E, q[back].view(torch.float8_e4m3fn), s[back], off, order=at.int(), per=1, dtype=torch.bfloat16)
    for e, (L, qe, se) in enumerate(parts):
        check_far(y[4 * each * e:4 * each * (e + 1)], qe, se, L.w, L.scale, "bf16")


@pytest.mark.parametrize("m", [4, 300])
def test_gemm_of_scales_whose_product_is_hardly_normal(m):
    """Below the smallest normal number the product of two scales has steps of 2^-149: half of one, times
    a block's sum of at most 128 * 448^2, is less than 2^-125."""
    log_case(f"f8 gemm small scales m={m}")
    g = torch.Generator().manual_seed(m)
    n, k = 300, 656
    L = make_matrix(n, k, g)
    q, s = make_rows(m, k, g)
    for a, b in ((-60.0, -66.0), (-60.0, -80.0), (-110.0, -20.0), (-126.0, -10.0), (0.0, -126.0)):
        sx, sw = torch.full_like(s, 2.0 ** a) * (1 + torch.rand(s.shape, generator=g).cuda()), torch.full_like(L.scale, 2.0 ** b) * 1.5
        y = tb.trellis_f8_gemm(tb.F8Linear(L.w, sw), q, sx, dtype=torch.bfloat16)
        ref, mass = FO.product(host(q), host(sx), host(L.w), host(sw))
        eights = 2.0 ** -100 * largest_of_eights(q, sx * 2.0 ** 50, L.w, sw * 2.0 ** 50)
        extra = 7 * 2.0 ** -13 * (1 + 2.0 ** -10) * eights + 2 * (16 + 6 + 32) * U * mass
        check_rounded(host(y), ref, "bf16", 0.0, extra + 6 * 2.0 ** -125)
        assert (host(y) != 0).mean() > 0.9


def test_gemm_overflow_is_infinite():
    log_case("f8 gemm overflow")
    L = tb.F8Linear(torch.full((16, 128), 448.0).to(torch.float8_e4m3fn).cuda(), torch.ones((1, 1), device="cuda"))
    q = torch.full((3, 128), 448.0).to(torch.float8_e4m3fn).cuda()
    q[1] = -q[1].float()
    q[2] = 0
    y = tb.trellis_f8_gemm(L, q, torch.ones((3, 1), device="cuda"))
    assert (y[0] == float("inf")).all() and (y[1] == float("-inf")).all() and (y[2] == 0).all()
    y = tb.trellis_f8_gemm(L, q, torch.ones((3, 1), device="cuda"), dtype=torch.bfloat16)
    assert torch.isfinite(y).all()


def grouped(counts, n, k, g, per=0, tokens=0):
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    L = make_matrix(n, k, g, E)
    total = int(off[-1])
    if per:
        order = torch.randperm(tokens * per, generator=g)[:total].to(torch.int32)
        q, s = make_rows(tokens, k, g)
        src = order.long() // per
    else:
        order, src = None, torch.arange(total)
        q, s = make_rows(total, k, g)
    return L, q, s, ints(off.tolist()), order, src


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("counts,n,k,per", [
    ([1], 128, 128, 0), ([0, 0, 3, 0], 136, 144, 0), ([5, 0, 1, 17, 16, 0, 33, 2], 264, 272, 4),
    ([130, 1, 0, 257, 128, 64], 392, 656, 2), ([1] * 70 + [0] * 30 + [2] * 30, 160, 384, 8), ([300, 700], 512, 1024, 0),
    ([0] * 199 + [40], 128, 256, 8), ([2, 3, 1, 2, 0, 4, 2, 2], 1024, 2048, 8),
    ([20, 40, 0, 7], 264, 400, 2), ([60, 1, 30], 136, 640, 0), ([1] * 300, 32, 144, 4),
])
def test_moe_gemm(dtype, counts, n, k, per):
    log_case(f"f8 moe_gemm {dtype} experts={len(counts)} rows={sum(counts)} n={n} k={k} per={per}")
    g = torch.Generator().manual_seed(sum(counts) + n)
    total = sum(counts)
    tokens = -(-total // per) + 3 if per else 0
    L, q, s, off, order, src = grouped(counts, n, k, g, per, tokens)
    extra = 5  # rows behind the last expert's
    if per:
        full = torch.full((total + extra,), -1, dtype=torch.int32)
        full[:total] = order
        order = full.cuda()
    else:
        q, s = torch.cat((q, q[:1].expand(extra, -1).clone())), torch.cat((s, s[:1].expand(extra, -1)))
    out = torch.full((total + extra, n), 5.0, dtype=DT[dtype], device="cuda")
    y = tb.trellis_f8_moe_gemm(L, q, s, off, order=order, per=max(per, 1), out=out)
    assert (y[total:] == 5.0).all()
    src, o = src.cuda(), off.tolist()
    for e in range(len(counts)):
        if counts[e]:
            at = src[o[e]:o[e + 1]]
            check_product(y[o[e]:o[e + 1]], q.view(torch.uint8)[at].view(torch.float8_e4m3fn), s[at], L.w[e], L.scale[e], dtype)
    again = torch.full_like(out, 5.0)
    assert torch.equal(tb.trellis_f8_moe_gemm(L, q, s, off, order=order, per=max(per, 1), out=again), y)
    assert tb.error_word() == 0


def test_moe_gemm_without_rows():
    log_case("f8 moe_gemm no rows")
    g = torch.Generator().manual_seed(0)
    L = make_matrix(128, 128, g, 3)
    q, s = make_rows(6, 128, g)
    out = torch.full((6, 128), 5.0, dtype=torch.float16, device="cuda")
    tb.trellis_f8_moe_gemm(L, q, s, ints([0, 0, 0, 0]), out=out)
    assert (out == 5.0).all() and tb.error_word() == 0
    assert tb.trellis_f8_moe_gemm(L, q[:0], s[:0], ints([0, 0, 0, 0])).shape == (0, 128)
    assert tb.trellis_f8_gemm(make_matrix(128, 128, g), q[:0], s[:0]).shape == (0, 128)


@pytest.mark.parametrize("offsets,done", [([0, 4, 2, 9], 4), ([0, 4, 8, 99], 8), ([1, 4, 8, 9], 0), ([0, -3, 8, 9], 0), ([0, 4, 8, 9], 9)])
def test_moe_gemm_bad_offsets(offsets, done):
    """The call ends at the first pair that is out of order: rows before it are right, the rest left."""
    log_case(f"f8 moe_gemm offsets={offsets}")
    g = torch.Generator().manual_seed(1)
    L = make_matrix(128, 256, g, 3)
    q, s = make_rows(12, 256, g)
    good = torch.zeros((12, 128), dtype=torch.float16, device="cuda")
    tb.trellis_f8_moe_gemm(L, q, s, ints([0, 4, 8, 9]), out=good)
    out = torch.full((12, 128), 5.0, dtype=torch.float16, device="cuda")
    tb.clear_error_word()
    tb.trellis_f8_moe_gemm(L, q, s, ints(offsets), out=out)
    assert torch.equal(out[:done], good[:done]) and (out[done:] == 5.0).all()
    assert tb.error_word() == (0 if done == 9 else 1)
    tb.clear_error_word()


@pytest.mark.parametrize("rows,offsets,done", [(1, [0, 1, 5], 1), (1, [0, 1, 0], 1), (40, [0, 20, 40, 41], 40), (200, [0, 100, 200, 100], 200)])
def test_moe_gemm_bad_offsets_behind_the_last_row(rows, offsets, done):
    """They are found also where every row has its expert before them."""
    log_case(f"f8 moe_gemm rows={rows} offsets={offsets}")
    g = torch.Generator().manual_seed(1)
    L = make_matrix(128, 256, g, len(offsets) - 1)
    q, s = make_rows(rows, 256, g)
    good = tb.trellis_f8_moe_gemm(L, q, s, ints(offsets[:-1] + [rows]))
    tb.clear_error_word()
    assert torch.equal(tb.trellis_f8_moe_gemm(L, q, s, ints(offsets))[:done], good[:done]) and tb.error_word() == 1
    tb.clear_error_word()


@pytest.mark.parametrize("rows", [9, 140])
def test_moe_gemm_bad_order(rows):
    log_case(f"f8 moe_gemm bad order rows={rows}")
    g = torch.Generator().manual_seed(2)
    L = make_matrix(136, 144, g, 2)
    q, s = make_rows(10, 144, g)
    order = torch.arange(rows, dtype=torch.int32, device="cuda") % 20
    good = tb.trellis_f8_moe_gemm(L, q, s, ints([0, 3, rows]), order=order, per=2)
    for at, v in ((1, -1), (4, 20), (6, 2 ** 31 - 1), (rows - 1, -(2 ** 31))):
        order[at] = v
        good[at] = 0
    tb.clear_error_word()
    assert torch.equal(tb.trellis_f8_moe_gemm(L, q, s, ints([0, 3, rows]), order=order, per=2), good)
    assert tb.error_word() == 1
    tb.clear_error_word()


def test_refusals():
    log_case("f8 refusals")
    g = torch.Generator().manual_seed(0)
    L, E = make_matrix(128, 128, g), make_matrix(128, 128, g, 2)
    q, s = make_rows(4, 128, g)
    x = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    off = ints([0, 2, 4])
    for error, f in (
            (ValueError, lambda: tb.trellis_f8_gemm(E, q, s)), (ValueError, lambda: tb.trellis_f8_moe_gemm(L, q, s, off)),
            (ValueError, lambda: tb.trellis_f8_gemm(L, q[:, :112], s)), (ValueError, lambda: tb.trellis_f8_gemm(L, q, s[:3])),
            (TypeError, lambda: tb.trellis_f8_gemm(L, q.view(torch.uint8), s)), (TypeError, lambda: tb.trellis_f8_gemm(L, q, s, dtype=torch.float32)),
            (ValueError, lambda: tb.trellis_f8_gemm(L, q, s, out=x)), (ValueError, lambda: tb.trellis_f8_moe_gemm(E, q, s, off[:2])),
            (TypeError, lambda: tb.trellis_f8_moe_gemm(E, q, s, off.long())), (tb.TrellisError, lambda: tb.trellis_f8_moe_gemm(E, q, s, off, per=0)),
            (ValueError, lambda: tb.F8Linear(L.w, L.scale[:, :0])), (TypeError, lambda: tb.F8Linear(x, L.scale)),
            (tb.TrellisError, lambda: tb.trellis_f8_norm(x[:, :200], None, 1e-6)), (tb.TrellisError, lambda: tb.trellis_f8_norm(x, None, 0.0)),
            (tb.TrellisError, lambda: tb.trellis_f8_norm(x[:, 1:241], None, 1e-6)), (ValueError, lambda: tb.trellis_f8_norm(x.t(), None, 1e-6)),
            (TypeError, lambda: tb.trellis_f8_norm(x, x[0].float(), 1e-6)), (ValueError, lambda: tb.trellis_f8_norm(x, x[0, :128].contiguous(), 1e-6)),
            (tb.TrellisError, lambda: tb.trellis_f8_norm(x, None, 1e-6, y=x)), (ValueError, lambda: tb.trellis_f8_norm(x, None, 1e-6, quantize=False, q=q)),
            (ValueError, lambda: tb.trellis_f8_silu_mul(x[:, :255])), (tb.TrellisError, lambda: tb.trellis_f8_silu_mul(x[:, :48]))):
        with pytest.raises(error):
            f()


def test_sizes_above_32_bits_are_refused():
    """Not cut off to the small sizes that their lower 32 bits are."""
    log_case("f8 sizes above 32 bits")
    g = torch.Generator().manual_seed(0)
    L, E = make_matrix(128, 128, g), make_matrix(128, 128, g, 2)
    q, s = make_rows(4, 128, g)
    many = 2 ** 32 + 4
    x = torch.zeros((1, 32), dtype=torch.float16, device="cuda").expand(many, 32)
    ids = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    for f in (lambda: tb.trellis_f8_norm(x, None, 1e-6), lambda: tb.trellis_f8_silu_mul(x), lambda: tb.trellis_moe_sort(ids, many),
              lambda: tb.trellis_f8_gemm(L, q[:1].expand(many, 128), s[:1].expand(many, 1)),
              lambda: tb.trellis_f8_moe_gemm(E, q, s, ints([0, 2, 4]), order=ints([0, 1, 2, 3]), per=2 ** 32 + 1),
              lambda: tb.trellis_moe_gather(x, ints([0, 1]), 1), lambda: tb.trellis_moe_gather(q, ints([0, 1]), 2 ** 32 + 1)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("m", [1, 48, 300])
def test_gemm_in_a_graph_and_on_streams(m):
    """Captured with a workspace of its own and replayed with other inputs, beside eager calls on
    two streams with theirs."""
    log_case(f"f8 gemm graph m={m}")
    g = torch.Generator().manual_seed(m)
    n, k = 640, 4096
    L, E = make_matrix(n, k, g), make_matrix(n, k, g, 3)
    q, s = make_rows(m, k, g)
    off = ints([0, m // 3, m // 3, m])
    ws = torch.zeros(max(tb.trellis_f8_workspace_bytes(L, m), tb.trellis_f8_workspace_bytes(E, m)), dtype=torch.uint8, device="cuda")
    y, z = (torch.empty((m, n), dtype=torch.float16, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    tb.trellis_f8_gemm(L, q, s, out=y, ws=ws)
    tb.trellis_f8_moe_gemm(E, q, s, off, out=z, ws=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tb.trellis_f8_gemm(L, q, s, out=y, ws=ws)
        tb.trellis_f8_moe_gemm(E, q, s, off, out=z, ws=ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(4):
        q2, s2 = make_rows(m, k, g)
        q.copy_(q2)
        s.copy_(s2)
        torch.cuda.synchronize()
        graph.replay()
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append((tb.trellis_f8_gemm(L, q2, s2), tb.trellis_f8_moe_gemm(E, q2, s2, off)))
        torch.cuda.synchronize()
        for a, b in got:
            assert torch.equal(a, y) and torch.equal(b, z)
        check_product(y, q2, s2, L.w, L.scale, "fp16")
    assert tb.error_word() == 0 and tb.error_word(ws) == 0


@pytest.mark.parametrize("m", [20, 1100])
def test_rows_past_4_gib(m):
    """Rows whose strides carry them past 2^32 bytes: read and written where they are."""
    log_case(f"f8 rows past 4 GiB m={m}")
    g = torch.Generator().manual_seed(m)
    n, k = 272, 400
    stride = (2 ** 32 // (m - 2) // 16 + 1) * 16
    L, E = make_matrix(n, k, g), make_matrix(n, k, g, 2)
    q, s = make_rows(m, k, g)
    far = torch.empty((m, stride), dtype=torch.float8_e4m3fn, device="cuda")[:, :k]
    far.copy_(q)
    out = torch.empty((m, stride // 2), dtype=torch.float16, device="cuda")[:, :n]
    tb.trellis_f8_gemm(L, far, s, out=out)
    assert torch.equal(out, tb.trellis_f8_gemm(L, q, s))
    off = ints([0, m // 2, m])
    tb.trellis_f8_moe_gemm(E, far, s, off, out=out)
    assert torch.equal(out, tb.trellis_f8_moe_gemm(E, q, s, off))
    x = out[:, :256]
    for a, b in ((tb.trellis_f8_norm(x, None, 1e-6), tb.trellis_f8_norm(x.contiguous(), None, 1e-6)),
                 (tb.trellis_f8_silu_mul(x), tb.trellis_f8_silu_mul(x.contiguous()))):
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    order = ints([m - 1, 0, m - 2])
    assert torch.equal(tb.trellis_moe_gather(x, order, 1), x[order.long()])


def test_moe_gemm_of_very_many_tiles():
    """More tiles than a launch has workgroups: each takes a row of them."""
    log_case("f8 moe_gemm very many tiles")
    experts, n, k, each = 65536, 4112, 16, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randint(0, 0x7F, (experts, n, k), dtype=torch.uint8, device="cuda", generator=g).view(torch.float8_e4m3fn)
    L = tb.F8Linear(w, torch.rand((experts, n // 128 + 1, 1), device="cuda", generator=g))
    q = torch.randint(0, 0x7F, (experts * each, k), dtype=torch.uint8, device="cuda", generator=g).view(torch.float8_e4m3fn)
    s = torch.rand((experts * each, 1), device="cuda", generator=g) / 256
    off = torch.arange(0, experts * each + 1, each, dtype=torch.int32, device="cuda")
    y = tb.trellis_f8_moe_gemm(L, q, s, off, dtype=torch.bfloat16)
    for e in (0, 1, 31337, experts - 1):
        at = slice(e * each, (e + 1) * each)
        check_product(y[at], q[at], s[at], L.w[e], L.scale[e], "bf16")
    assert tb.error_word() == 0
