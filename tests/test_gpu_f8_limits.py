"""Block-scaled FP8 and routed tokens at the ends of what their headers allow: no rows at all, the most
rows, entries and choices, outputs in place of inputs, an expert's rows all but one elsewhere.

Large calls are compared with small ones over the same rows, bit for bit: a row's result does not depend
on the others."""
import numpy as np
import pytest
import torch

from oracle import f8 as FO
from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case
from test_gpu_f8 import DT, U, check_product, check_rounded, host, ints, make_matrix, make_rows
from test_gpu_route import routing

pytestmark = pytest.mark.gpu


def raw(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return all(x is y or torch.equal(raw(x), raw(y)) for x, y in zip(a, b))


def test_nothing():
    log_case("f8 nothing")
    x = torch.zeros((0, 256), dtype=torch.float16, device="cuda")
    q, s, h = tb.trellis_f8_norm(x, None, 1e-6, residual=x)
    assert q.shape == (0, 256) and s.shape == (0, 2) and h.shape == (0, 256)
    q, s = tb.trellis_f8_silu_mul(x)
    assert q.shape == (0, 128) and s.shape == (0, 1)
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    out = torch.full((6, 256), 5.0, dtype=torch.float16, device="cuda")
    assert (tb.trellis_moe_gather(x, none.view(-1), 2, out=out) == 5.0).all()
    assert (tb.trellis_moe_combine(x, none) == 0).all()
    add = torch.randn((3, 256), device="cuda").half()
    assert torch.equal(tb.trellis_moe_combine(x, none, add=add), add)
    d_y, d_w = tb.trellis_moe_combine_grad(add, x, none)
    assert d_y.shape == (0, 256) and (d_w == 0).all()
    empty = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert tb.trellis_moe_combine(out, empty).shape == (0, 256)
    d_y, d_w = tb.trellis_moe_combine_grad(x, out, empty, out=out)
    assert (out == 5.0).all() and d_w.shape == (0, 2) and tb.error_word() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_norm_in_place_of_its_input(dtype):
    log_case(f"f8 norm in place {dtype}")
    g = torch.Generator().manual_seed(0)
    x, r = (torch.randn((37, 2064), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    gamma = torch.rand((2064,), generator=g).to(DT[dtype]).cuda()
    want = tb.trellis_f8_norm(x, gamma, 1e-6, residual=r)
    z = x.clone()
    got = tb.trellis_f8_norm(z, gamma, 1e-6, residual=r, h=z)
    assert got[2] is z and same(got, want)
    z = x.clone()  # without a residual h is x
    got = tb.trellis_f8_norm(z, gamma, 1e-6, h=z)
    assert torch.equal(z, x) and same(got[:2], tb.trellis_f8_norm(x, gamma, 1e-6)[:2])
    both = x.clone()  # x as its own residual
    assert same(tb.trellis_f8_norm(both, gamma, 1e-6, residual=both, h=both), tb.trellis_f8_norm(x, gamma, 1e-6, residual=x))


def test_most_rows_of_norm_and_activation():
    log_case("f8 most rows")
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = 2 ** 22 - 1
    x = torch.randn((rows, 32), device="cuda", generator=g, dtype=torch.float16)
    got = tb.trellis_f8_norm(x, None, 1e-6, residual=x)
    for at in (slice(0, 70), slice(rows // 2, rows // 2 + 70), slice(rows - 70, rows)):
        assert same([t[at] for t in got], tb.trellis_f8_norm(x[at], None, 1e-6, residual=x[at]))
    del got
    rows = 2 ** 25 + 33  # more blocks than the activation's grid takes at a time
    x = torch.randn((rows, 32), device="cuda", generator=g, dtype=torch.float16)
    got = tb.trellis_f8_silu_mul(x)
    for at in (slice(0, 70), slice(2 ** 25 - 40, 2 ** 25 + 33)):
        assert same([t[at] for t in got], tb.trellis_f8_silu_mul(x[at]))


@pytest.mark.parametrize("n,k", [(24, 16), (264, 144)])
def test_very_many_rows_by_one_matrix(n, k):
    log_case(f"f8 gemm very many rows n={n} k={k}")
    g = torch.Generator().manual_seed(n)
    L, rows = make_matrix(n, k, g), 2 ** 21 + 77
    q = torch.randint(0, 0x7F, (rows, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.rand((rows, -(-k // 128)), device="cuda")
    y = tb.trellis_f8_gemm(L, q, s, dtype=torch.bfloat16)
    for at in (slice(0, 300), slice(2 ** 20 - 100, 2 ** 20 + 200), slice(rows - 300, rows)):
        check_product(y[at], q[at], s[at], L.w, L.scale, "bf16")
    assert tb.error_word() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens,top,n", [(3, 65, 264), (2, 130, 2056), (1, 1024, 40)])
def test_combine_of_many_choices(dtype, tokens, top, n):
    log_case(f"moe combine {dtype} tokens={tokens} top={top} n={n}")
    g = torch.Generator().manual_seed(top)
    _, _, inv = tb.trellis_moe_sort(routing(tokens, top, 8, g, 0.7), 8)
    rows = tokens * top
    y, a = torch.randn((rows, n), generator=g).to(DT[dtype]).cuda(), torch.randn((tokens, n), generator=g).to(DT[dtype]).cuda()
    w = torch.randn((tokens, top), generator=g).cuda()
    ref, mass = FO.combine(host(y), inv.cpu().numpy(), host(w), host(a))
    check_rounded(host(tb.trellis_moe_combine(y, inv, w, add=a)), ref, dtype, 0.0, (top + 1) * U * mass)
    # one row for every choice: it may be named more than once
    one = torch.zeros_like(inv)
    ref, mass = FO.combine(host(y), one.cpu().numpy(), host(w))
    check_rounded(host(tb.trellis_moe_combine(y, one, w)), ref, dtype, 0.0, (top + 1) * U * mass)
    d_y, d_w = tb.trellis_moe_combine_grad(a, y, inv, w, out=torch.full_like(y, 9.0))
    r_y, r_w, r_m = FO.combine_grad(host(a), host(y), inv.cpu().numpy(), host(w))
    named = ~np.isnan(r_y[:, 0])
    assert (host(d_y)[~named] == 9.0).all()
    check_rounded(host(d_y)[named], r_y[named], dtype, U)
    assert (np.abs(host(d_w) - r_w) <= (8 * -(-n // 2048) + 8) * U * r_m).all()
    assert tb.error_word() == 0


def test_more_tokens_than_a_launch_has_workgroups():
    log_case("moe very many tokens")
    tokens, n = 2 ** 22 + 5, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x, d = (torch.randn((tokens, n), device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand((tokens, 1), device="cuda", generator=g)
    order = torch.randperm(tokens, device="cuda", generator=g)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(tokens, device="cuda")
    order, inv = order.int(), inv.int()[:, None]
    xs = tb.trellis_moe_gather(x, order, 1)
    assert torch.equal(xs, x[order.long()])
    out = tb.trellis_moe_combine(xs, inv, w)
    assert torch.equal(out, (x.float() * w).bfloat16())
    d_y, d_w = tb.trellis_moe_combine_grad(d, xs, inv, w)
    assert torch.equal(d_y, (d.float() * w).bfloat16()[order.long()])
    ref, mass = (d.double() * x.double()).sum(1), (d.double() * x.double()).abs().sum(1)
    assert ((d_w[:, 0].double() - ref).abs() <= 16 * U * mass).all() and tb.error_word() == 0


@pytest.mark.parametrize("tokens,top,experts", [(2 ** 21, 8, 2048), (2 ** 24, 1, 3), (2 ** 14, 1024, 100)])
def test_most_entries_of_a_sort(tokens, top, experts):
    log_case(f"moe sort tokens={tokens} top={top} experts={experts}")
    g = torch.Generator(device="cuda").manual_seed(experts)
    ids = torch.randint(-1, experts, (tokens, top), device="cuda", generator=g, dtype=torch.int32)
    off, order, inv = tb.trellis_moe_sort(ids, experts)
    key, at = torch.where(ids.view(-1) < 0, experts, ids.view(-1)).sort(stable=True)
    here = int((ids >= 0).sum())
    assert int(off[0]) == 0 and torch.equal(off[1:].long(), torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0))
    assert torch.equal(order[:here].long(), at[:here]) and (order[here:] == -1).all()
    want = torch.full_like(at, -1)
    want[at[:here]] = torch.arange(here, device="cuda")
    assert torch.equal(inv.view(-1).long(), want) and tb.error_word() == 0


@pytest.mark.parametrize("experts", [1, 2, 300])
def test_one_expert_with_nearly_all_rows(experts):
    """Planned for rows spread evenly, run with them at one expert."""
    log_case(f"f8 moe_gemm uneven experts={experts}")
    g = torch.Generator().manual_seed(experts)
    n, k, rows = 264, 400, 700
    L = make_matrix(n, k, g, experts)
    q, s = make_rows(rows, k, g)
    most = experts // 2
    off = [0] * (most + 1) + [rows - (experts > 1)] * (experts - most)
    off[-1] = rows
    y = tb.trellis_f8_moe_gemm(L, q, s, ints(off), dtype=torch.bfloat16)
    for e in range(experts):
        a, b = off[e], off[e + 1]
        if a < b:
            check_product(y[a:b], q[a:b], s[a:b], L.w[e], L.scale[e], "bf16")
    assert tb.error_word() == 0


@pytest.mark.parametrize("experts,n,k", [(64, 4096, 1040), (200, 2056, 784)])
def test_many_experts_with_few_and_many_rows(experts, n, k):
    """Calls that are planned for wide tiles, with experts of every number of rows between 0 and 600."""
    log_case(f"f8 moe_gemm uneven experts={experts} n={n} k={k}")
    g = torch.Generator().manual_seed(experts)
    counts = (torch.rand(experts, generator=g) ** 3 * 600).int().tolist()
    counts[:8] = [1, 0, 31, 32, 33, 64, 65, 600]
    off = np.concatenate([[0], np.cumsum(counts)])
    rows, per = int(off[-1]), 4
    gd = torch.Generator(device="cuda").manual_seed(experts)
    w = torch.randint(0, 0x7F, (experts, n, k), dtype=torch.uint8, device="cuda", generator=gd).view(torch.float8_e4m3fn)
    L = tb.F8Linear(w, torch.rand((experts, -(-n // 128), -(-k // 128)), device="cuda", generator=gd))
    q, s = make_rows(-(-rows // per), k, g)
    order = torch.randperm(len(q) * per, generator=g)[:rows].to(torch.int32).cuda()
    y = tb.trellis_f8_moe_gemm(L, q, s, ints(off.tolist()), order=order, per=per, dtype=torch.bfloat16)
    src = order.long() // per
    for e in [*range(8), 17, experts - 1]:
        at = src[off[e]:off[e + 1]]
        if counts[e]:
            check_product(y[off[e]:off[e + 1]], q.view(torch.uint8)[at].view(torch.float8_e4m3fn), s[at], L.w[e], L.scale[e], "bf16")
    assert tb.error_word() == 0
