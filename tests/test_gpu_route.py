"""Tokens sorted by expert and back on the GPU against the oracle, their gradients against the
formula's and against differences, and a whole routed-expert step.

Tolerances: a combined value takes top fused multiply-adds, top u sum |terms| before its rounding
to 16 bits; a weight's gradient a chain of at most 8 ceil(n / 2048) + 8 additions a thread and over
the workgroup; u = 2^-24."""
import numpy as np
import pytest
import torch

from oracle import f8 as FO
from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case
from test_gpu_f8 import DT, HALF, U, check_product, check_quantized, check_rounded, host, ints, make_matrix

pytestmark = pytest.mark.gpu


def routing(tokens, top, experts, g, share=1.0):
    """Distinct ids a token; with a share below 1 the others are -1."""
    ids = torch.rand((tokens, experts), generator=g).topk(min(top, experts), -1).indices.to(torch.int32)
    if top > experts:
        ids = torch.randint(0, experts, (tokens, top), generator=g, dtype=torch.int32)
    return torch.where(torch.rand((tokens, top), generator=g) < share, ids, torch.tensor(-1, dtype=torch.int32)).cuda()


@pytest.mark.parametrize("tokens,top,experts,share", [
    (1, 1, 1, 1.0), (1, 8, 256, 1.0), (3, 5, 2, 1.0), (64, 1, 64, 1.0), (65, 8, 7, 0.5), (33, 8, 256, 1.0), (128, 8, 2048, 1.0),
    (513, 8, 256, 0.25), (1024, 3, 63, 1.0), (5000, 6, 65, 0.9), (4, 1024, 100, 0.7), (20, 4, 16, 0.0), (8193, 8, 256, 1.0),
    (20000, 8, 64, 1.0), (16384, 4, 2048, 0.5), (100001, 8, 130, 0.6), (8192, 8, 64, 1.0), (65537, 1, 300, 0.9),
])
def test_sort(tokens, top, experts, share):
    log_case(f"moe sort tokens={tokens} top={top} experts={experts} share={share}")
    g = torch.Generator().manual_seed(tokens + experts)
    ids = routing(tokens, top, experts, g, share)
    off, order, inv = tb.trellis_moe_sort(ids, experts)
    ro, rr, ri, _ = FO.sort(ids.cpu().numpy(), experts)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(order.cpu().numpy(), rr) and np.array_equal(inv.cpu().numpy(), ri)
    assert tb.error_word() == 0


@pytest.mark.parametrize("experts", [1636, 1637, 1638, 1639, 2047])
@pytest.mark.parametrize("tokens", [7, 16500])
def test_sort_where_its_shared_memory_passes_64_kib(tokens, experts):
    """Which takes an opt-in that every byte of the kernel's counts for."""
    log_case(f"moe sort tokens={tokens} experts={experts}")
    g = torch.Generator().manual_seed(tokens + experts)
    ids = torch.randint(-1, experts, (tokens, 4), generator=g, dtype=torch.int32)
    ids[0, 0], ids[-1, -1] = experts - 1, 0
    off, order, inv = tb.trellis_moe_sort(ids.cuda(), experts)
    ro, rr, ri, _ = FO.sort(ids.numpy(), experts)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(order.cpu().numpy(), rr) and np.array_equal(inv.cpu().numpy(), ri)
    assert tb.error_word() == 0


@pytest.mark.parametrize("tokens", [1, 500, 20000])
def test_sort_of_one_expert_and_of_bad_ids(tokens):
    log_case(f"moe sort special tokens={tokens}")
    ids = torch.full((tokens, 8), 3, dtype=torch.int32, device="cuda")
    off, order, inv = tb.trellis_moe_sort(ids, 5)
    n = 8 * tokens
    assert off.tolist() == [0, 0, 0, 0, n, n] and torch.equal(order, ints(list(range(n)))) and torch.equal(inv.view(-1), order)
    ids[0, 2], ids[-1, 5], ids[-1, 6] = 5, -2, 2 ** 31 - 1
    tb.clear_error_word()
    off, order, inv = tb.trellis_moe_sort(ids, 5)
    ro, rr, ri, bad = FO.sort(ids.cpu().numpy(), 5)
    assert bad and np.array_equal(order.cpu().numpy(), rr) and np.array_equal(inv.cpu().numpy(), ri) and np.array_equal(off.cpu().numpy(), ro)
    assert tb.error_word() == 1
    tb.clear_error_word()


def test_sort_of_nothing():
    log_case("moe sort nothing")
    off, order, inv = tb.trellis_moe_sort(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert off.tolist() == [0] * 10 and order.numel() == 0 and inv.shape == (0, 4)


@pytest.mark.parametrize("dtype,n,stride", [
    (torch.float16, 6144, 0), (torch.bfloat16, 8, 0), (torch.float16, 2, 2), (torch.bfloat16, 5000, 6), (torch.float32, 33, 0),
    (torch.float8_e4m3fn, 5120, 16), (torch.float8_e4m3fn, 20, 0), (torch.float16, 2056, 8)])
@pytest.mark.parametrize("tokens,top,share", [(1, 1, 1.0), (40, 8, 0.5), (300, 3, 1.0)])
def test_gather(dtype, n, stride, tokens, top, share):
    log_case(f"moe gather {dtype} n={n} stride=+{stride} tokens={tokens} top={top} share={share}")
    g = torch.Generator().manual_seed(n + tokens)
    _, order, _ = tb.trellis_moe_sort(routing(tokens, top, 16, g, share), 16)
    x = torch.randn((tokens, n + stride), generator=g).to(dtype).cuda()[:, :n]
    out = torch.ones((tokens * top, n), device="cuda").to(dtype)
    tb.trellis_moe_gather(x, order, top, out=out)
    want = torch.ones((tokens * top, n), device="cuda")
    live = order >= 0
    want[live] = x.float()[order[live].long() // top]
    assert torch.equal(out.float(), want) and tb.error_word() == 0
    order[0], order[-1] = tokens * top, -9
    want[0] = want[-1] = 1.0
    out.copy_(torch.ones_like(want))
    tb.trellis_moe_gather(x, order, top, out=out)
    assert torch.equal(out.float(), want) and tb.error_word() == 1
    tb.clear_error_word()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens,top,n,share,weighted,add", [
    (1, 1, 8, 1.0, True, False), (1, 8, 6144, 1.0, True, True), (5, 3, 2056, 0.5, False, False), (33, 8, 6144, 1.0, True, False),
    (7, 17, 264, 0.8, True, True), (300, 2, 1032, 0.0, True, False), (300, 2, 1032, 0.1, False, True), (70, 6, 5120, 0.6, True, True)])
def test_combine_and_its_gradient(dtype, tokens, top, n, share, weighted, add):
    log_case(f"moe combine {dtype} tokens={tokens} top={top} n={n} share={share} weighted={weighted} add={add}")
    g = torch.Generator().manual_seed(tokens * 3 + n)
    _, _, inv = tb.trellis_moe_sort(routing(tokens, top, 32, g, share), 32)
    rows = tokens * top
    y = torch.randn((rows, n), generator=g).to(DT[dtype]).cuda()
    w = torch.randn((tokens, top), generator=g).cuda() if weighted else None
    a = torch.randn((tokens, n), generator=g).to(DT[dtype]).cuda() if add else None
    live = set(inv[inv >= 0].tolist())
    dead = torch.tensor([p for p in range(rows) if p not in live], dtype=torch.long, device="cuda")
    y[dead] = float("nan")  # rows that no entry names are not read
    out = tb.trellis_moe_combine(y, inv, w, add=a)
    hi, hy = inv.cpu().numpy(), np.nan_to_num(host(y))
    hw, ha = host(w) if weighted else None, host(a) if add else None
    ref, mass = FO.combine(hy, hi, hw, ha)
    check_rounded(host(out), ref, dtype, 0.0, (top + 1) * U * mass)
    if add:
        assert torch.equal(tb.trellis_moe_combine(y, inv, w, add=a, out=a), out)

    d = torch.randn((tokens, n), generator=g).to(DT[dtype]).cuda()
    d_y, d_w = tb.trellis_moe_combine_grad(d, y, inv, w, out=torch.full_like(y, 9.0))
    r_y, r_w, r_m = FO.combine_grad(host(d), hy, hi, hw)
    named = ~np.isnan(r_y[:, 0])
    assert (host(d_y)[~named] == 9.0).all() and named.sum() == len(live)
    check_rounded(host(d_y)[named], r_y[named], dtype, U)
    assert (np.abs(host(d_w) - r_w) <= (8 * -(-n // 2048) + 8) * U * r_m).all()
    assert (host(d_w)[hi < 0] == 0).all()
    # in place, and without the weights' gradient
    y2 = y.clone()
    d_y2, d_w2 = tb.trellis_moe_combine_grad(d, y2, inv, w, out=y2)
    assert torch.equal(d_w2, d_w) and torch.equal(d_y2[torch.from_numpy(named).cuda()], d_y[torch.from_numpy(named).cuda()])
    assert tb.error_word() == 0


def test_gradients_are_the_differences():
    """Of the kernel itself: it is linear in each input, so a difference of two results is the
    gradient's product but for the results' roundings, 2^-8 of each value at most in bf16."""
    log_case("moe gradient differences")
    g = torch.Generator().manual_seed(5)
    tokens, top, n = 20, 4, 512
    ids = routing(tokens, top, 8, g, 0.8)
    _, order, inv = tb.trellis_moe_sort(ids, 8)
    y, e = (torch.randn((tokens * top, n), generator=g).bfloat16().cuda() for _ in range(2))
    w, v = (torch.randn((tokens, top), generator=g).cuda() for _ in range(2))
    d = torch.randn((tokens, n), generator=g).bfloat16().cuda()
    d_y, d_w = tb.trellis_moe_combine_grad(d, y, inv, w, out=torch.zeros_like(y))
    f = lambda y, w: host(tb.trellis_moe_combine(y, inv, w))  # noqa: E731
    base, hd = f(y, w), host(d)
    moved = f(e, w)  # the step from 0 to e
    room = HALF["bf16"] * (np.abs(hd) * np.abs(moved)).sum() + HALF["bf16"] * (np.abs(host(d_y)) * np.abs(host(e))).sum()
    assert abs((hd * moved).sum() - (host(d_y) * host(e)).sum()) <= room
    step = f(y, w + v) - base
    room = HALF["bf16"] * (np.abs(hd) * (np.abs(f(y, w + v)) + np.abs(base))).sum() + 1e-3
    assert abs((hd * step).sum() - (host(d_w) * host(v)).sum()) <= room
    # the gather's: d x is combine without weights
    x = torch.randn((tokens, n), generator=g).bfloat16().cuda()
    xs = tb.trellis_moe_gather(x, order, top, out=torch.zeros_like(y))
    d_x = host(tb.trellis_moe_combine(y, inv))
    room = HALF["bf16"] * (np.abs(host(x)) * np.abs(d_x)).sum()
    assert abs((host(xs) * host(y)).sum() - (host(x) * d_x).sum()) <= room


def test_bad_positions():
    log_case("moe bad positions")
    g = torch.Generator().manual_seed(6)
    inv = ints([[0, 1], [2, 6], [-5, 3], [2 ** 31 - 1, 5]])
    y = torch.randn((6, 264), generator=g).half().cuda()
    w, d = torch.randn((4, 2), generator=g).cuda(), torch.randn((4, 264), generator=g).half().cuda()
    tb.clear_error_word()
    out = tb.trellis_moe_combine(y, inv, w)
    assert tb.error_word() == 1
    tb.clear_error_word()
    ref, mass = FO.combine(host(y), inv.cpu().numpy(), host(w))
    check_rounded(host(out), ref, "fp16", 0.0, 3 * U * mass)
    d_y, d_w = tb.trellis_moe_combine_grad(d, y, inv, w, out=torch.full_like(y, 9.0))
    assert tb.error_word() == 1 and (d_y[4] == 9.0).all() and d_w[1, 1] == 0 and d_w[2, 0] == 0 and d_w[3, 0] == 0
    tb.clear_error_word()


def test_refusals():
    log_case("moe refusals")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    y = torch.zeros((8, 64), dtype=torch.float16, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    for error, f in (
            (tb.TrellisError, lambda: tb.trellis_moe_sort(ids, 0)), (tb.TrellisError, lambda: tb.trellis_moe_sort(ids, 2049)),
            (TypeError, lambda: tb.trellis_moe_sort(ids.long(), 4)), (ValueError, lambda: tb.trellis_moe_sort(ids.t(), 4)),
            (ValueError, lambda: tb.trellis_moe_sort(ids, 4, order=ids[:1])), (tb.TrellisError, lambda: tb.trellis_moe_sort(ids, 4, inverse=ids)),
            (tb.TrellisError, lambda: tb.trellis_moe_gather(y, ids.view(-1), 0)), (tb.TrellisError, lambda: tb.trellis_moe_gather(y[:, :3], ids.view(-1), 2)),
            (TypeError, lambda: tb.trellis_moe_combine(y.float(), ids)), (ValueError, lambda: tb.trellis_moe_combine(y, ids, w[:3])),
            (ValueError, lambda: tb.trellis_moe_combine(y[:, :32], ids)), (ValueError, lambda: tb.trellis_moe_combine(y, ids, add=y)),
            (tb.TrellisError, lambda: tb.trellis_moe_combine(y, ids, out=y[:4])), (ValueError, lambda: tb.trellis_moe_combine_grad(y, y, ids)),
            (tb.TrellisError, lambda: tb.trellis_moe_combine_grad(y[:4], y.clone(), ids, out=y))):
        with pytest.raises(error):
            f()


def step(x, residual, gamma, ids, weights, up, down, top):
    """A routed-expert layer: norm, products with the experts' gate | up, activation, down, back
    into the residual."""
    q, s, h = tb.trellis_f8_norm(x, gamma, 1e-6, residual=residual)
    off, order, inv = tb.trellis_moe_sort(ids, up.experts)
    gu = tb.trellis_f8_moe_gemm(up, q, s, off, order=order, per=top, dtype=x.dtype)
    qa, sa = tb.trellis_f8_silu_mul(gu)
    rows = tb.trellis_f8_moe_gemm(down, qa, sa, off, dtype=x.dtype)
    return tb.trellis_moe_combine(rows, inv, weights, add=h), (q, s, h, off, order, inv, gu, qa, sa, rows)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens,top,experts,hidden,inter,gain", [
    (1, 2, 4, 256, 128, 1), (37, 4, 16, 640, 272, 1), (300, 2, 4, 512, 256, 1), (1, 2, 4, 256, 128, 40), (37, 4, 16, 640, 272, 40),
    (300, 2, 4, 512, 256, 40)])
def test_routed_expert_step(dtype, tokens, top, experts, hidden, inter, gain):
    """The operators together, each stage against the oracle on the stage before, then captured and
    replayed with other tokens."""
    log_case(f"moe step {dtype} tokens={tokens} top={top} experts={experts} hidden={hidden} inter={inter} gain={gain}")
    g = torch.Generator().manual_seed(tokens)
    up, down = make_matrix(2 * inter, hidden, g, experts, gain), make_matrix(hidden, inter, g, experts, gain)
    gamma = (1 + 0.1 * torch.randn(hidden, generator=g)).to(DT[dtype]).cuda()
    x, res = (torch.randn((tokens, hidden), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    ids, w = routing(tokens, top, experts, g), torch.softmax(torch.randn((tokens, top), generator=g), -1).cuda()
    for _ in range(2):  # (the second pass: the workspace as the first left it)
        out, (q, s, h, off, order, inv, gu, qa, sa, rows) = step(x, res, gamma, ids, w, up, down, top)
    v, rh = FO.norm(host(x), 1e-6, host(gamma), host(res))
    check_quantized(host(q), host(s), v, 2.0 ** -20, 2.0 ** -19)
    check_rounded(host(h), rh, dtype, U)
    o, src = off.tolist(), order.long() // top
    raw = lambda t, i: t.view(torch.uint8)[i].view(torch.float8_e4m3fn)  # noqa: E731
    for e in range(experts):
        a, b = o[e], o[e + 1]
        if a < b:
            check_product(gu[a:b], raw(q, src[a:b]), s[src[a:b]], up.w[e], up.scale[e], dtype)
            check_product(rows[a:b], qa[a:b], sa[a:b], down.w[e], down.scale[e], dtype)
    check_quantized(host(qa), host(sa), FO.silu_mul(host(gu)), 2.0 ** -20, 2.0 ** -20)
    ref, mass = FO.combine(host(rows), inv.cpu().numpy(), host(w), host(h))
    check_rounded(host(out), ref, dtype, 0.0, (top + 1) * U * mass)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(x, res, gamma, ids, w, up, down, top)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cap, _ = step(x, res, gamma, ids, w, up, down, top)
    for i in range(3):
        x.copy_(torch.randn((tokens, hidden), generator=g))
        ids.copy_(routing(tokens, top, experts, g, 0.8))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, step(x, res, gamma, ids, w, up, down, top)[0])
    assert tb.error_word() == 0


def test_rows_past_4_gib():
    log_case("moe rows past 4 GiB")
    rows, n, tokens, top = 2 ** 21 + 5, 1024, 3, 4
    g = torch.Generator().manual_seed(0)
    y = torch.empty((rows, n), dtype=torch.float16, device="cuda")
    inv = ints([rows - 1 - i for i in range(tokens * top)]).view(tokens, top)
    few, w = torch.randn((tokens * top, n), generator=g).half().cuda(), torch.rand((tokens, top), generator=g).cuda()
    d = torch.randn((tokens, n), generator=g).half().cuda()
    y[rows - tokens * top:] = few
    back = (tokens * top - 1 - torch.arange(tokens * top, dtype=torch.int32)).view(tokens, top).cuda()
    assert torch.equal(tb.trellis_moe_combine(y, inv, w), tb.trellis_moe_combine(few, back, w))
    want, dw = tb.trellis_moe_combine_grad(d, few, back, w)
    got, dv = tb.trellis_moe_combine_grad(d, y, inv, w, out=y)
    assert got is y and torch.equal(y[rows - tokens * top:], want) and torch.equal(dv, dw)
    order = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    order[rows - 2:] = ints([2, 1])
    tb.trellis_moe_gather(d, order, 1, out=y)
    assert torch.equal(y[rows - 2:], d[[2, 1]]) and torch.equal(y[rows - tokens * top:rows - 2], want[:-2])
    assert tb.error_word() == 0


@pytest.mark.parametrize("tokens", [40, 9000])
def test_routing_and_its_gradients_in_a_graph(tokens):
    """Captured with a workspace of its own and replayed with other routings (9000 tokens: the sort's
    three launches), between eager calls."""
    log_case(f"moe routing graph tokens={tokens}")
    g = torch.Generator().manual_seed(tokens)
    top, experts, n = 8, 64, 136
    x, d = (torch.randn((tokens, n), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w, ids = torch.rand((tokens, top), generator=g).cuda(), routing(tokens, top, experts, g, 0.8)
    xs, dy = (torch.zeros((tokens * top, n), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def run(ws=None):
        xs.zero_()
        dy.zero_()
        off, order, inv = tb.trellis_moe_sort(ids, experts, ws=ws)
        tb.trellis_moe_gather(x, order, top, out=xs, ws=ws)
        out = tb.trellis_moe_combine(xs, inv, w, add=x, ws=ws)
        _, dw = tb.trellis_moe_combine_grad(d, xs, inv, w, out=dy, ws=ws)
        return off, order, inv, out, dw, tb.trellis_moe_combine(dy, inv, ws=ws)

    run()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ws)
    for _ in range(4):
        ids.copy_(routing(tokens, top, experts, g, 0.8))
        graph.replay()
        kept = [t.clone() for t in got] + [xs.clone(), dy.clone()]
        assert all(torch.equal(a, b) for a, b in zip(kept, list(run()) + [xs, dy]))
    assert tb.error_word() == 0 and tb.error_word(ws) == 0
