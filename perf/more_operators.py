"""The operators of a routed-expert step over matrices held in block-scaled FP8, for measurement.

Each case is one pass of a model's step: the norm in front of a product (with the residual's
addition, its result quantised to E4M3 with one scale per 128 channels), the experts'
activation quantised the same way, products of E4M3 activations with E4M3 weights that have one
scale per 128 x 128 block (one matrix, or one per expert), and tokens sorted by expert and
brought back with their weights, forwards and backwards.  `own` selects the library's kernels;
otherwise the same operators run as elementary torch operations in 32 bits.

E4M3 results are returned as float8_e4m3fn tensors beside the scales that multiply them.
"""
import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
_E4M3 = torch.float8_e4m3fn
_MAX = 448.0


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one token of one chat, in front of a product: latency
        dict(name="norm_token", op="norm", dtype="fp16", rows=1, n=5120, residual=True),
        # a scheduler's step of prompt chunks, an odd number of rows
        dict(name="norm_prompt", op="norm", dtype="bf16", rows=4097, n=6144, residual=True),
        # the experts' activation of a decode step: few rows
        dict(name="act_batch", op="act", dtype="bf16", rows=264, n=2048),
        # the dense layer's activation over a prompt
        dict(name="act_prompt", op="act", dtype="fp16", rows=2048, n=17408),
        # one token through a wide projection: the weights are read once
        dict(name="gemm_token", op="gemm", dtype="fp16", rows=1, n=17408, k=5120),
        # a decode batch through an output projection
        dict(name="gemm_batch", op="gemm", dtype="bf16", rows=37, n=5120, k=6144),
        # a prompt through a wide projection
        dict(name="gemm_prompt", op="gemm", dtype="fp16", rows=2048, n=17408, k=5120),
        # a decode batch's routed entries through their gate and up matrices: about two rows an expert
        dict(name="experts_batch", op="experts", dtype="bf16", tokens=33, top=8, experts=256, n=4096, k=6144, here=1.0,
             gather=True),
        # a prompt's routed entries through one shard's gate and up matrices: hundreds of rows an expert
        dict(name="experts_prompt", op="experts", dtype="fp16", tokens=4096, top=8, experts=64, n=4096, k=6144, here=1.0,
             gather=True),
        # a decode batch's tokens sorted by expert, and back
        dict(name="route_batch", op="route", dtype="fp16", tokens=33, top=8, experts=256, n=6144, here=1.0),
        # a prompt's tokens sorted by expert, and back, on a shard that holds half of the experts
        dict(name="route_prompt", op="route", dtype="bf16", tokens=4097, top=8, experts=256, n=6144, here=0.5),
        # the gradients of both directions over a training batch
        dict(name="route_grad", op="route_grad", dtype="bf16", tokens=4096, top=8, experts=64, n=5120, here=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "act", "gemm", "gemm", "experts", "experts", "route", "route_grad"))
    c = dict(op=op, dtype=rng.choice(("fp16", "bf16")))
    if op == "norm":
        n = 16 * _log(rng, 8, 1024)
        c.update(rows=_log(rng, 1, min(8000, 40000000 // n)), n=n, residual=rng.random() < 0.7)
    elif op == "act":
        n = 16 * _log(rng, 8, 1200)
        c.update(rows=_log(rng, 1, min(40000, 40000000 // n)), n=n)
    elif op == "gemm":
        n, k = 8 * _log(rng, 12, 2400), 16 * _log(rng, 8, 640)
        c.update(rows=_log(rng, 1, 3000), n=n, k=k)
    elif op == "experts":
        experts = _log(rng, 4, 256)
        k = 16 * _log(rng, 16, 450)
        n = 8 * _log(rng, 32, max(32, min(700, 1500000000 // (8 * k * experts))))
        c.update(tokens=_log(rng, 1, 2500), top=min(experts, rng.choice((1, 2, 4, 6, 8))), experts=experts, n=n, k=k,
                 here=rng.choice((1.0, 1.0, 0.5)), gather=rng.random() < 0.6)
    else:
        experts = _log(rng, 4, 512)
        c.update(tokens=_log(rng, 1, 5000), top=min(experts, rng.choice((1, 2, 4, 6, 8))), experts=experts,
                 n=8 * _log(rng, 16, 900), here=rng.choice((1.0, 1.0, 0.25)))
    return c


def _popularity(experts):
    """How often each expert is chosen, in relation: the busiest about ten times the idlest."""
    return [math.exp(0.55 * (4.0 * (e + 0.5) / experts - 2.0)) for e in range(experts)]


def _expected(case):
    """(experts with at least one entry, entries whose expert is here), in expectation."""
    p = _popularity(case["experts"])
    total = sum(p)
    n = case["tokens"] * case["top"]
    touched = sum(1.0 - (1.0 - min(1.0, case["top"] * x / total)) ** case["tokens"] for x in p)
    return case["here"] * touched, case["here"] * n


def work(case):
    op = case["op"]
    if op == "norm":
        e = case["rows"] * case["n"]
        per = 2 + 1 + 4 / 128 + (4 if case["residual"] else 0)
        return {"bytes": e * per + 2 * case["n"], "flops": 8 * e}
    if op == "act":
        e = case["rows"] * case["n"]
        return {"bytes": e * (4 + 1 + 4 / 128), "flops": 8 * e}
    if op == "gemm":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": m * k * (1 + 4 / 128) + n * k * (1 + 4 / 16384) + 2 * m * n, "flops": 2 * m * n * k}
    touched, rows = _expected(case)
    n = case["n"]
    if op == "experts":
        k = case["k"]
        x_rows = case["tokens"] if case["gather"] else rows
        return {"bytes": touched * n * k * (1 + 4 / 16384) + x_rows * k * (1 + 4 / 128) + rows * (2 * n + 4),
                "flops": 2 * rows * n * k}
    ids = 4 * case["tokens"] * case["top"]
    rows_bytes, tokens_bytes = 2 * n * rows, 2 * n * case["tokens"]
    if op == "route":  # ids in, three lists out; tokens in, rows out; rows, weights in, tokens out
        return {"bytes": 3 * ids + 2 * (rows_bytes + tokens_bytes) + 2 * ids, "flops": 2 * n * rows}
    # d out, rows, weights in, d rows and d weights out; d rows in, d tokens out
    return {"bytes": 3 * rows_bytes + 2 * tokens_bytes + 4 * ids, "flops": 4 * n * rows}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------

def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=g, dtype=dtype)


def _hidden(rows, n, g, dtype):
    """Activations as a deep model has them: rows of different size, a few channels that stand out."""
    x = _randn((rows, n), g) * torch.exp(0.3 * _randn((rows, 1), g))
    x[:, ::97] *= 12.0
    return x.to(dtype)


def _blocks(x):
    """[..., n] padded with zeros to whole blocks: [..., blocks, 128]."""
    n = x.shape[-1]
    return torch.nn.functional.pad(x, (0, -n % 128)).unflatten(-1, (-1, 128))


def _weights(case, g):
    """E4M3 matrices [n, k] with a scale per 128 x 128 block, as a checkpoint holds them."""
    experts, n, k = case.get("experts", 1), case["n"], case["k"]
    if "experts" in case:
        experts = max(1, int(round(case["experts"] * case["here"])))
    nb, kb = -(-n // 128), -(-k // 128)
    w = torch.empty((experts, n, k), dtype=_E4M3, device="cuda")
    s = torch.empty((experts, nb, kb), device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for e in range(0, experts, step):
        v = _randn((min(step, experts - e), n, k), g) / math.sqrt(k)
        v[..., ::61] *= 3.0
        a = torch.nn.functional.pad(v, (0, -k % 128, 0, -n % 128)).unflatten(-1, (kb, 128)).unflatten(1, (nb, 128))
        s[e:e + step] = a.abs().amax((2, 4)) / _MAX
        full = s[e:e + step].repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
        w[e:e + step] = (v / full).to(_E4M3)
    return (w, s) if "experts" in case else (w[0], s[0])


def _quantised(x):
    b = _blocks(x.float())
    s = b.abs().amax(-1) / _MAX
    return (b / s[..., None]).to(_E4M3).flatten(-2)[..., :x.shape[-1]].contiguous(), s


def _routing(case, g):
    """int32 [tokens, top]: distinct experts a token, some more popular than others; with a share
    of the experts here, the others' ids are -1."""
    e = case["experts"]
    p = torch.log(torch.tensor(_popularity(e), device="cuda"))[torch.randperm(e, device="cuda", generator=g)]
    u = torch.rand((case["tokens"], e), device="cuda", generator=g).clamp(min=1e-7, max=1 - 1e-7)
    ids = (p - torch.log(-torch.log(u))).topk(case["top"], -1).indices.int()
    held = max(1, int(round(e * case["here"])))
    return torch.where(ids < held, ids, -1), held


def _sorted(ids, held):
    """(offsets, order, inverse) of a routing."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, held)
    order = torch.argsort(key, stable=True)
    offsets = torch.zeros(held + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=held + 1)[:held], 0)
    at = torch.arange(flat.numel(), device="cuda")
    inverse = torch.empty_like(at)
    inverse[order] = at
    inverse = torch.where(flat >= 0, inverse, -1)
    order = torch.where(at < offsets[-1], order, -1)
    return offsets.int(), order.int(), inverse.int().view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    dtype, op = _DT[case["dtype"]], case["op"]
    st = {"case": case, "dtype": dtype}
    if op == "norm":
        st["x"] = _hidden(case["rows"], case["n"], g, dtype)
        st["residual"] = (4.0 * _hidden(case["rows"], case["n"], g, torch.float32)).to(dtype) if case["residual"] else None
        st["gamma"] = (1.0 + 0.2 * _randn((case["n"],), g)).to(dtype)
    elif op == "act":
        st["x"] = (1.5 * _randn((case["rows"], 2 * case["n"]), g)).to(dtype)  # gate | up
    elif op == "gemm":
        st["w"], st["sw"] = _weights(case, g)
        st["q"], st["sx"] = _quantised(_hidden(case["rows"], case["k"], g, torch.float32))
    elif op == "experts":
        ids, held = _routing(case, g)
        st["offsets"], st["order"], _ = _sorted(ids, held)
        st["w"], st["sw"] = _weights(case, g)
        counts = (st["offsets"][1:] - st["offsets"][:-1]).tolist()
        st["most"] = max(1, max(counts))
        x = _hidden(case["tokens"], case["k"], g, torch.float32)
        if not case["gather"]:
            x = x[st["order"].clamp(min=0).long() // case["top"]]
        st["q"], st["sx"] = _quantised(x)
        # rows behind the last expert's stay as they are
        st["y"] = torch.zeros((case["tokens"] * case["top"], case["n"]), dtype=dtype, device="cuda")
    else:
        t, k, n = case["tokens"], case["top"], case["n"]
        st["ids"], st["held"] = _routing(case, g)
        st["weights"] = torch.softmax(_randn((t, k), g), -1)
        st["rows"] = _randn((t * k, n), g).to(dtype)  # the experts' outputs
        if op == "route":
            st["x"] = _hidden(t, n, g, dtype)
            st["xs"] = torch.zeros((t * k, n), dtype=dtype, device="cuda")
        else:
            _, _, st["inverse"] = _sorted(st["ids"], st["held"])
            st["d_out"] = _randn((t, n), g).to(dtype)
            st["d_xs"] = _randn((t * k, n), g).to(dtype)
            st["d_rows"] = torch.zeros((t * k, n), dtype=dtype, device="cuda")
    return st


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------

_EPS = 1e-6


def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from trellis_coded_bit_amd import binding as tb
    c = st["case"]
    if c["op"] == "norm":
        q, s, h = tb.trellis_f8_norm(st["x"], st["gamma"], _EPS, residual=st["residual"])
        return {"q": q, "scale": s, "h": h}
    if c["op"] == "act":
        q, s = tb.trellis_f8_silu_mul(st["x"])
        return {"q": q, "scale": s}
    if c["op"] == "gemm":
        return tb.trellis_f8_gemm(tb.F8Linear(st["w"], st["sw"]), st["q"], st["sx"], dtype=st["dtype"])
    if c["op"] == "experts":
        order, per = (st["order"], c["top"]) if c["gather"] else (None, 1)
        return tb.trellis_f8_moe_gemm(tb.F8Linear(st["w"], st["sw"]), st["q"], st["sx"], st["offsets"], order=order, per=per,
                                      dtype=st["dtype"], out=st["y"])
    if c["op"] == "route":
        offsets, order, inverse = tb.trellis_moe_sort(st["ids"], st["held"])
        xs = tb.trellis_moe_gather(st["x"], order, c["top"], out=st["xs"])
        out = tb.trellis_moe_combine(st["rows"], inverse, st["weights"])
        return {"offsets": offsets, "order": order, "inverse": inverse, "xs": xs, "out": out}
    d_rows, d_w = tb.trellis_moe_combine_grad(st["d_out"], st["rows"], st["inverse"], st["weights"], out=st["d_rows"])
    return {"d_rows": d_rows, "d_weights": d_w, "d_x": tb.trellis_moe_combine(st["d_xs"], st["inverse"])}


def _plain(st):
    c, dtype = st["case"], st["dtype"]
    if c["op"] == "norm":
        h = st["x"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        v = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS) * st["gamma"].float()
        q, s = _quantised(v)
        return {"q": q, "scale": s, "h": None if st["residual"] is None else h.to(dtype)}
    if c["op"] == "act":
        gate, up = st["x"].float().chunk(2, -1)
        q, s = _quantised(gate / (1.0 + torch.exp(-gate)) * up)
        return {"q": q, "scale": s}
    if c["op"] == "gemm":
        return (_values(st["q"], st["sx"]) @ _matrix(st["w"], st["sw"]).T).to(dtype)
    if c["op"] == "experts":
        return _plain_experts(st)
    top = c["top"]
    if c["op"] == "route":
        offsets, order, inverse = _sorted(st["ids"], st["held"])
        here = (order >= 0)[:, None]
        xs = torch.where(here, st["x"][order.clamp(min=0).long() // top], 0)
        rows = torch.where(inverse[..., None] >= 0, st["rows"][inverse.clamp(min=0).long()].float(), 0.0)
        out = (rows * st["weights"][..., None]).sum(1).to(dtype)
        return {"offsets": offsets, "order": order, "inverse": inverse, "xs": xs, "out": out}
    inverse = st["inverse"]
    at, here = inverse.clamp(min=0).long(), inverse[..., None] >= 0
    d_out = st["d_out"].float()[:, None]
    d_w = torch.where(here, st["rows"][at].float() * d_out, 0.0).sum(-1)
    d_rows = torch.zeros_like(st["d_rows"])
    t, j = torch.nonzero(inverse >= 0, as_tuple=True)
    d_rows[inverse[t, j].long()] = (st["weights"][t, j, None] * st["d_out"][t].float()).to(dtype)
    d_x = torch.where(here, st["d_xs"][at].float(), 0.0).sum(1).to(dtype)
    return {"d_rows": d_rows, "d_weights": d_w, "d_x": d_x}


def _values(q, s):
    """What E4M3 codes with a scale per 128 of the last axis stand for, in 32 bits."""
    return (_blocks(q.float()) * s[..., None]).flatten(-2)[..., :q.shape[-1]]


def _matrix(w, s):
    """What E4M3 codes [..., n, k] with a scale per 128 x 128 block stand for, in 32 bits."""
    n = w.shape[-2]
    return _values(w, s.repeat_interleave(128, -2)[..., :n, :])


def _plain_experts(st):
    """Every expert's rows padded to the fullest expert's number, one batch of products."""
    c, offsets, order = st["case"], st["offsets"].long(), st["order"].long()
    held, most = offsets.numel() - 1, st["most"]
    at = offsets[:-1, None] + torch.arange(most, device="cuda")
    live = at < offsets[1:, None]
    at = torch.where(live, at, 0)
    src = order.clamp(min=0)[at] // c["top"] if c["gather"] else at
    x = torch.where(live[..., None], _values(st["q"], st["sx"])[src], 0.0)
    y = torch.bmm(_matrix(st["w"], st["sw"]), x.transpose(1, 2).contiguous())  # [experts, n, most]
    out = torch.zeros_like(st["y"])
    e, i = torch.nonzero(live, as_tuple=True)
    out[at[e, i]] = y.transpose(1, 2)[e, i].to(st["dtype"])
    return out


# ---------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------

def _e4m3(v):
    """Nearest E4M3 value, ties to even mantissas: three bits behind the leading one, steps of
    2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def _quantised64(v):
    out, scales = torch.empty_like(v), []
    for b in range(0, v.shape[-1], 128):
        part = v[:, b:b + 128]
        s = part.abs().amax(-1, keepdim=True) / _MAX
        out[:, b:b + 128] = _e4m3(part / s)
        scales.append(s)
    return out, torch.cat(scales, -1)


def _product64(q, sx, w, sw):
    """rows [m, k] with scales [m, blocks] by one matrix [n, k] with scales per block."""
    y = torch.zeros((q.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    x, cols = q.double(), torch.arange(w.shape[0], device="cuda") // 128
    for b in range(sx.shape[1]):
        part = slice(128 * b, 128 * b + 128)
        y += (x[:, part] * sx[:, b, None].double()) @ (w[:, part].double() * sw[cols, b, None].double()).T
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double() + (0 if st["residual"] is None else st["residual"].double())
        v = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["n"] + _EPS) * st["gamma"].double()
        q, s = _quantised64(v)
        return {"q": q, "scale": s, "h": None if st["residual"] is None else h}
    if op == "act":
        x = st["x"].double()
        gate, up = x[:, :case["n"]], x[:, case["n"]:]
        q, s = _quantised64(gate * up / (1.0 + torch.exp(-gate)))
        return {"q": q, "scale": s}
    if op == "gemm":
        return _product64(st["q"], st["sx"], st["w"], st["sw"])
    if op == "experts":
        out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        offsets, order = st["offsets"].tolist(), st["order"].long()
        for e in range(len(offsets) - 1):
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                src = order[a:b] // case["top"] if case["gather"] else torch.arange(a, b, device="cuda")
                out[a:b] = _product64(st["q"][src], st["sx"][src], st["w"][e], st["sw"][e])
        return out
    t, k, n = case["tokens"], case["top"], case["n"]
    out = torch.zeros((t, n), dtype=torch.float64, device="cuda")
    weights = st["weights"].double()
    if op == "route":  # by lists on the host: each expert's entries in order
        ids = st["ids"].reshape(-1).tolist()
        lists = [[] for _ in range(st["held"])]
        for entry, e in enumerate(ids):
            if e >= 0:
                lists[e].append(entry)
        flat = [entry for entries in lists for entry in entries]
        place = [-1] * len(ids)
        for pos, entry in enumerate(flat):
            place[entry] = pos
        ends = [0]
        for entries in lists:
            ends.append(ends[-1] + len(entries))
        xs = torch.zeros((t * k, n), dtype=torch.float64, device="cuda")
        src = torch.tensor(flat, dtype=torch.int64, device="cuda")
        xs[:len(flat)] = st["x"][src // k].double()
        out.index_add_(0, src // k, st["rows"][:len(flat)].double() * weights.reshape(-1)[src, None])
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"offsets": ints(ends), "order": ints(flat + [-1] * (len(ids) - len(flat))), "inverse": ints(place).view(t, k),
                "xs": xs, "out": out}
    d_rows = torch.zeros((t * k, n), dtype=torch.float64, device="cuda")
    d_w = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        live = torch.nonzero(st["inverse"][:, j] >= 0)[:, 0]
        at = st["inverse"][live, j].long()
        d_rows[at] = weights[live, j, None] * st["d_out"][live].double()
        d_w[live, j] = (st["rows"][at].double() * st["d_out"][live].double()).sum(-1)
        out[live] += st["d_xs"][at].double()
    return {"d_rows": d_rows, "d_weights": d_w, "d_x": out}
