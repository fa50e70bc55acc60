"""Attention over the 4-bit cache where the values' sizes differ from tile to tile (a tile: 128
tokens), or between the two blocks of a head of 256: zeros between large values, sizes that fall and
rise by far more than the sums' types hold of one of them, large values that no weight reaches.

Bound per (row, head), in the 2-norm over its elements, from the formats alone.  A weight is rounded to
2^-11 of itself (fp16, or finer in three E4M3 parts), but to no less than a step of 2^-24 where its
tile's largest value scale is at least 1/2; an element of a rotated query to 2^-13.9 of its block's
largest (the last of its three E2M3 parts), which moves a score by at most s = |scale| 2^-13.9
max|q'| sum|k'| and a weight by twice that; the sums are fp32; the result is rounded to its type (u):
    |y - ref| <= (2^-11 + 2 s + 2^-17) sum_j p_j |v_j| + 2^-24 sum_j top(tile of j) / l + u |ref|
with p_j = e^(s_j - m) / l and top the largest |v| of a tile's tokens, per 128-block.
"""
import numpy as np
import pytest
import torch

from oracle import kv4 as KO
from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case
from test_gpu_kv4 import DT, UNIT, Setup, host, ints

pytestmark = pytest.mark.gpu

TILE = 128


def rotated(x):
    return (x.reshape(*x.shape[:-1], -1, 128) @ KO.H).reshape(x.shape)


def check(st, new, q, scale):
    """The last `new` rows of slot 0 against the oracle, each 128-block within the bound above."""
    rows, heads, D = q.shape
    length = st.host_lens[0]
    y = tb.trellis_kv4_attn(st.cache, 0, st.table, st.lens, ints([0, rows]), q, scale=scale, max_q=rows)
    torch.cuda.synchronize()
    assert tb.error_word() == 0
    got, qh = host(y), host(q)
    assert np.isfinite(got).all()
    oc, table = st.oracle(), st.table.cpu().numpy()
    k, v = (oc.rows(0, table[0], length, w) for w in (0, 1))
    qr, kr = rotated(qh), rotated(k)
    tiles = -(-length // TILE)
    for i in range(rows):
        n = length - rows + i + 1
        for h in range(heads):
            hk = h // (heads // st.Hk)
            s = scale * (k[:n, hk] @ qh[i, h])
            e = np.exp(s - s.max())
            p = e / e.sum()
            moved = abs(scale) * 2.0 ** -13.9 * np.abs(qr[i, h]).max() * np.abs(kr[:n, hk]).sum(-1)[p > 1e-30].max()
            for b in range(0, D, 128):
                size = np.linalg.norm(v[:, hk, b:b + 128], axis=-1)
                top = np.array([size[t * TILE:(t + 1) * TILE].max() for t in range(tiles)]).repeat(TILE)[:n]
                ref = p @ v[:n, hk, b:b + 128]
                bound = (2.0 ** -11 + 2 * moved + 2.0 ** -17) * (p @ size[:n]) + 2.0 ** -24 * top.sum() / e.sum() + \
                    UNIT[st.dtype] * np.linalg.norm(ref) + 1e-7 * (st.dtype == "fp16")  # (fp16's smallest numbers)
                err = np.linalg.norm(got[i, h, b:b + 128] - ref)
                assert err <= bound, (i, h, b, err, bound, np.linalg.norm(ref))


def filled(sizes, dtype, D, tail=70, even=False, keys=None):
    """A sequence of one tile per entry of `sizes` (a number, or one per block) and `tail` tokens more
    of the last one's size."""
    tokens = [s for s in sizes for _ in range(TILE)] + [sizes[-1]] * tail
    f = np.stack([np.repeat(np.broadcast_to(np.atleast_1d(np.float64(s)), D // 128), 128) for s in tokens])
    g = torch.Generator().manual_seed(31)
    st = Setup([len(tokens)], T=64, Hk=1, D=D, dtype=dtype, fill=False)
    v = 2 * torch.ones((len(tokens), 1, D), dtype=torch.float64) if even else \
        torch.randn((len(tokens), 1, D), generator=g).clamp(-2, 2).double()
    k = torch.randn((len(tokens), 1, D), generator=g) if keys is None else keys(tokens, g)
    v = v * torch.from_numpy(f)[:, None]
    tb.trellis_kv4_append(st.cache, 0, st.table, st.lens, ints([0, len(tokens)]), k.to(DT[dtype]).cuda(), v.to(DT[dtype]).cuda())
    return st


FP16 = [
    [30000.0] * 8 + [0.0],
    [30000.0] * 4 + [0.0],
    [20000.0] * 20 + [0.0, 20000.0],
    [0.0, 0.0, 1.0, 0.0, 1e-3, 1000.0, 0.0],
    [0.0, 0.0],
]
BF16 = [
    [2.0 ** 60, 2.0 ** -60],
    [2.0 ** 60, 2.0 ** -60, 2.0 ** 60],
    [2.0 ** 100, 0.0, 2.0 ** -90, 2.0 ** -30, 0.0, 2.0 ** 90],
    [2.0 ** -90, 2.0 ** 30, 2.0 ** -90, 2.0 ** -10],
    [2.0 ** 30, 0.0],
]


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("even", [True, False])
@pytest.mark.parametrize("dtype,sizes", [("fp16", s) for s in FP16] + [("bf16", s) for s in BF16])
def test_values_that_differ_between_tiles(dtype, sizes, even, D, new):
    """All keys weigh the same: the sums hold what every tile's values come to."""
    log_case(f"attn tiles' values {dtype} {sizes} even={even} D={D} new={new}")
    st = filled(sizes, dtype, D, even=even)
    check(st, new, torch.zeros((new, 4, D), dtype=DT[dtype], device="cuda"), D ** -0.5)


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("sizes", [
    [(0.0, 2.0 ** 60), (0.0, 2.0 ** 60)],
    [(2.0 ** 60, 0.0), (2.0 ** 60, 0.0)],
    [(2.0 ** 60, 2.0 ** -60), (2.0 ** 60, 2.0 ** -60)],
    [(2.0 ** -60, 2.0 ** 60), (2.0 ** -60, 2.0 ** 60), (0.0, 2.0 ** 60)],
    [(2.0 ** -60, 2.0 ** 60), (2.0 ** 60, 2.0 ** -60), (1.0, 1.0)],
    [(2.0 ** 100, 2.0 ** -90), (0.0, 2.0 ** -90), (2.0 ** -90, 2.0 ** 100)],
])
def test_blocks_of_a_head_that_differ(sizes, new):
    """Heads of 256 whose two blocks have values of unlike sizes."""
    log_case(f"attn blocks' values {sizes} new={new}")
    st = filled(sizes, "bf16", 256)
    g = torch.Generator().manual_seed(32)
    check(st, new, torch.randn((new, 4, 256), generator=g).to(torch.bfloat16).cuda(), 1 / 16)


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("dtype,big,small", [("fp16", 30000.0, 0.01), ("bf16", 2.0 ** 60, 2.0 ** -20), ("bf16", 2.0 ** 50, 2.0 ** -50)])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_large_values_without_weight(dtype, big, small, at, D, new):
    """A tile of large values whose keys weigh e^-100 or less: what the small ones come to stands."""
    log_case(f"attn large values without weight {dtype} {big} {small} at={at} D={D} new={new}")
    g = torch.Generator().manual_seed(33)
    w = torch.randn((1, D), generator=g)

    def keys(tokens, gen):
        k = 0.1 * torch.randn((len(tokens), 1, D), generator=gen)
        k[[i for i, t in enumerate(tokens) if t == big]] -= 4.0 * w
        return k

    st = filled([big if t == at else small for t in range(4)], dtype, D, keys=keys)
    q = (4.0 * w + 0.1 * torch.randn((new, 4, D), generator=g)).to(DT[dtype]).cuda()
    check(st, new, q, D ** -0.5)
