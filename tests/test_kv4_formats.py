"""What the attention kernels' number formats hold, worked out on the CPU: the parts that a query element
and a weight are split into, how far the last one leaves them, and that the tolerances of
test_gpu_kv4_precision would not let a lost part pass."""
import numpy as np
import pytest

import kv4_bounds as B
from oracle import kv4 as KO


def rounded(x, mantissa, lowest, largest):
    """Nearest number (ties to even) with `mantissa` bits after the point, steps no finer than
    2^(lowest - mantissa), saturating."""
    x = np.asarray(x, np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))), lowest)
    step = np.exp2(e - mantissa)
    return np.clip(np.round(x / step) * step, -largest, largest)


def e2m3(x):
    return rounded(x, 3, 0, 7.5)


def e4m3(x):
    return rounded(x, 3, -6, 448.0)


def query_parts(q, n):
    """A rotated block as n E2M3 parts: the largest magnitude comes to [3.75, 7.5), the next parts' units
    are 16 and 512 times smaller."""
    top = np.abs(q).max(-1, keepdims=True)
    unit = np.exp2(np.floor(np.log2(top / 3.75)))
    left, total = np.array(q, np.float64), np.zeros_like(q)
    for down in (1, 16, 512)[:n]:
        part = e2m3(left * down / unit) * unit / down
        total += part
        left -= part
    return total


def weight_parts(w, n):
    """Weights of at most 256 as n E4M3 parts, each brought up 32 times more than the last."""
    left, total = np.array(w, np.float64), np.zeros_like(w)
    for up in (1, 32, 1024)[:n]:
        part = e4m3(left * up) / up
        total += part
        left -= part
    return total


def test_parts_hold_what_the_bounds_say():
    g = np.random.default_rng(0)
    q = g.standard_normal((4000, 128)) * np.exp2(g.uniform(-20, 20, (4000, 1)))
    top = np.abs(q).max(-1, keepdims=True)
    assert (np.abs(query_parts(q, 3) - q) / top).max() <= B.QUERY
    assert (np.abs(query_parts(q, 2) - q) / top).max() > 16 * B.QUERY
    w = 256 * np.exp2(-g.uniform(0, 14, 200000))
    assert (np.abs(weight_parts(w, 3) - w) / w).max() <= B.WEIGHT_FEW
    assert (np.abs(weight_parts(w, 2) - w) / w).max() > 8 * B.WEIGHT_FEW
    # below 2^-14 of the largest the third part's step takes over: 2^-27 of the largest at most
    w = 256 * np.exp2(-g.uniform(14, 40, 200000))
    assert np.abs(weight_parts(w, 3) - w).max() <= 2.0 ** -28 * 256
    w = 256 * np.exp2(-g.uniform(-7, 20, 200000))
    assert (np.abs(w.astype(np.float16).astype(np.float64) - w) / w).max() <= B.WEIGHT_MANY


@pytest.mark.parametrize("q_parts,w_parts,holds", [(3, 3, True), (3, 2, False), (2, 3, False)])
def test_bounds_tell_a_lost_part(q_parts, w_parts, holds):
    """Attention over a few keys with the parts as the kernels have them, or one less: the bounds of a
    tensor hold, or do not."""
    g = np.random.default_rng(1)
    n, heads, length = 200, 4, 5
    got, ref, lse_err, lse_bound = [], [], [], []
    for _ in range(n):
        k, v = ((KO.e2m1_values(c) * KO.bf16_value(s)[..., None]) for c, s in
                (KO.quantize(g.standard_normal((length, 128))) for _ in range(2)))  # rotated, as stored
        q = 1.5 * g.standard_normal((heads, 128))
        scale = 128 ** -0.5
        s, t = scale * (q @ k.T), scale * (query_parts(q, q_parts) @ k.T)
        p, r = np.exp(s - s.max(-1, keepdims=True)), np.exp(t - t.max(-1, keepdims=True))
        ref.append(p @ v / p.sum(-1, keepdims=True))
        # (a tile's largest value scale is brought to [128, 256): here to 255, a number of many bits)
        size = np.abs(v).max(-1)
        w = r * size * (255 / size.max())
        got.append(weight_parts(w, w_parts) @ (v / size[:, None]) * size.max() / 255 / r.sum(-1, keepdims=True))
        lse_err.append(np.log(r.sum(-1)) + t.max(-1) - np.log(p.sum(-1)) - s.max(-1))
        lse_bound.append(B.score_rms(q, k, scale))
    got, ref = np.concatenate(got).astype(np.float16).astype(np.float64), np.concatenate(ref)
    ok = np.linalg.norm(got - ref) <= B.rel("fp16", few=True) * np.linalg.norm(ref)
    ok &= B.rms(np.concatenate(lse_err)) <= B.rms(np.concatenate(lse_bound))
    assert bool(ok) == holds
