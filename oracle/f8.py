"""Oracle of the block-scaled FP8 operators and of the routed tokens, in numpy and 64 bits, from the
definitions in include/trellis_f8.h and include/trellis_route.h.  TEST INFRASTRUCTURE ONLY."""
import numpy as np

MIN_NORMAL = 2.0 ** -126


def _e4m3_table() -> np.ndarray:
    """Value of every E4M3 code: sign, four bits of exponent (bias 7), three of mantissa; 0x7F and
    0xFF are NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c >= 128, -v, v)


E4M3 = _e4m3_table()


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value, ties to the even mantissa, for |v| <= 464 (what rounds to 448 at most)."""
    a = np.abs(v)
    pos = E4M3[:127]
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    mid = (pos[lo] + pos[hi]) / 2
    code = np.where((a < mid) | ((a == mid) & (lo % 2 == 0)), lo, hi)
    return np.copysign(pos[code], v)


def blocks(n: int) -> int:
    return -(-n // 128)


def block_top(v: np.ndarray) -> np.ndarray:
    """[rows, blocks]: the largest magnitude of each block of 128 (NaN if one is not a number)."""
    rows, n = v.shape
    pad = np.zeros((rows, blocks(n) * 128))
    pad[:, :n] = np.abs(v)
    return pad.reshape(rows, -1, 128).max(-1)


def quantize(v: np.ndarray):
    """(values of the codes [rows, n], scales [rows, blocks]) of rows v."""
    top = block_top(v)
    s = top / 448.0
    bad = ~np.isfinite(s)
    s = np.where(bad, np.nan, np.where(s < MIN_NORMAL, 0.0, s))
    full = np.repeat(s, 128, 1)[:, :v.shape[1]]
    with np.errstate(all="ignore"):
        t = np.where((full > 0) & np.isfinite(v), v / full, 0.0)
    return e4m3_round(t), s


def norm(x, eps, gamma=None, residual=None):
    """(v, h): the norm's result before rounding, and x + residual."""
    h = x if residual is None else x + residual
    with np.errstate(all="ignore"):
        v = h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    return (v if gamma is None else v * gamma), h


def silu_mul(x):
    g, u = np.split(x, 2, -1)
    with np.errstate(all="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def dequantize(q, s):
    return q * np.repeat(s, 128, -1)[..., :q.shape[-1]]


def matrix(w, s):
    """[..., out, in] codes' values with scales per 128 x 128."""
    return dequantize(w, np.repeat(s, 128, -2)[..., :w.shape[-2], :])


def product(q, s, w, sw):
    """(y, sum of the terms' magnitudes) of rows by one matrix."""
    x, m = dequantize(q, s), matrix(w, sw)
    return x @ m.T, np.abs(x) @ np.abs(m).T


def sort(ids, n_experts):
    """(offsets, order, inverse, whether an id is out of range)."""
    flat = ids.reshape(-1)
    lists = [[] for _ in range(n_experts)]
    bad = False
    for entry, e in enumerate(flat.tolist()):
        if 0 <= e < n_experts:
            lists[e].append(entry)
        elif e != -1:
            bad = True
    order = [entry for entries in lists for entry in entries]
    inverse = np.full(flat.size, -1, np.int32)
    inverse[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    return offsets, np.array(order + [-1] * (flat.size - len(order)), np.int32), inverse.reshape(ids.shape), bad


def combine(y, inverse, weights=None, add=None):
    """(out, sum of the terms' magnitudes); positions that are no row's add nothing."""
    tokens, top = inverse.shape
    out = np.zeros((tokens, y.shape[1])) if add is None else add.copy()
    mass = np.abs(out)
    for t in range(tokens):
        for j in range(top):
            p = inverse[t, j]
            if 0 <= p < y.shape[0]:
                w = 1.0 if weights is None else weights[t, j]
                out[t] += w * y[p]
                mass[t] += np.abs(w * y[p])
    return out, mass


def combine_grad(d_out, y, inverse, weights=None):
    """(d_y with NaN in rows that no entry names, d_weights, sums of magnitudes of d_weights)."""
    tokens, top = inverse.shape
    d_y = np.full(y.shape, np.nan)
    d_w, mass = np.zeros((tokens, top)), np.zeros((tokens, top))
    for t in range(tokens):
        for j in range(top):
            p = inverse[t, j]
            if 0 <= p < y.shape[0]:
                d_y[p] = (1.0 if weights is None else weights[t, j]) * d_out[t]
                d_w[t, j] = d_out[t] @ y[p]
                mass[t, j] = np.abs(d_out[t]) @ np.abs(y[p])
    return d_y, d_w, mass
