"""Attention over the 4-bit cache against the oracle within the bounds of its formats (kv4_bounds): few
keys, where a weight's last part shows; the logarithm's error, where a query's does; and as many columns
as the kernels for few and for many divide at, and one less and more: 48 in a call of several sequences,
128 in a call of one."""
import numpy as np
import pytest
import torch

import kv4_bounds as B
from oracle import kv4 as KO
from trellis_coded_bit_amd import binding as tb

from gpu_util import log_case
from test_gpu_kv4 import DT, Setup, host, ints

pytestmark = pytest.mark.gpu


def rotated(x):
    return (B.blocks(x) @ KO.H).reshape(x.shape)


def attend(st, new, heads, few, max_q, seed):
    """The last new[b] tokens of each sequence b; every row, and the whole, within the bounds."""
    g = torch.Generator().manual_seed(seed)
    rows, scale = sum(new), st.D ** -0.5
    q = (1.5 * torch.randn((rows, heads, st.D), generator=g)).to(DT[st.dtype]).cuda()
    lse = torch.empty((rows, heads), device="cuda")
    y = tb.trellis_kv4_attn(st.cache, st.layer, st.table, st.lens, ints(np.concatenate([[0], np.cumsum(new)])), q, lse=lse,
                            max_q=max_q)
    torch.cuda.synchronize()
    assert tb.error_word() == 0
    oc, table = st.oracle(), st.table.cpu().numpy()
    got, logs, qr = host(y), host(lse), rotated(host(q))
    refs, diffs, log_err, log_rms, at = [], [], [], [], 0
    group = heads // st.Hk
    weight = B.WEIGHT_FEW if few else B.WEIGHT_MANY
    for b, n in enumerate(new):
        length = st.host_lens[b]
        k, v = (rotated(oc.rows(st.layer, table[b], length, w)) for w in (0, 1))
        for i in range(n):
            seen = length - n + i + 1
            for h in range(st.Hk):
                x = qr[at + i, h * group:(h + 1) * group]
                s = scale * (x @ k[:seen, h].T)
                top = s.max(-1, keepdims=True)
                e = np.exp(s - top)
                p = e / e.sum(-1, keepdims=True)
                ref = rotated(p @ v[:seen, h])
                y1 = got[at + i, h * group:(h + 1) * group]
                most = B.score_most(x, k[:seen, h], scale)
                bound = (weight + 2 * most + B.SUMS) * (p @ np.linalg.norm(v[:seen, h], axis=-1)) + \
                    B.UNIT[st.dtype] * np.linalg.norm(ref, axis=-1) + 1e-6
                assert (np.linalg.norm(y1 - ref, axis=-1) <= bound).all(), (b, i, h)
                err = logs[at + i, h * group:(h + 1) * group] - (top[:, 0] + np.log(e.sum(-1)))
                assert (np.abs(err) <= most + 2.0 ** -18 * (1 + np.abs(s).max())).all(), (b, i, h)
                refs.append(ref)
                diffs.append(y1 - ref)
                log_err.append(err)
                log_rms.append(B.score_rms(x, k[:seen, h], scale) + 2.0 ** -21 * (1 + np.abs(s).max()))
        at += n
    ratio = np.linalg.norm(np.concatenate(diffs)) / np.linalg.norm(np.concatenate(refs))
    print(f"relative L2 {ratio:.2e} of {B.rel(st.dtype, few):.2e}; logarithm {B.rms(np.concatenate(log_err)):.2e} of "
          f"{B.rms(np.concatenate(log_rms)):.2e}")
    assert ratio <= B.rel(st.dtype, few)
    assert B.rms(np.concatenate(log_err)) <= B.rms(np.concatenate(log_rms))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("group,new", [(1, 1), (4, 1), (4, 2), (16, 1), (12, 3)])
def test_few_keys(D, group, new):
    """Single and drafted tokens over up to seven keys: columns held four times, twice and once."""
    log_case(f"attn few keys D={D} group={group} new={new}")
    st = Setup([new + b % 6 for b in range(48)], T=16, Hk=4, D=D, seed=50)
    attend(st, [new] * 48, 4 * group, True, new, 51)


@pytest.mark.parametrize("D", [128, 256])
def test_few_keys_many_rows(D):
    """Prompts whose first rows see few keys."""
    log_case(f"attn few keys, many rows D={D}")
    st = Setup([30] * 12, T=16, Hk=4, D=D, seed=52)
    attend(st, [30] * 12, 32, False, 30, 53)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("group,new", [(1, [47, 48, 49]), (4, [12, 13, 11]), (16, [4, 3, 1]), (3, [16, 17, 1])])
def test_columns_where_the_kernels_divide(group, new, known, D, dtype):
    log_case(f"attn at the bound {dtype} D={D} group={group} new={new} known={known}")
    st = Setup([n + 100 * b + 7 for b, n in enumerate(new)], T=32, Hk=2, D=D, dtype=dtype, seed=54)
    attend(st, new, 2 * group, False, max(new) if known else 0, 55)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("group,new", [(1, 127), (1, 128), (1, 129), (4, 32), (4, 33), (64, 2), (64, 3)])
def test_columns_where_the_kernels_divide_one_sequence(group, new, D, dtype):
    log_case(f"attn at the bound, one sequence {dtype} D={D} group={group} new={new}")
    st = Setup([new + 150], T=64, Hk=1, D=D, dtype=dtype, seed=56)
    attend(st, [new], group, group * new <= 128, new, 57)
