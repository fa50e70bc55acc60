"""The C ABI of the block-scaled FP8 operators and the routed tokens without a GPU: what the host
refuses, under the sanitizers too, the binding's own checks, and the oracle against values worked
out by hand and against differences."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import f8 as FO
from trellis_coded_bit_amd import binding as tb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header", ["trellis_f8.h", "trellis_route.h"])
def test_declared_functions_are_exported(header):
    if not os.path.exists(tb.LIB_PATH):
        from trellis_coded_bit_amd import build
        build.build(verbose=False)
    names = tb.header_functions(os.path.join(ROOT, "include", header))
    assert len(names) == 6
    for n in names:
        assert hasattr(tb.lib(), n) and (n.endswith("_bytes") or hasattr(tb, n)), n


def test_abi_layer_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "f8_driver")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(ROOT, "trellis_coded_bit_amd", "csrc", "api_f8.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "f8_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "failures 0" in r.stdout, r.stdout + r.stderr


def test_binding_refuses_before_the_library():
    e4 = torch.float8_e4m3fn
    x = torch.zeros((2, 256), dtype=torch.float16)
    for f in (lambda: tb.trellis_f8_norm(x, None, 1e-6), lambda: tb.trellis_f8_silu_mul(x),
              lambda: tb.trellis_moe_sort(torch.zeros((2, 2), dtype=torch.int32), 4),
              lambda: tb.F8Linear(torch.zeros((128, 128)).to(e4), torch.ones((1, 1)))):
        with pytest.raises(ValueError):  # host tensors
            f()
    with pytest.raises(TypeError):
        tb.trellis_f8_norm(x.float(), None, 1e-6)
    with pytest.raises(ValueError):
        tb.trellis_moe_sort(torch.zeros(4, dtype=torch.int32), 4)


@pytest.mark.parametrize("shape", [(2 ** 32 + 128, 16), (128, 2 ** 32 + 16), (2 ** 32 + 2, 128, 128), (2 ** 31, 16)])
def test_matrices_above_32_bits_are_refused(monkeypatch, shape):
    """Not cut off to the small sizes that their lower 32 bits are.  (Tensors without storage stand for
    those on a GPU.)"""
    monkeypatch.setattr(tb, "_req", lambda *args, **kw: None)
    w = torch.empty(shape, dtype=torch.float8_e4m3fn, device="meta")
    scale = torch.empty((*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128)), device="meta")
    with pytest.raises(ValueError):
        tb.F8Linear(w, scale)
    L = tb.F8Linear(w[..., :16, :16], scale[..., :1, :1]) if len(shape) == 2 else None
    assert L is None or (L._c.n_experts, L._c.in_features, L._c.out_features) == (1, 16, 16)


def test_new_outputs_are_seen_by_modes(monkeypatch):
    """New outputs are made by torch.empty where a mode or deterministic algorithms want to see them."""
    from torch.overrides import TorchFunctionMode
    from torch.utils._python_dispatch import TorchDispatchMode
    seen = []

    class Dispatch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(func)
            return func(*args, **(kwargs or {}))

    class Function(TorchFunctionMode):
        def __torch_function__(self, func, types, args=(), kwargs=None):
            seen.append(func)
            return func(*args, **(kwargs or {}))

    monkeypatch.setattr(tb, "_empty_cuda", lambda shape, stride, dtype: None)
    cpu = torch.device("cpu")
    assert tb._new1(3, torch.int32, cpu) is None and tb._new2(3, 4, torch.int32, cpu) is None
    for mode in (Dispatch, Function):
        with mode():
            t = tb._new2(3, 4, torch.float16, cpu)
        assert seen and t.shape == (3, 4) and t.dtype == torch.float16 and t.stride() == (4, 1)
        seen.clear()
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.isnan(tb._new1(5, torch.float32, cpu)).all()
    finally:
        torch.use_deterministic_algorithms(False)
    assert tb._new1(3, torch.int32, cpu) is None


def test_oracle_e4m3_by_hand():
    v = FO.E4M3
    assert v[0x7E] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0xB8] == -1.0 and np.isnan(v[0x7F])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, v, equal_nan=True)
    # midpoints go to even mantissas, the neighbours of midpoints to their own side
    pos = v[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, pos[:-1], pos[1:])
    assert np.array_equal(FO.e4m3_round(mid), even) and np.array_equal(FO.e4m3_round(-mid), -even)
    assert np.array_equal(FO.e4m3_round(mid * (1 - 1e-12)), pos[:-1]) and np.array_equal(FO.e4m3_round(mid * (1 + 1e-12)), pos[1:])
    x = np.random.default_rng(0).uniform(-448, 448, 4096).astype(np.float32)
    assert np.array_equal(FO.e4m3_round(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_oracle_quantiser_by_hand():
    x = np.zeros((1, 272))
    x[0, 5], x[0, 130], x[0, 131], x[0, 260] = 448.0, -2.0, 1.0, np.inf
    q, s = FO.quantize(x)
    assert s[0, 0] == 1.0 and s[0, 1] == 2.0 / 448 and np.isnan(s[0, 2])
    assert q[0, 5] == 448 and q[0, 130] == -448 and q[0, 131] == 224 and (q[0, 256:] == 0).all()
    q, s = FO.quantize(np.zeros((1, 16)))
    assert s[0, 0] == 0 and (q == 0).all()
    assert np.allclose(FO.norm(np.array([[3.0, 4.0]]), 0.5)[0], np.array([[3.0, 4.0]]) / np.sqrt(13.0))
    assert np.allclose(FO.silu_mul(np.array([[1.0, 0.0, 2.0, 5.0]])), [[2.0 / (1 + np.exp(-1.0)), 0.0]])


def test_oracle_product_by_hand():
    q, w = np.zeros((1, 144)), np.zeros((130, 144))
    q[0, 0], q[0, 128] = 2.0, 3.0
    w[129, 0], w[129, 128] = 5.0, 7.0
    y, mass = FO.product(q, np.array([[10.0, 100.0]]), w, np.array([[1.0, 1.0], [0.5, 0.25]]))
    assert y[0, 129] == 2 * 10 * 5 * 0.5 + 3 * 100 * 7 * 0.25 == mass[0, 129] and (y[0, :129] == 0).all()


def test_oracle_route_by_hand():
    off, order, inv, bad = FO.sort(np.array([[2, 0], [-1, 2], [2, 2]], np.int32), 3)
    assert off.tolist() == [0, 1, 1, 5] and order.tolist() == [1, 0, 3, 4, 5, -1] and not bad
    assert inv.tolist() == [[1, 0], [-1, 2], [3, 4]]
    assert FO.sort(np.array([[3]], np.int32), 3)[3]
    y = np.arange(12.0).reshape(6, 2)
    out, _ = FO.combine(y, inv, np.array([[2.0, 1.0], [9.0, 0.5], [1.0, 1.0]]))
    assert out.tolist() == [[4.0, 7.0], [2.0, 2.5], [14.0, 16.0]]


def test_oracle_gradients_are_the_differences():
    """combine is linear in y and in the weights: its differences are its gradient's products."""
    g = np.random.default_rng(1)
    ids = g.integers(-1, 3, (5, 3)).astype(np.int32)
    _, order, inv, _ = FO.sort(ids, 3)
    y, w, d = g.standard_normal((15, 7)), g.standard_normal((5, 3)), g.standard_normal((5, 7))
    d_y, d_w, _ = FO.combine_grad(d, y, inv, w)
    d_y = np.nan_to_num(d_y)
    for _ in range(4):
        ey, ew = g.standard_normal(y.shape), g.standard_normal(w.shape)
        step = (FO.combine(y + ey, inv, w)[0] - FO.combine(y - ey, inv, w)[0]) / 2
        assert np.isclose((step * d).sum(), (ey * d_y).sum())
        step = (FO.combine(y, inv, w + ew)[0] - FO.combine(y, inv, w - ew)[0]) / 2
        assert np.isclose((step * d).sum(), (ew * d_w).sum())
    # gathering is out[p] = x[order[p] // top]: its gradient sums a token's rows
    x, dxs = g.standard_normal((5, 7)), g.standard_normal((15, 7))
    live = order >= 0
    lhs = (x[order[live] // 3] * dxs[live]).sum()
    assert np.isclose(lhs, (x * FO.combine(dxs, inv)[0]).sum())


def test_tiles_of_sorted_rows(tmp_path):
    """The kernels' look at the offsets, run on the host lane by lane: also offsets that change under it
    lead to no expert and no row that is not there."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "tiles_driver")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-Wno-unknown-pragmas", "-Wno-clobbered", "-fsanitize=undefined",
           "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "sanitize", "tiles_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "failures 0" in r.stdout, r.stdout + r.stderr
