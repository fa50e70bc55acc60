"""The key/value cache's C ABI without a GPU: what the host refuses, under the sanitizers too,
the binding's own checks, and the oracle against values worked out by hand."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import kv4 as KO
from trellis_coded_bit_amd import binding as tb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_declared_functions_are_exported():
    if not os.path.exists(tb.LIB_PATH):
        from trellis_coded_bit_amd import build
        build.build(verbose=False)
    names = tb.header_functions(os.path.join(ROOT, "include", "trellis_kv4.h"))
    assert {"trellis_kv4_append", "trellis_kv4_read", "trellis_kv4_attn", "trellis_kv4_reserve", "trellis_kv4_fork",
            "trellis_kv4_compact", "trellis_kv4_free", "trellis_kv4_page_bytes"} <= set(names)
    for n in names:
        assert hasattr(tb.lib(), n), n


def test_abi_layer_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "kv4_driver")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           os.path.join(ROOT, "trellis_coded_bit_amd", "csrc", "api_kv4.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "kv4_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "failures 0" in r.stdout, r.stdout + r.stderr


def test_binding_refuses_before_the_library():
    assert tb.trellis_kv4_page_bytes(16, 8, 128) == 132 * 16 * 8
    for bad in ((8, 8, 128), (16, 0, 128), (16, 8, 96)):
        with pytest.raises(ValueError):
            tb.trellis_kv4_page_bytes(*bad)
    with pytest.raises(ValueError):  # a host tensor
        tb.KV4Cache(torch.zeros((1, 4, 132 * 16), dtype=torch.uint8), 16, 1, 128)
    with pytest.raises(TypeError):
        tb.KV4Cache(torch.zeros((1, 4, 132 * 16), dtype=torch.int8), 16, 1, 128)


def test_oracle_quantiser_by_hand():
    # one element: the rotated block is x / sqrt(128) everywhere, the largest magnitude
    x = np.zeros(128)
    x[0] = 6.0 * np.sqrt(128.0)
    codes, s = KO.quantize(x)
    assert (codes == 7).all() and KO.bf16_value(s) == 1.0
    # a rotated block given directly: H is its own inverse
    r = np.tile([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.3, 0.74, 1.26, 4.9, -6.0], 8)
    ties = KO.e2m1_values(KO.e2m1_codes(r[:16]))
    assert np.array_equal(ties, [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -4, 0.5, 0.5, 1.5, 4, -6])
    codes, s = KO.quantize(r @ KO.H)
    assert KO.bf16_value(s) == 1.0 and np.abs(KO.e2m1_values(codes) - r).max() <= 1.0 + 1e-9
    assert np.array_equal(KO.H @ KO.H, KO.H @ KO.H.T) and np.allclose(KO.H @ KO.H, np.eye(128), atol=1e-12)
    # non-finite and vanishing blocks
    bad = np.array([[1.0] * 127 + [np.nan], [1.0] * 127 + [np.inf], [1e-45] * 128])
    codes, s = KO.quantize(bad)
    assert (codes == 0).all() and s.tolist() == [0x7FC0, 0x7FC0, 0]
    # bf16: nearest, ties to even, once (not by way of float32)
    assert KO.bf16_bits(np.array([1.0, 1.00390625, 1.01171875, 1.00390625 + 1e-12])).tolist() == [0x3F80, 0x3F80, 0x3F82, 0x3F81]


def test_oracle_attention_masks_by_hand():
    k = np.zeros((5, 1, 4))
    v = np.arange(5.0).reshape(5, 1, 1) * np.ones(4)
    q = np.ones((2, 1, 4))
    y, lse, _, _ = KO.attention(q, k, v, 1.0)
    assert np.allclose(y[:, 0, 0], [1.5, 2.0]) and np.allclose(lse[:, 0], np.log([4, 5]))
    y, _, _, _ = KO.attention(q, k, v, 1.0, window=1)
    assert np.allclose(y[:, 0, 0], [3, 4])
    y, _, _, _ = KO.attention(q, k, v, 1.0, window=1, sinks=2)
    assert np.allclose(y[:, 0, 0], [(0 + 1 + 3) / 3, (0 + 1 + 4) / 3])
    y, lse, _, _ = KO.attention(np.ones((3, 1, 4)), k[:1], v[:1], 1.0)
    assert (lse[:2] == -np.inf).all() and (y[:2] == 0).all()


def test_oracle_pages_by_hand():
    c = KO.Cache(1, 6, 16, 1, 128)
    c.pool[...] = np.random.default_rng(0).integers(0, 256, c.pool.shape, np.uint8)
    p = KO.Pages(c, np.array([[5, 2, -1], [-1, -1, -1], [-1, -1, -1]], np.int32), np.array([20, 0, 0], np.int32),
                 np.array([0, 0, 1, 0, 0, 1], np.int32))
    assert p.fork([0], [1])
    assert p.table[1].tolist() == [5, 0, -1] and p.ref.tolist() == [1, 0, 1, 0, 0, 2] and p.lens.tolist() == [20, 20, 0]
    assert p.reserve([1, 2], [13, 1])  # 20 -> 33: a third page; slot 2's first
    assert p.table[1].tolist() == [5, 0, 1] and p.table[2, 0] == 3
    assert p.compact([0], [0], [[19, 3]])
    assert p.table[0, 0] == 4 and p.lens[0] == 2 and p.ref.tolist() == [1, 1, 0, 1, 1, 1]
    assert not p.reserve([0], [32]) and p.lens[0] == 2
    p.free([1])
    assert p.ref.tolist() == [0, 0, 0, 1, 1, 0]
