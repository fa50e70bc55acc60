"""One workspace under several host threads: every call's launches reach the stream together, so what
a call's first launch leaves in the scratch is there for its next.  On the CPU the C-ABI layer itself,
against launchers that note who else is in one; on the GPU the calls of two launches and more."""
import os
import shutil
import subprocess
import threading

import pytest
import torch

from trellis_coded_bit_amd import binding as tb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_with_one_workspace_take_turns(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "turns_driver")
    csrc = os.path.join(ROOT, "trellis_coded_bit_amd", "csrc")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-pthread", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           *(os.path.join(csrc, f) for f in ("api.cpp", "api_kv4.cpp", "api_f8.cpp")),
           os.path.join(ROOT, "tests", "sanitize", "turns_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.gpu
def test_threads_on_one_stream():
    """Four threads on the default stream with its one workspace: products whose blocks are shared
    among workgroups and sorts of three launches, of different sizes."""
    from gpu_util import log_case
    from test_gpu_f8 import make_matrix, make_rows
    from test_gpu_route import routing
    log_case("threads on one stream")
    g = torch.Generator().manual_seed(0)
    work = []
    for i, (m, n, k) in enumerate(((70, 4099, 6160), (130, 1544, 16400), (200, 2051, 8208), (70, 2050, 16400))):
        L = make_matrix(n, k, g)
        q, s = make_rows(m, k, g)
        assert tb.trellis_f8_workspace_bytes(L, m) > tb.trellis_f8_workspace_bytes(L, 1)
        work.append((L, q, s, routing(9000 + 1000 * i, 8, 40 + i, g, 0.9), 40 + i))
    run = lambda w: (tb.trellis_f8_gemm(*w[:3]), *tb.trellis_moe_sort(w[3], w[4]))  # noqa: E731
    want = [run(w) for w in work]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(work))

    def loop(i):
        try:
            start.wait()
            got = [run(work[i]) for _ in range(50)]
            torch.cuda.synchronize()
            wrong = sum(not all(torch.equal(a, b) for a, b in zip(r, want[i])) for r in got)
            if wrong:
                errors.append((i, wrong))
        except Exception as e:  # noqa: BLE001
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and tb.error_word() == 0
