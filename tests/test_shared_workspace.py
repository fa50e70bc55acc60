"""One workspace under several host threads: every call's launches reach the stream together, so what
a call's first launch leaves in the scratch is there for its next.  On the CPU the C-ABI layer itself,
against launchers that note who else is in one; on the GPU the calls of two launches and more."""
import os
import shutil
import subprocess
import threading
import time

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


def _host_workspaces(monkeypatch):
    for name in ("_ws", "_ws_outgrown", "_ws_held"):
        monkeypatch.setattr(tb, name, {}, raising=False)
    monkeypatch.setattr(tb, "_stream", lambda: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return torch.device("cpu", 0)


def test_errors_of_a_call_whose_workspace_is_outgrown_meanwhile(monkeypatch):
    """A thread looks its workspace up, another one's call replaces it, then the first one's kernel
    sets its error word: it is known, until it is cleared, and the buffer does not stay for good."""
    cpu = _host_workspaces(monkeypatch)
    a = tb.workspace(1000, cpu)
    b = tb.workspace(2000, cpu)
    a[:4].view(torch.int32)[0] = 8
    assert b is not a and tb.error_word() == 8
    del a
    c = tb.workspace(3000, cpu)  # (b is held now)
    assert tb.error_word() == 8 and int(c[:4].view(torch.int32)) == 8 and sum(map(len, tb._ws_held.values())) == 1
    b[:4].view(torch.int32)[0] = 1
    del b, c
    d = tb.workspace(4000, cpu)
    assert tb.error_word() == 9 and int(d[:4].view(torch.int32)) == 9 and not tb._ws_held
    tb.clear_error_word()
    assert tb.error_word() == 0


@pytest.mark.parametrize("first", [0, 500])
def test_threads_that_need_a_workspace_at_once_get_the_same(monkeypatch, first):
    cpu = _host_workspaces(monkeypatch)
    if first:
        tb.workspace(first, cpu)
    zeros, got, start = torch.zeros, [], threading.Barrier(4)

    def slow(*args, **kw):
        w = zeros(*args, **kw)
        time.sleep(0.05)
        return w

    monkeypatch.setattr(torch, "zeros", slow)

    def call():
        start.wait()
        got.append(tb.workspace(1000, cpu))

    threads = [threading.Thread(target=call) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4 and all(w is got[0] for w in got)
    got[2][:4].view(torch.int32)[0] = 1
    assert tb.error_word() == 1


def _in_threads(calls, want, rounds):
    """Every call from a thread of its own, all on the default stream: (call, wrong results or error)."""
    errors, start = [], threading.Barrier(len(calls))

    def loop(i):
        try:
            start.wait()
            got = [calls[i]() for _ in range(rounds)]
            torch.cuda.synchronize()
            wrong = sum(not all(torch.equal(a, b) for a, b in zip(r, want[i])) for r in got)
            if wrong:
                errors.append((i, wrong))
        except Exception as e:  # noqa: BLE001
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


@pytest.mark.gpu
def test_threads_on_one_stream():
    """Four threads on the default stream with its one workspace: products whose blocks are shared
    among workgroups and sorts of three launches, of different sizes."""
    from gpu_util import log_case
    from test_gpu_f8 import make_matrix, make_rows
    from test_gpu_route import routing
    log_case("threads on one stream")
    g = torch.Generator().manual_seed(0)
    calls = []
    for i, (m, n, k) in enumerate(((70, 4099, 6160), (130, 1544, 16400), (200, 2051, 8208), (70, 2050, 16400))):
        L = make_matrix(n, k, g)
        q, s = make_rows(m, k, g)
        assert tb.trellis_f8_workspace_bytes(L, m) > tb.trellis_f8_workspace_bytes(L, 1)
        ids = routing(9000 + 1000 * i, 8, 40 + i, g, 0.9)
        calls.append(lambda L=L, q=q, s=s, ids=ids, e=40 + i: (tb.trellis_f8_gemm(L, q, s), *tb.trellis_moe_sort(ids, e)))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    assert not _in_threads(calls, want, 50) and tb.error_word() == 0


@pytest.mark.gpu
def test_threads_at_one_kernel_with_more_and_less_shared_memory():
    """Each launch has what it needs, whatever another thread's call of the same kernel asked for."""
    from gpu_util import log_case
    from test_gpu_f8 import make_matrix, make_rows
    log_case("threads at one kernel")
    g = torch.Generator().manual_seed(1)
    calls = []
    for experts in (1700, 2048):
        ids = torch.randint(-1, experts, (500, 4), generator=g, dtype=torch.int32).cuda()
        calls.append(lambda ids=ids, e=experts: tb.trellis_moe_sort(ids, e))
    for n in (4096, 32768):  # (128 and 1024 tiles of 32 rows: eight waves, four)
        L = make_matrix(n, 1024, g)
        q, s = make_rows(3, 1024, g)
        calls.append(lambda L=L, q=q, s=s: (tb.trellis_f8_gemm(L, q, s),))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    assert not _in_threads(calls, want, 200) and tb.error_word() == 0
