"""A workspace that serves a step and a call around a training block in turn, on
the CPU: the library's host side (zero_api.cpp, zero_block_api.cpp) built over
stub launches that write host memory where the kernels write the workspace. A
step whose table was overwritten has to upload it again; taking the sums for
its table, the kernels would follow them as pointers."""
import os
import subprocess

import pytest

from sharded_optimizer_step_amd import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    exe = tmp_path_factory.mktemp("host") / "host"
    src = [os.path.join(_build.CSRC, f) for f in ("zero_api.cpp", "zero_block_api.cpp", "zero_host_adamw.cpp")]
    # what these calls do not reach of HIP and of the kernels stays unresolved
    cmd = ["g++", "-O1", "-std=c++17", "-w", "-pthread", "-mavx2", "-ffp-contract=off", "-D__HIP_PLATFORM_AMD__", "-no-pie",
           "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, "-I", "/opt/rocm/include", "-o", str(exe),
           os.path.join(HERE, "block_workspace_host.cpp"), *src, "-Wl,--unresolved-symbols=ignore-all"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def run(*args):
        r = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, (args, r.returncode, r.stderr)
        return list(map(int, r.stdout.split()))

    return run


CALLS = [("wgrad", "-", 0, 0), ("check", "-", 0, 0)]
CALLS += [("norm_grad", which, cols, gate_rows) for which in ("-", "p", "o", "g", "og", "po", "pog")
          for cols, gate_rows in ((256, 0), (256, 1), (256, 8), (8192, 0), (8192, 1), (8192, 8)) if not ("g" in which and gate_rows == 0)]


@pytest.mark.parametrize("what,which,cols,gate_rows", CALLS)
@pytest.mark.parametrize("offset", [0, 256])
def test_a_step_after_a_call_on_its_workspace_uploads_its_table(host, what, which, cols, gate_rows, offset):
    first, again, after, plan, table, _, _ = host(what, which, cols, gate_rows, offset)
    assert first > 0 and again == 0
    assert after == first and plan and table


@pytest.mark.parametrize("what,which,cols,gate_rows", CALLS)
def test_a_call_that_overwrites_a_table_overwrites_its_signature(host, what, which, cols, gate_rows):
    # a step that does not pass the host record (its launches were captured earlier) sees the signature alone
    signature, table = host(what, which, cols, gate_rows, 0)[5:]
    assert table or not signature


def test_a_step_keeps_its_table_beside_a_call_on_another_workspace(host):
    for what, which, cols, gate_rows in CALLS:
        first, again, after, plan, table, _, _ = host(what, which, cols, gate_rows, 8 << 20)
        assert (first > 0, again, after, plan, table) == (True, 0, 0, 1, 1), (what, which)
