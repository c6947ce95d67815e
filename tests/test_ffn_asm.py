"""What the inline assembly of the feed-forward products says that it changes,
from the compiler's intermediate form of a device-only build (no GPU needed):
the compiler may hold a value across it in every register that it does not name."""
import os
import re
import shutil
import subprocess

import pytest

from sharded_optimizer_step_amd import _build


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """[(text, constraints)] of every piece of inline assembly in zero_ffn.hip"""
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not found")
    out = tmp_path_factory.mktemp("ir") / "k.ll"
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    r = subprocess.run(["hipcc", *flags, "--cuda-device-only", "-S", "-emit-llvm", "-o", str(out), "-I", os.path.join(_build.ROOT, "include"),
                        "-I", _build.CSRC, os.path.join(_build.CSRC, "zero_ffn.hip")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    found = re.findall(r' asm (?:sideeffect )?"([^"]*)", "([^"]*)"', out.read_text())
    assert len(found) > 1000
    return found


def test_assembly_that_writes_scalar_registers_names_them(assembly):
    seen = 0
    for text, constraints in assembly:
        named = set(re.findall(r"~\{(\w+)\}", constraints))
        for op, to in re.findall(r"(?:^|\\0A|\\09)\s*(s_\w+) (\w+)", text):
            if op in ("s_nop", "s_waitcnt"):
                continue
            seen += 1
            assert to in named, (text, constraints)
            if op.startswith("s_add"):
                assert "scc" in named, (text, constraints)
    assert seen > 100


def test_assembly_that_loads_names_memory(assembly):
    for text, constraints in assembly:
        if "buffer_load" in text or "s_waitcnt" in text:
            assert "~{memory}" in constraints, (text, constraints)
