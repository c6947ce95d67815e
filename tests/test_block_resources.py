"""Register, scratch, LDS and occupancy figures of the kernels around a
training block, from the compiler's remarks on a device-only build with the
library's own flags (no GPU needed). No kernel may spill, none may contain a
packed fp32 instruction, and those whose speed rests on how many of their
waves run at once keep that number."""
import os
import re
import shutil
import subprocess

import pytest

from sharded_optimizer_step_amd import _build

SOURCES = ("zero_act8.hip", "zero_wgrad.hip", "zero_block_norm.hip")


@pytest.fixture(scope="module")
def usage(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not found")
    out = {}
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    for src in SOURCES:
        asm = tmp_path_factory.mktemp("asm") / "k.s"
        cmd = ["hipcc", *flags, "--cuda-device-only", "-S", "-o", str(asm), "-I", os.path.join(_build.ROOT, "include"), "-I",
               _build.CSRC, os.path.join(_build.CSRC, src), "-Rpass-analysis=kernel-resource-usage"]
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        text = asm.read_text()
        assert not re.search(r"v_pk_(add|mul|fma)_f32", text), src
        cur = None
        for line in r.stderr.splitlines():
            m = re.search(r"remark: .*Function Name: (\S+)|remark: Function Name: (\S+)", line)
            if m:
                cur = out.setdefault(m.group(1) or m.group(2), {"source": src})
                continue
            m = re.search(r"remark:\s+([A-Za-z ]+?)(?: \[[^\]]*\])?: (\S+) \[-Rpass", line)
            if m and cur is not None:
                cur[m.group(1).strip()] = m.group(2)
    return out


def test_no_kernel_spills(usage):
    assert len(usage) >= 50
    for name, u in usage.items():
        assert u["ScratchSize"] == "0" and u["VGPRs Spill"] == "0", (name, u)


def test_weight_gradient_tiles_leave_room_for_their_workgroups(usage):
    seen = 0
    for name, u in usage.items():
        m = re.search(r"4TileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name)
        if m is None:
            continue
        seen += 1
        bm, bn, bk, wm, wn, slots = map(int, m.groups())
        lds = int(u["LDS Size"])
        assert slots * lds <= 160 * 1024, (name, u)
        assert int(u["Occupancy"]) * 4 >= slots * wm * wn, (name, u)  # waves a compute unit
    assert seen == 6  # three tiles, two formats


def test_norms_keep_the_waves_their_split_counts_on(usage):
    # 16 waves a compute unit forwards (every row width) and for narrow coded rows backwards
    for name, u in usage.items():
        if "block_norm_kernel" in name:
            assert int(u["Occupancy"]) >= 4, (name, u)
        m = re.search(r"block_norm_grad_kernelILb(\d)ELi(\d+)ELb(\d)ELb(\d)ELb(\d)ELb(\d)E", name)
        if m:
            assert int(u["Occupancy"]) * 4 >= int(m.group(2)) // 64, (name, u)  # its largest workgroup starts


def test_norm_gradients_run_the_waves_that_their_split_is_measured_with(usage):
    # 12 waves a compute unit (168 registers); 8 of some kernels for rows as they are with many gate rows; the kernels of
    # 16-wave workgroups need 16
    seen = 0
    for name, u in usage.items():
        m = re.search(r"block_norm_grad_kernelILb(\d)ELi(\d+)ELb(\d)ELb(\d)ELb(\d)ELb(\d)E", name)
        if m is None:
            continue
        seen += 1
        most, coded, many = int(m.group(2)), m.group(4) == "1", m.group(5) == "1"
        waves = 4 * int(u["Occupancy"])
        assert waves >= (16 if most == 1024 else 8 if many and not coded else 12), (name, u)
    assert seen == 34  # as grad_shape and grad_split make them
