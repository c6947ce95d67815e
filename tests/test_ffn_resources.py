"""Register, scratch and LDS figures of the layer norm's and the feed-forward
block's kernels, from the compiler's remarks on a device-only build with the
library's own flags (no GPU needed), and what their assembly has to hold to:
the matrix instructions of the products stand in inline assembly, so that
nobody but this test sees to what the hardware does not wait for by itself."""
import os
import re
import shutil
import subprocess

import pytest

from sharded_optimizer_step_amd import _build

SOURCES = ("zero_layer_norm.hip", "zero_ffn.hip", "zero_ffn_act.hip")


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    """{source: assembly}, {kernel: figures}"""
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not found")
    texts, usage = {}, {}
    flags = [f for f in _build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    for src in SOURCES:
        asm = tmp_path_factory.mktemp("asm") / "k.s"
        cmd = ["hipcc", *flags, "--cuda-device-only", "-S", "-o", str(asm), "-I", os.path.join(_build.ROOT, "include"), "-I",
               _build.CSRC, os.path.join(_build.CSRC, src), "-Rpass-analysis=kernel-resource-usage"]
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        texts[src], cur = asm.read_text(), None
        for line in r.stderr.splitlines():
            m = re.search(r"remark: .*Function Name: (\S+)|remark: Function Name: (\S+)", line)
            if m:
                cur = usage.setdefault(m.group(1) or m.group(2), {"source": src})
                continue
            m = re.search(r"remark:\s+([A-Za-z ]+?)(?: \[[^\]]*\])?: (\S+) \[-Rpass", line)
            if m and cur is not None:
                cur[m.group(1).strip()] = m.group(2)
    return texts, usage


def test_no_kernel_spills_or_packs(built):
    texts, usage = built
    assert len(usage) >= 50
    for name, u in usage.items():
        assert u["ScratchSize"] == "0" and u["VGPRs Spill"] == "0", (name, u)
    for src, text in texts.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", text), src


def test_tiles_leave_room_for_their_workgroups(built):
    seen = 0
    for name, u in built[1].items():
        m = re.search(r"10ffn_kernelINS0_4TileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name)
        if m is None:
            continue
        seen += 1
        slots, waves = int(m.group(6)), int(m.group(3)) * int(m.group(4))
        assert slots * int(u["LDS Size"]) <= 160 * 1024, (name, u)
        assert int(u["Occupancy"]) * 4 >= slots * waves, (name, u)
    assert seen == 13  # five tiles forward and for dh, three for the weight gradients


def test_norms_keep_the_waves_their_split_counts_on(built):
    for name, u in built[1].items():
        if "layer_norm_kernel" in name or "layer_norm_grad_kernel" in name:
            assert int(u["Occupancy"]) >= 4, (name, u)


def registers(operand):
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.fullmatch(r"([va])(\d+)", operand)
    return {(m.group(1), int(m.group(2)))} if m else set()


def instructions(text):
    for line in text.splitlines():
        s = line.split(";")[0].strip()
        if s and not s.startswith(".") and not s.endswith(":"):
            op, *rest = s.split(None, 1)
            yield op, re.split(r",\s*", rest[0]) if rest else []


def test_operands_of_products_are_not_written_just_before(built):
    """A matrix instruction that reads what a vector instruction wrote needs two instructions between them."""
    products, before = 0, []
    for op, args in instructions(built[0]["zero_ffn.hip"]):
        if op.startswith("v_mfma"):
            products += 1
            read = set().union(*(registers(a) for a in args[1:4]))
            for o, written in before[-2:]:
                if o.startswith("v_") and not o.startswith("v_mfma"):
                    assert not registers(written[0]) & read, (o, written, args)
            assert args[0] == args[3], args  # in place
        before = before[-2:] + [(op, args)]
    assert products > 1000


def test_sums_are_read_long_after_the_last_product(built):
    """A sum is read by something else than a product 18 instructions (or waits of as many) after its last one at the
    earliest. (Other registers of its kind may hold what has no room elsewhere.)"""
    now, written, reads = 0, {}, 0
    for op, args in instructions(built[0]["zero_ffn.hip"]):
        now += int(args[0]) + 1 if op == "s_nop" else 1
        if op.startswith("v_mfma"):
            written.update({r: now for r in registers(args[0])})
            continue
        writes = op.startswith("v_") or op.startswith("ds_read")
        for arg in args[1:] if writes else args:
            for r in registers(arg) & written.keys():
                reads += 1
                assert now - written[r] >= 18, (op, args)
        for r in registers(args[0]) & written.keys() if writes and args else ():
            assert now - written[r] >= 18, (op, args)
            del written[r]
        if op == "s_endpgm":
            written = {}
    assert reads > 100


def test_loads_to_lds_follow_their_address(built):
    """The register that says where in LDS a load goes is written by the instruction pair just before it, and by nothing else."""
    last = []
    loads = 0
    for op, args in instructions(built[0]["zero_ffn.hip"]):
        if op == "buffer_load_dwordx4" and args[-1].split()[-1] == "lds":
            loads += 1
            assert last[-2][0] == "s_add_u32" and last[-2][1][0] == "m0" and last[-1][0] == "s_nop", (last, args)
        elif "m0" in args:
            assert op == "s_add_u32", (op, args)
        last = last[-1:] + [(op, args)]
    assert loads > 100
