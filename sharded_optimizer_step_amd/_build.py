"""Build the library of the per-rank ZeRO shard step in-tree: the gfx950 HIP
kernels and the C ABI with hipcc (it cross-compiles without a GPU), the host
optimizer of the CPU-offloaded step with g++."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
# compiled side by side: each has its own kernels (no device code is shared between objects)
SOURCES = [os.path.join(CSRC, f) for f in ("zero_kernels.hip", "zero_api.cpp", "zero_act8.hip", "zero_wgrad.hip",
                                            "zero_block_norm.hip", "zero_layer_norm.hip", "zero_ffn.hip",
                                            "zero_ffn_act.hip", "zero_block_api.cpp")]
# host-only C++ (the optimizer half of the CPU-offloaded step), built by the
# host compiler into an object that the library links
HOST_SOURCES = [os.path.join(CSRC, "zero_host_adamw.cpp")]
LIB = os.path.join(PKG, "libzero_step.so")
OBJ_DIR = os.path.join(PKG, "_build")

HOST_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-pthread", "-Wall",
    # x86-64 with AVX2 (every EPYC host of an MI355X)
    "-mavx2",
    # binary64 arithmetic exactly as written: no fused multiply-adds, no
    # fast-math; sqrt without errno so that it vectorizes (still IEEE)
    "-fno-fast-math", "-ffp-contract=off", "-fno-math-errno",
]

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC", "-shared",
    # exact binary32 adds and multiplies unless an fma is written out
    "-ffp-contract=off",
    # no packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _run(cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + out)
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    obj = lambda src: os.path.join(OBJ_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    cmds = [["g++", *HOST_FLAGS, "-I", CSRC, "-c", "-o", obj(s), s] for s in HOST_SOURCES]
    cmds += [["hipcc", *compile_flags, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", "-o", obj(s), s]
             for s in SOURCES]
    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as pool:
        out = "\n".join(o for o in pool.map(_run, cmds) if o.strip())
    tmp = LIB + ".tmp"
    link = [f for f in HIPCC_FLAGS if f in ("-fPIC", "-shared") or f.startswith("--offload-arch")]
    out += _run(["hipcc", *link, "-o", tmp, *[obj(s) for s in SOURCES + HOST_SOURCES], "-lpthread"])
    if verbose and out.strip():
        print(out)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
