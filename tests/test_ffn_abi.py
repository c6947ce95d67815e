"""The layer norm and the gated feed-forward block on the CPU: their structures'
layouts, the sizes that they report, and every refusal, before anything touches
a GPU. No call here launches a kernel."""
import ctypes
import os
import subprocess

import pytest
import torch

import sharded_optimizer_step_amd as z

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, SMALL, OK = 1, 2, 0
BF16, F32 = 1, 2
STRUCTS = {"zero_layer_norm_args": z._CLayerNorm, "zero_layer_norm_grad_args": z._CLayerNormGrad,
           "zero_block_ffn_args": z._CBlockFfn, "zero_block_ffn_grad_args": z._CBlockFfnGrad}


def rows(data=4096, ld=64, dtype=BF16, reserved=0):
    return z._CRows(data, ld, dtype, reserved)


NONE, FP32 = rows(data=None), rows(dtype=F32)


def at(n, **kw):
    """A valid operand of its own address."""
    return rows(data=(n + 1) << 20, **kw)


def test_struct_layouts_and_constants(tmp_path):
    consts = {"ZERO_FFN_SILU": z.FFN_SILU, "ZERO_FFN_GELU": z.FFN_GELU, "ZERO_FFN_GELU_TANH": z.FFN_GELU_TANH}
    body = [f'printf("{n} %zu\\n", sizeof({n}));' for n in STRUCTS]
    body += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for n, c in STRUCTS.items() for f, _ in c._fields_]
    body += [f'printf("{n} %zu\\n", (size_t){n});' for n in consts]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zero_step.h"\nint main(void){' + "".join(body) + "return 0;}\n")
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", "-o", str(exe),
                    str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for n, c in STRUCTS.items():
        assert int(got[n]) == ctypes.sizeof(c)
        for f, _ in c._fields_:
            assert int(got[f"{n}.{f}"]) == getattr(c, f).offset, (n, f)
    for n, v in consts.items():
        assert int(got[n]) == v, n


@pytest.mark.parametrize("packed,c", [(z._LAYER_NORM, z._CLayerNorm), (z._LAYER_NORM_GRAD, z._CLayerNormGrad),
                                      (z._BLOCK_FFN, z._CBlockFfn), (z._BLOCK_FFN_GRAD, z._CBlockFfnGrad)])
def test_packed_structures_are_the_c_ones(packed, c):
    assert packed.size == ctypes.sizeof(c)
    flat = []

    def walk(cls, start):
        for f, t in cls._fields_:
            o = start + getattr(cls, f).offset
            walk(t, o) if issubclass(t, ctypes.Structure) else flat.append((o, t))

    walk(c, 0)
    values = [float(i) if t is ctypes.c_double else i for i, (_, t) in enumerate(flat)]
    image = packed.pack(*values)
    for (o, t), v in zip(flat, values):
        assert (t.from_buffer_copy(image, o).value or 0) == v, (c, o)


def call(name, struct, base, ws=None, **kw):
    c = struct()
    for k, v in {**base, **kw}.items():
        setattr(c, k, v)
    return getattr(z.lib(), name)(ctypes.byref(c), *(() if ws is None else ws), None)


NORM = dict(rows=8, cols=64, eps=1e-5, x=at(0), h=at(1))


def norm(**kw):
    return call("zero_layer_norm", z._CLayerNorm, NORM, **kw)


def test_layer_norm_refusals():
    nan, inf = float("nan"), float("inf")
    add = dict(y=at(2), x_out=at(3))
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(cols=-1), dict(cols=z.BLOCK_NORM_MAX_COLS + 1), dict(reserved=1), dict(eps=-1e-9),
               dict(eps=nan), dict(eps=inf), dict(eps=1e39), dict(x=NONE), dict(x=rows(ld=63)), dict(x=rows(dtype=5)),
               dict(x=rows(data=4097)), dict(x=rows(reserved=1)), dict(h=NONE), dict(h=FP32), dict(h=rows(ld=1)), dict(x_out=at(3)),
               dict(add, x_out=NONE), dict(add, x_out=at(3, dtype=F32)), dict(add, y=at(2, dtype=F32)), dict(add, y=at(2, ld=9)),
               dict(w=rows(dtype=0)), dict(b=rows(data=4099, dtype=F32)), dict(mean=4097), dict(rstd=4098), dict(ckpt_xn=4096, format=0),
               dict(ckpt_h=4096, format=3), dict(ckpt_xn=4104, format=1), dict(ckpt_h=4104, format=2)):
        assert norm(**kw) == BAD, kw
    full = dict(add, mean=1 << 16, rstd=1 << 17, ckpt_xn=1 << 18, ckpt_h=1 << 19, format=1)
    for kw in (dict(h=full["x_out"]), dict(rstd=1 << 16), dict(ckpt_h=1 << 18), dict(mean=1 << 18)):
        assert norm(**{**full, **kw}) == BAD, kw
    assert z.lib().zero_layer_norm(None, None) == BAD
    assert norm(rows=0, x=NONE, h=NONE) == OK and norm(cols=0) == OK


NGRAD = dict(rows=8, cols=64, dh=at(0), x_out=at(1), mean=4096, rstd=8192, dx=at(2), dw=at(3), db=at(4))


def norm_grad(ws=4096, wsb=1 << 40, **kw):
    return call("zero_layer_norm_grad", z._CLayerNormGrad, NGRAD, (ws, wsb), **kw)


def test_layer_norm_grad_refusals():
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(cols=-1), dict(cols=z.BLOCK_NORM_MAX_COLS + 1), dict(flags=2), dict(dh=NONE),
               dict(dh=FP32), dict(dh=rows(ld=5)), dict(dx=NONE), dict(dx=rows(dtype=9)), dict(dx=at(2, dtype=F32)), dict(dx_out=FP32),
               dict(dx_out=rows(ld=1)), dict(dy=FP32), dict(w=rows(dtype=3)), dict(x_out=NONE), dict(x_out=FP32), dict(mean=None),
               dict(mean=4097), dict(rstd=None), dict(rstd=8193), dict(dw=rows(dtype=8)), dict(flags=z.GRAD_ACCUMULATE),
               dict(ckpt_xn=4096, format=0), dict(ckpt_xn=4104, format=1), dict(ws=None), dict(ws=4100),
               # two outputs at one address
               dict(dw=NGRAD["db"]), dict(dy=NGRAD["dx"]), dict(db=NGRAD["dx"])):
        assert norm_grad(**kw) == BAD, kw
    n = z.zero_layer_norm_grad_workspace_bytes(8, 64)
    assert n > 0 and norm_grad(wsb=n - 1) == SMALL
    # an act8 buffer stands for x_out and mean
    assert norm_grad(wsb=n - 1, ckpt_xn=4096, format=1, x_out=NONE, mean=None) == SMALL
    assert z.lib().zero_layer_norm_grad(None, None, 0, None) == BAD
    assert norm_grad(cols=0) == OK
    for bad in ((-1, 4), (4, -1), (1 << 31, 4), (4, z.BLOCK_NORM_MAX_COLS + 1)):
        assert z.zero_layer_norm_grad_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("r,c", [(1, 1), (1, 64), (16384, 4096), (100000, 64), (3000, 16384), (2**31 - 1, 1), (5, 8193)])
def test_layer_norm_grad_workspace_is_two_rows_a_unit(r, c):
    n = z.zero_layer_norm_grad_workspace_bytes(r, c)
    wide = 8 * r if c > 8192 else 0  # and two values a row
    assert n > wide and (n - wide) % (8 * c) == 0 and (n - wide) // (8 * c) <= min(r, 4096)


FFN = dict(rows=8, cols=64, hidden=64, h=at(0), w_gate=at(1), w_up=at(2), a=at(3), act=z.FFN_SILU)


def ffn(ws=4096, wsb=1 << 40, **kw):
    return call("zero_block_ffn", z._CBlockFfn, FFN, (ws, wsb), **kw)


SIZES = (dict(rows=-1), dict(rows=1 << 31), dict(cols=-1), dict(cols=(1 << 30) + 1), dict(hidden=-1), dict(hidden=(1 << 30) + 1),
         dict(rows=1 << 26, hidden=1 << 20), dict(cols=1 << 18, hidden=1 << 20), dict(rows=1 << 20, cols=1 << 20))


def test_ffn_refusals():
    for kw in SIZES + (dict(act=0), dict(act=4), dict(h=NONE), dict(h=FP32), dict(h=rows(ld=63)), dict(h=rows(data=4097)), dict(w_gate=NONE),
                       dict(w_gate=FP32), dict(w_gate=rows(ld=1)), dict(w_up=NONE), dict(w_up=FP32), dict(w_up=rows(reserved=3)),
                       dict(a=NONE), dict(a=FP32), dict(a=rows(ld=2)), dict(gate=FP32), dict(up=rows(ld=7)), dict(ckpt_gate=4096, format=0),
                       dict(ckpt_up=4096, format=5), dict(ckpt_gate=4104, format=1), dict(ckpt_up=4104, format=1),
                       # two outputs at one address
                       dict(gate=FFN["a"]), dict(gate=at(7), up=at(7)), dict(ckpt_gate=4096, ckpt_up=4096, format=1)):
        assert ffn(**kw) == BAD, kw
    assert z.lib().zero_block_ffn(None, None, 0, None) == BAD
    assert ffn(rows=0, h=NONE, a=NONE) == OK and ffn(hidden=0, w_gate=NONE, w_up=NONE, a=NONE) == OK
    n = z.zero_block_ffn_workspace_bytes(64, 20000, 64)
    wide = dict(rows=64, cols=20000, **{k: at(i, ld=20000) for i, k in enumerate(("h", "w_gate", "w_up"))})
    assert n > 0 and ffn(ws=None, **wide) == BAD and ffn(ws=4100, wsb=n, **wide) == BAD and ffn(wsb=n - 1, **wide) == SMALL


GRAD = dict(rows=8, cols=64, hidden=64, da=at(0), gate=at(1), up=at(2), w_gate=at(3), w_up=at(4), h=at(5), dgate=at(6), dup=at(7), dh=at(8),
            dw_gate=at(9), dw_up=at(10), act=z.FFN_GELU)


def ffn_grad(ws=4096, wsb=1 << 40, **kw):
    return call("zero_block_ffn_grad", z._CBlockFfnGrad, GRAD, (ws, wsb), **kw)


def test_ffn_grad_refusals():
    coded = dict(gate=NONE, up=NONE, ckpt_gate=4096, ckpt_up=8192, format=1)
    for kw in SIZES + (dict(act=0), dict(act=9), dict(flags=2), dict(reserved=1), dict(da=NONE), dict(da=FP32), dict(da=rows(ld=1)),
                       dict(gate=NONE), dict(up=FP32), dict(dgate=NONE), dict(dgate=FP32), dict(dup=NONE), dict(dup=rows(ld=63)),
                       dict(w_gate=NONE), dict(w_up=FP32), dict(dh=FP32), dict(dh=NONE), dict(h=NONE), dict(h=FP32), dict(dw_gate=rows(dtype=7)),
                       dict(dw_up=rows(ld=1)), dict(flags=z.GRAD_ACCUMULATE), dict(col_scale=at(11)), dict(ckpt_a=4096, format=0),
                       dict(ckpt_a=4104, format=1), dict(coded, ckpt_up=None), dict(coded, format=0), dict(coded, ckpt_gate=4104),
                       dict(ckpt_h=4104, format=1), dict(ckpt_h=4096, format=0), dict(ckpt_h=4096, format=1, col_scale=rows(dtype=6)),
                       # without a weight gradient nothing that only it reads
                       dict(dw_gate=NONE, dw_up=NONE), dict(dw_gate=NONE, dw_up=NONE, h=NONE, ckpt_h=4096, format=1),
                       # two outputs at one address
                       dict(dup=GRAD["dgate"]), dict(dw_up=GRAD["dw_gate"]), dict(dh=GRAD["dup"]), dict(ckpt_a=(9 + 1) << 20, format=1)):
        assert ffn_grad(**kw) == BAD, kw
    assert z.lib().zero_block_ffn_grad(None, None, 0, None) == BAD
    n = z.zero_block_ffn_grad_workspace_bytes(64, 64, 20000)
    wide = dict(rows=64, hidden=20000, **{k: at(i, ld=20000) for i, k in enumerate(("da", "gate", "up", "dgate", "dup"))})
    assert n > 0 and ffn_grad(ws=None, **wide) == BAD and ffn_grad(ws=4100, wsb=n, **wide) == BAD and ffn_grad(wsb=n - 1, **wide) == SMALL
    assert ffn_grad(rows=0, flags=z.GRAD_ACCUMULATE, dw_gate=at(9, dtype=F32), dw_up=at(10, dtype=F32)) == OK
    assert ffn_grad(hidden=0, dh=NONE, w_gate=NONE, w_up=NONE) == OK


@pytest.mark.parametrize("bad", [(-1, 4, 4), (4, -1, 4), (4, 4, -1), (1 << 31, 4, 4), (4, 1 << 31, 4), (4, 1 << 20, 1 << 20)])
def test_ffn_workspace_of_invalid_sizes(bad):
    assert z.zero_block_ffn_workspace_bytes(*bad) == 0 and z.zero_block_ffn_grad_workspace_bytes(*bad) == 0


def test_ffn_workspaces_hold_the_weight_gradients_from_8_bits_too():
    for r, c, h in ((1, 1, 1), (192, 768, 2048), (8192, 4096, 11008), (30000, 64, 64), (5000, 333, 200)):
        assert z.zero_block_ffn_grad_workspace_bytes(r, c, h) >= z.zero_act8_wgrad_workspace_bytes(r, h, c)


def test_binding_refuses_host_tensors_and_formats():
    t = torch.zeros(4, 8, dtype=torch.bfloat16)
    for f in (lambda: z.zero_layer_norm(z.LayerNorm(x=t, h=t)), lambda: z.zero_layer_norm_grad(z.LayerNormGrad(dx=t, dh=t, rstd=t)),
              lambda: z.zero_block_ffn(z.BlockFfn(h=t, w_gate=t, w_up=t, a=t)),
              lambda: z.zero_block_ffn_grad(z.BlockFfnGrad(da=t, dgate=t, dup=t))):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(ValueError, match="formats"):
        z._one_format(z.Act8(1, 1, 1, t), None, z.Act8(1, 1, 2, t))
    assert z._one_format(None, z.Act8(1, 1, 2, t)) == 2 and z._one_format() == 0
