"""The calls around a training block on the CPU: their structures' layouts, the
sizes that they report, and every refusal, before anything touches a GPU. No
call here launches a kernel."""
import ctypes
import os
import subprocess

import pytest
import torch

import sharded_optimizer_step_amd as z

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, SMALL, OK = 1, 2, 0
BF16, F32 = 1, 2


def rows(data=4096, ld=64, dtype=BF16, reserved=0):
    return z._CRows(data, ld, dtype, reserved)


def ref(x):
    return ctypes.byref(x) if x is not None else None


def test_struct_layouts_and_constants(tmp_path):
    structs = {"zero_rows": z._CRows, "zero_block_norm_args": z._CBlockNorm, "zero_block_norm_grad_args": z._CBlockNormGrad}
    consts = {"ZERO_ACT8_E4M3": z.ACT8_E4M3, "ZERO_ACT8_INT8": z.ACT8_INT8, "ZERO_GRAD_ACCUMULATE": z.GRAD_ACCUMULATE,
              "ZERO_BLOCK_NORM_MAX_COLS": z.BLOCK_NORM_MAX_COLS, "ZERO_BF16": z._DTYPES[torch.bfloat16],
              "ZERO_F32": z._DTYPES[torch.float32]}
    body = [f'printf("{n} %zu\\n", sizeof({n}));' for n in structs]
    body += [f'printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for n, c in structs.items() for f, _ in c._fields_]
    body += [f'printf("{n} %zu\\n", (size_t){n});' for n in consts]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zero_step.h"\nint main(void){' + "".join(body) + "return 0;}\n")
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", "-o", str(exe),
                    str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for n, c in structs.items():
        assert int(got[n]) == ctypes.sizeof(c)
        for f, _ in c._fields_:
            assert int(got[f"{n}.{f}"]) == getattr(c, f).offset, (n, f)
    for n, v in consts.items():
        assert int(got[n]) == v, n


@pytest.mark.parametrize("r,c,n", [(0, 5, 0), (5, 0, 0), (1, 1, 33), (3, 32, 99), (3, 33, 198), (16384, 4096, 16384 * 4224),
                                   (-1, 4, 0), (4, -1, 0), (1 << 31, 4, 0), (4, (1 << 30) + 1, 0), (1 << 30, 1 << 20, 0)])
def test_checkpoint_bytes(r, c, n):
    assert z.zero_act8_bytes(r, c) == n


def test_save_and_load_refusals():
    L = z.lib()

    def both(x, r, c, f, ck, want):
        assert L.zero_act8_save(ref(x), r, c, f, ck, None) == want
        assert L.zero_act8_load(ck, r, c, f, ref(x), None) == want

    both(rows(), -1, 8, 1, 4096, BAD)
    both(rows(), 8, -1, 1, 4096, BAD)
    both(rows(), 1 << 31, 8, 1, 4096, BAD)
    both(rows(), 8, 1 << 31, 1, 4096, BAD)
    both(rows(ld=1 << 29), 1 << 20, 1 << 20, 1, 4096, BAD)  # more vectors than a grid counts
    both(rows(), 8, 8, 0, 4096, BAD)
    both(rows(), 8, 8, 3, 4096, BAD)
    both(None, 8, 8, 1, 4096, BAD)
    both(rows(data=None), 8, 8, 1, 4096, BAD)
    both(rows(ld=7), 8, 8, 1, 4096, BAD)
    both(rows(dtype=0), 8, 8, 1, 4096, BAD)
    both(rows(dtype=3), 8, 8, 1, 4096, BAD)
    both(rows(reserved=1), 8, 8, 1, 4096, BAD)
    both(rows(data=4097), 8, 8, 1, 4096, BAD)
    both(rows(data=4098, dtype=F32), 8, 8, 1, 4096, BAD)
    both(rows(), 8, 8, 1, None, BAD)
    both(rows(), 8, 8, 1, 4104, BAD)
    both(rows(data=None), 0, 8, 1, None, OK)
    both(rows(data=None), 8, 0, 2, None, OK)


def test_wgrad_refusals():
    L = z.lib()

    def call(dy=rows(), ck=4096, r=8, o=64, c=64, f=1, scale=None, dw=rows(dtype=F32), flags=0, ws=None, wsb=0):
        return L.zero_act8_wgrad(ref(dy), ck, r, o, c, f, ref(scale), ref(dw), flags, ws, wsb, None)

    for kw in (dict(r=-1), dict(o=-1), dict(c=-1), dict(r=1 << 31), dict(o=1 << 31), dict(c=1 << 31),
               dict(o=1 << 25, c=1 << 20, dy=rows(ld=1 << 25), dw=rows(ld=1 << 20)),
               dict(o=(1 << 31) - 1, dy=rows(ld=1 << 31)), dict(f=0), dict(f=3), dict(flags=2),
               dict(flags=4 | z.GRAD_ACCUMULATE), dict(dy=None), dict(dw=None), dict(dy=rows(data=None)), dict(dy=rows(ld=63)),
               dict(dy=rows(dtype=F32)), dict(dy=rows(data=4097)), dict(dw=rows(data=None)), dict(dw=rows(ld=63)),
               dict(dw=rows(dtype=BF16), flags=z.GRAD_ACCUMULATE), dict(dw=rows(data=4098, dtype=F32)), dict(dw=rows(dtype=7)),
               dict(ck=None), dict(ck=4100), dict(scale=rows(dtype=0)), dict(scale=rows(data=4097)), dict(scale=rows(data=None))):
        assert call(**kw) == BAD, kw
    # a split sum needs its workspace
    n = z.zero_act8_wgrad_workspace_bytes(20000, 64, 64)
    assert n > 0 and n % (64 * 64 * 4) == 0
    assert call(r=20000) == BAD
    assert call(r=20000, ws=4100, wsb=n) == BAD
    assert call(r=20000, ws=4096, wsb=n - 1) == SMALL
    assert call(o=0, dy=rows(data=None)) == OK and call(c=0) == OK
    assert call(r=0, flags=z.GRAD_ACCUMULATE, dy=rows(data=None), ck=None) == OK
    for bad in ((-1, 4, 4), (4, -1, 4), (4, 4, -1), (1 << 31, 4, 4), (4, 1 << 31, 4), (4, 1 << 25, 1 << 20)):
        assert z.zero_act8_wgrad_workspace_bytes(*bad) == 0


NORM = dict(rows=8, cols=64, gate_rows=0, residual_scale=1.0, eps=1e-6, x=rows(), y=rows(), x_out=rows(), reserved=0)
PRE = dict(w_pre=rows(), h=rows())


def norm(**kw):
    c = z._CBlockNorm()
    for k, v in {**NORM, **kw}.items():
        setattr(c, k, v)
    return z.lib().zero_block_norm(ctypes.byref(c), None)


def test_norm_refusals():
    none = rows(data=None)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(cols=-1), dict(cols=z.BLOCK_NORM_MAX_COLS + 1), dict(reserved=1),
               dict(residual_scale=nan), dict(residual_scale=inf), dict(residual_scale=1e39), dict(eps=-1e-9), dict(eps=nan), dict(eps=inf),
               dict(x=none), dict(x=rows(ld=63)), dict(x=rows(dtype=5)), dict(x=rows(data=4099)), dict(x=rows(reserved=2)),
               dict(y=rows(dtype=F32)), dict(y=rows(ld=2)), dict(x_out=none), dict(x_out=rows(dtype=F32)), dict(x_out=rows(ld=3)),
               dict(w_post=rows(dtype=9)), dict(gate=rows()), dict(gate=rows(), gate_rows=-1), dict(gate=rows(ld=9), gate_rows=1),
               dict(rstd_post=4096), dict(w_post=rows(), rstd_post=4097), dict(h=rows()), dict(rstd_pre=4096),
               dict(ckpt_pre=4096, format=1), dict(ckpt_post=4096, format=0), dict(ckpt_post=4096, format=3), dict(ckpt_post=4104, format=1),
               dict(PRE, h=none), dict(PRE, h=rows(dtype=F32)), dict(PRE, h=rows(ld=8)), dict(PRE, w_pre=rows(dtype=4)),
               dict(PRE, rstd_pre=4098), dict(PRE, ckpt_pre=4104, format=2),
               # no block output: nothing that belongs to it, and something to compute
               dict(y=none, x_out=none), dict(PRE, y=none), dict(PRE, y=none, x_out=none, w_post=rows()),
               dict(PRE, y=none, x_out=none, gate=rows(), gate_rows=1), dict(PRE, y=none, x_out=none, ckpt_post=4096, format=1)):
        assert norm(**kw) == BAD, kw
    assert z.lib().zero_block_norm(None, None) == BAD
    assert norm(rows=0) == OK and norm(cols=0) == OK


GRAD = dict(rows=8, cols=64, gate_rows=0, residual_scale=1.0, dx_out=rows(), dx=rows(), dy=rows(data=8192), flags=0)
GPRE = dict(dh=rows(), w_pre=rows(), rstd_pre=4096, x_out=rows())
GPOST = dict(w_post=rows(), rstd_post=4096, y=rows())


def grad(ws=4096, wsb=1 << 40, **kw):
    c = z._CBlockNormGrad()
    for k, v in {**GRAD, **kw}.items():
        setattr(c, k, v)
    return z.lib().zero_block_norm_grad(ctypes.byref(c), ws, wsb, None)


def test_norm_grad_refusals():
    none, f32 = rows(data=None), rows(dtype=F32)
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(cols=-1), dict(cols=z.BLOCK_NORM_MAX_COLS + 1), dict(flags=2),
               dict(residual_scale=float("nan")), dict(residual_scale=1e39), dict(dx=none), dict(dx=rows(ld=5)), dict(dx=rows(dtype=0)),
               dict(dx_out=none), dict(dx_out=f32), dict(dx_out=rows(ld=1)), dict(dy=f32), dict(dy=rows(ld=1)),
               dict(w_pre=rows()), dict(dw_pre=rows()), dict(dw_post=rows()), dict(dgate=rows()), dict(gate=rows()),
               dict(gate=rows(ld=1), gate_rows=1), dict(GPRE, dh=f32), dict(GPRE, dh=rows(ld=1)), dict(GPRE, w_pre=none),
               dict(GPRE, rstd_pre=None), dict(GPRE, rstd_pre=4097), dict(GPRE, x_out=none), dict(GPRE, x_out=f32),
               dict(GPRE, x_out=none, ckpt_pre=4096, format=0), dict(GPRE, x_out=none, ckpt_pre=4104, format=1),
               dict(GPOST, w_post=rows(dtype=3)), dict(GPOST, rstd_post=None), dict(GPOST, rstd_post=4098), dict(GPOST, y=none),
               dict(GPOST, y=f32), dict(GPOST, y=none, ckpt_post=4104, format=1), dict(GPOST, y=none, ckpt_post=4096, format=9),
               dict(GPOST, dw_post=rows(), flags=z.GRAD_ACCUMULATE), dict(GPRE, dw_pre=rows(), flags=z.GRAD_ACCUMULATE),
               dict(gate=rows(), gate_rows=2, dgate=rows(), y=none), dict(gate=rows(), gate_rows=2, dgate=rows(ld=1), y=rows()),
               dict(GPOST, ws=None), dict(GPOST, ws=4100)):
        assert grad(**kw) == BAD, kw
    assert z.lib().zero_block_norm_grad(None, None, 0, None) == BAD
    n = z.zero_block_norm_grad_workspace_bytes(8, 64, 0)
    assert n > 0 and grad(wsb=n - 1, **GPOST) == SMALL
    assert grad(cols=0) == OK
    for bad in ((-1, 4, 0), (4, -1, 0), (4, 4, -1), (1 << 31, 4, 0), (4, z.BLOCK_NORM_MAX_COLS + 1, 0)):
        assert z.zero_block_norm_grad_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("r,c,g", [(1, 1, 0), (1, 64, 1), (7, 64, 3), (16384, 4096, 0), (16384, 4096, 2048), (16384, 4096, 1),
                                   (100000, 64, 1), (100000, 64, 7), (3000, 16384, 1), (3000, 16384, 0), (511, 4096, 1), (2**31 - 1, 1, 0)])
def test_grad_workspace_is_two_rows_a_unit(r, c, g):
    n = z.zero_block_norm_grad_workspace_bytes(r, c, g)
    wide = 8 * r if c > 6144 else 0  # and two values a row
    assert n > wide and (n - wide) % (8 * c) == 0
    units = (n - wide) // (8 * c)
    # never more units than rows (the last gate row counted whole), nor many more than the waves that fill the chip
    assert units <= (-(-r // g) * g if g else r) and units <= 2 * 4096


def test_two_outputs_at_one_address_are_refused():
    a, b = rows(data=1 << 20), rows(data=1 << 21)
    f = dict(PRE, w_post=rows(), x_out=a, h=b, rstd_post=4096, rstd_pre=8192, ckpt_post=4096, ckpt_pre=8192, format=1)
    for kw in (dict(f, h=a), dict(f, rstd_pre=4096), dict(f, ckpt_pre=4096)):
        assert norm(**kw) == BAD, kw
    full = dict(GPRE, **GPOST, gate=rows(), gate_rows=8, dw_pre=rows(data=1 << 16), dw_post=rows(data=1 << 17),
                dgate=rows(data=1 << 18))
    small = z.zero_block_norm_grad_workspace_bytes(8, 64, 8) - 1
    assert grad(wsb=small, **full) == SMALL  # nothing else is wrong with it
    for kw in (dict(dw_post=full["dw_pre"]), dict(dgate=full["dw_pre"]), dict(dgate=full["dw_post"]), dict(dy=GRAD["dx"])):
        assert grad(wsb=small, **{**full, **kw}) == BAD, kw


def test_packed_structures_are_the_c_ones():
    for packed, c in ((z._ROWS, z._CRows), (z._BLOCK_NORM, z._CBlockNorm), (z._BLOCK_NORM_GRAD, z._CBlockNormGrad)):
        assert packed.size == ctypes.sizeof(c)
        flat = []

        def walk(cls, at):
            for f, t in cls._fields_:
                o = at + getattr(cls, f).offset
                walk(t, o) if issubclass(t, ctypes.Structure) else flat.append((o, t))

        walk(c, 0)
        values = [float(i) if t is ctypes.c_double else i for i, (_, t) in enumerate(flat)]
        image = packed.pack(*values)
        for (o, t), v in zip(flat, values):
            got = t.from_buffer_copy(image, o).value
            assert (got or 0) == v, (c, o)


def test_binding_refuses_host_tensors_and_shapes():
    """What the binding itself checks; the C calls are not reached."""
    t = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: z.zero_act8_save(t, None), lambda: z.zero_act8_load(None, t),
                 lambda: z.zero_act8_wgrad(t, z.Act8(4, 8, 1, t), t), lambda: z.zero_block_norm(z.BlockNorm(x=t)),
                 lambda: z.zero_block_norm_grad(z.BlockNormGrad(dx=t))):
        with pytest.raises((ValueError, TypeError), match="device tensor"):
            call()
    with pytest.raises(TypeError, match="Tensor"):
        z.zero_act8_save([1.0], None)
    with pytest.raises(ValueError, match="matrix"):
        z.zero_act8_save(t[0], None)
    with pytest.raises(ValueError, match="device tensor"):
        z._row_major(t, "t", 4, 8, 0)
    # -1 is the host: as if on the device
    assert z._row_major(None, "t", 4, 8, -1) == (0, 0, 0, 0)
    assert z._row_major(t, "t", 4, 8, -1) == (t.data_ptr(), 8, 1, 0)
    assert z._row_major(t[:, :3], "t", 4, 3, -1)[1] == 8 and z._row_major(t[0], "t", 1, 8, -1)[1] == 8
    assert z._row_major(t[:1, 2:5].float(), "t", 1, 3, -1)[1:] == (3, 2, 0)
    with pytest.raises(ValueError, match="expected"):
        z._row_major(t, "t", 4, 9, -1)
    with pytest.raises(ValueError, match="expected"):
        z._row_major(t[None], "t", 4, 8, -1)
    with pytest.raises(TypeError, match="expected"):
        z._row_major(t, "t", 4, 8, -1, torch.float32)
    with pytest.raises(TypeError, match="expected"):
        z._row_major(t.half(), "t", 4, 8, -1)
    with pytest.raises(ValueError, match="next to each other"):
        z._row_major(t.t(), "t", 8, 4, -1)
    with pytest.raises(ValueError, match="overlap"):
        z._row_major(t[0:1].expand(4, 8), "t", 4, 8, -1)
    with pytest.raises(TypeError):
        z._act8(t, "c", 4, 8, -1)
    with pytest.raises(TypeError, match="Act8"):
        z._checkpoint(None)

    class Stream:
        device_index, cuda_stream = 1, 7

    assert z._stream_of(Stream, 1) == 7
    with pytest.raises(ValueError, match="stream"):
        z._stream_of(Stream, 0)
    with pytest.raises(ValueError, match="holds"):
        z._act8(z.Act8(4, 9, 1, t), "c", 4, 8, -1)
    with pytest.raises(ValueError, match="formats"):
        z._act8_format(z.Act8(1, 1, 1, t), z.Act8(1, 1, 2, t))
    assert z._act8_format(None, z.Act8(1, 1, 2, t)) == 2 and z._act8_format(None, None) == 0
    with pytest.raises(ValueError, match="gate_rows"):
        z._gates(4, 0)
