"""Plain 64-bit forms of the calls around a training block, written from their
formulas, and the error bounds that their tests use.

Bounds count roundings. u = 2^-24 is half a step of fp32; a sum whose terms
pass through at most n roundings is off by at most n u (sum of |terms|), to
first order. `mag` below is always that sum of |terms| in 64 bits. A result
rounded to bf16 adds half a step, 2^-8 of itself."""
import math

import numpy as np
import torch

import sharded_optimizer_step_amd as z

U = 2.0**-24
HALF_STEP = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}
BLOCK = 32
FORMATS = {"e4m3": z.ACT8_E4M3, "int8": z.ACT8_INT8}


def grid(fmt):
    """The non-negative values of the codes 0, 1, 2, ..."""
    if fmt == z.ACT8_INT8:
        return np.arange(128.0)
    return np.array([m * 2.0**-9 for m in range(8)] +
                    [(1 + m / 8) * 2.0**(e - 7) for e in range(1, 16) for m in range(8)])[:127]


def round_act8(x, fmt):
    """What an 8-bit checkpoint of x (float64 numpy, rows x cols) decodes to."""
    g = grid(fmt)
    out = np.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        b = x[:, c:c + BLOCK]
        top = np.abs(b).max(1, keepdims=True)
        bad = ~np.isfinite(top)
        k = np.full(top.shape, -117)
        for _ in range(256):  # the first power of two, from the bottom, that reaches
            k = np.where(np.where(bad, 0, top) > g[-1] * 2.0**k.astype(np.float64), k + 1, k)
        unit = 2.0**k.astype(np.float64)
        a = np.where(bad, 0, np.abs(b)) / unit
        hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)
        lo = hi - 1
        up = (a - g[lo] > g[hi] - a) | ((a - g[lo] == g[hi] - a) & (hi % 2 == 0))
        q = np.where(up, g[hi], g[lo]) * unit
        q = np.where(q >= 2.0**128, np.inf, q)
        out[:, c:c + BLOCK] = np.where(bad, np.nan, np.copysign(q, b))
    return out


def decode_act8(ckpt):
    """(values, unit of every block) of a checkpoint's bytes, float64 numpy."""
    rows, cols = ckpt.rows, ckpt.cols
    pitch = -(-cols // BLOCK) * BLOCK
    b = ckpt.buf.cpu().numpy()
    codes = b[:rows * pitch].reshape(rows, pitch)
    scale = b[rows * pitch:rows * (pitch + pitch // BLOCK)].reshape(rows, -1)
    g = grid(ckpt.format)
    if ckpt.format == z.ACT8_E4M3:
        table = np.concatenate([g, [np.nan], -g, [np.nan]])
    else:
        table = np.concatenate([g, [np.nan], -g[:0:-1]])
    unit = np.where(scale == 255, np.nan, 2.0**(scale.astype(np.float64) - 127))
    assert np.all(codes[:, cols:] == 0), "padding columns"
    v = (table[codes].reshape(rows, -1, BLOCK) * unit[:, :, None]).reshape(rows, pitch)[:, :cols]
    return v, unit


def assert_saved(ckpt, want, rel, where=""):
    """The checkpoint holds `want` (float64 numpy) rounded to its codes, where
    the kernel's own fp32 values are within rel of it: the block's unit is the
    smallest that reaches, and every value is within half a step (and rel)."""
    got, unit = decode_act8(ckpt)
    rows, cols = want.shape
    pad = np.zeros((rows, -cols % BLOCK))
    b = np.concatenate([np.abs(want), pad], 1).reshape(rows, -1, BLOCK)
    top, f = b.max(2), grid(ckpt.format)[-1]
    assert np.all(top <= f * unit * (1 + rel)), where
    assert np.all((top > f * unit / 2 * (1 - rel)) | (unit == 2.0**-117)), where
    per = np.repeat(unit, BLOCK, 1)[:, :cols]
    if ckpt.format == z.ACT8_E4M3:
        half = np.maximum(2.0**-4 * np.abs(want), 2.0**-10 * per)
    else:
        half = 0.5 * per
    err = np.abs(got - want)
    assert np.all(err <= half * (1 + 2 * rel) + rel * np.abs(want)), (where, float((err - half).max()))


def assert_within(got, want, mag, rel, where=""):
    """|got - want| <= half a step of got's type + rel * mag, all finite."""
    assert tuple(got.shape) == tuple(want.shape), (where, got.shape, want.shape)
    g, w = got.double().cpu(), want.double().cpu()
    bound = HALF_STEP[got.dtype] * w.abs() * (1 + 2.0**-7) + rel * mag.double().cpu() + 1e-37
    err = (g - w).abs()
    assert torch.isfinite(g).all() and torch.isfinite(w).all(), where
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, (where, worst)


def by_row(gate, gate_rows, rows):
    return gate.double().repeat_interleave(gate_rows, 0)[:rows]


def norm_reference(b, xn_from):
    """zero_block_norm's formulas in 64 bits. xn_from: the stored x_out whose
    norm is taken. Returns {name: (value, mag)}."""
    out = {}
    rows = b.x.shape[0]
    x = b.x.double()
    if b.y is not None:
        y = b.y.double()
        if b.w_post is not None:
            out["rstd_post"] = (y.square().mean(1) + np.float32(b.eps).item()).rsqrt()
            y = y * out["rstd_post"][:, None]
        out["yn"] = y
        t = float(np.float32(b.residual_scale)) * y
        if b.w_post is not None:
            t = t * b.w_post.double()
        if b.gate is not None:
            t = t * by_row(b.gate, b.gate_rows, rows)
        out["x_out"], out["x_out_mag"] = x + t, x.abs() + t.abs()
    if b.w_pre is not None:
        xo = xn_from.double()
        out["rstd_pre"] = (xo.square().mean(1) + np.float32(b.eps).item()).rsqrt()
        out["xn"] = xo * out["rstd_pre"][:, None]
        out["h"] = out["xn"] * b.w_pre.double()
    return out


def grad_reference(b, xn, yn):
    """zero_block_norm_grad's formulas in 64 bits from the rows xn and yn, with
    the sums of |terms|: {name: (value, mag)}."""
    rows, cols = b.dx.shape
    dev = b.dx.device
    zero = torch.zeros(rows, cols, dtype=torch.float64, device=dev)
    alpha = float(np.float32(b.residual_scale))
    out = {}
    d = b.dx_out.double() if b.dx_out is not None else zero
    mag = d.abs()
    if b.dh is not None:
        dh, r = b.dh.double(), b.rstd_pre.double()[:, None]
        v = dh * b.w_pre.double()
        d = d + r * (v - xn * (v * xn).mean(1, keepdim=True))
        mag = mag + r * (v.abs() + xn.abs() * (v * xn).abs().mean(1, keepdim=True))
        out["dw_pre"] = ((dh * xn).sum(0, keepdim=True), (dh * xn).abs().sum(0, keepdim=True))
    out["dx"] = (d, mag)
    g = alpha * (by_row(b.gate, b.gate_rows, rows) if b.gate is not None else torch.ones(1, 1, dtype=torch.float64, device=dev))
    w = b.w_post.double() if b.w_post is not None else torch.ones(cols, dtype=torch.float64, device=dev)
    if b.w_post is not None:
        r = b.rstd_post.double()[:, None]
        e = g * w
        out["dy"] = (r * (e * d - yn * (e * d * yn).mean(1, keepdim=True)),
                     r * ((e * mag).abs() + yn.abs() * (e * mag * yn).abs().mean(1, keepdim=True)))
        out["dw_post"] = ((g * d * yn).sum(0, keepdim=True), (g * mag * yn).abs().sum(0, keepdim=True))
    else:
        out["dy"] = ((g * d).expand(rows, cols), (g * mag).abs().expand(rows, cols))
    if b.gate is not None and yn is not None:
        n = b.gate.shape[0]
        at = torch.arange(rows, device=dev) // b.gate_rows
        f = lambda t: torch.zeros(n, cols, dtype=torch.float64, device=dev).index_add_(0, at, t)  # noqa: E731
        out["dgate"] = (f(alpha * d * w * yn), f((alpha * mag * w * yn).abs()))
    return out


def strided(t, pad, offset=0):
    """t as a view of a larger buffer: row stride cols + pad, the first element
    `offset` elements into the allocation; the rest is a canary."""
    if t is None:
        return None, None
    rows, cols = t.shape
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 7,), 77.0, dtype=t.dtype, device=t.device)
    v = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v, buf


def canary_ok(buf, rows, cols, pad, offset):
    ld = cols + pad
    whole = torch.ones_like(buf, dtype=torch.bool)
    whole[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
    return bool((buf[whole] == 77.0).all())
