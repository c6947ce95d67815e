"""Plain 64-bit forms of the layer norm and the gated feed-forward block,
written from their formulas, and the error bounds that their tests use (see
block_cases.py for how bounds count roundings)."""
import math

import numpy as np
import torch

import sharded_optimizer_step_amd as z
from block_cases import BLOCK, HALF_STEP, U, decode_act8, grid

ACTS = {"silu": z.FFN_SILU, "gelu": z.FFN_GELU, "gelu_tanh": z.FFN_GELU_TANH}


def act64(act, g):
    """(act(g), act'(g)) of float64 values."""
    if act == z.FFN_SILU:
        p, q = torch.sigmoid(g), torch.sigmoid(-g)
        return g * p, p * (1 + g * q)
    if act == z.FFN_GELU:
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = 2 * c * (g + 0.044715 * g**3)
    p, q = torch.sigmoid(s), torch.sigmoid(-s)
    return g * p, p + g * p * q * 2 * c * (1 + 3 * 0.044715 * g * g)


def nearest_bf16(x):
    """float64 values rounded to bf16 once (with its subnormals), as float64."""
    e = (torch.frexp(x)[1].to(torch.int64) - 8).clamp(min=-133)
    step = ((e + 1023) << 52).view(torch.float64)
    r = torch.round(x / step) * step
    return torch.where(torch.isfinite(x), r, x)


def assert_saved_within(ckpt, want, off, where=""):
    """The checkpoint holds `want` (float64) rounded to its codes, where the
    kernel's own fp32 values are within `off` of it: the block's unit is the
    smallest that reaches, and every value is within half a step and off."""
    got, unit = decode_act8(ckpt)
    want, off = want.cpu().numpy(), off.cpu().numpy()
    rows, cols = want.shape
    pad = np.zeros((rows, -cols % BLOCK))
    blocks = lambda t: np.concatenate([t, pad], 1).reshape(rows, -1, BLOCK).max(2)  # noqa: E731
    f = grid(ckpt.format)[-1]
    assert np.all(blocks(np.abs(want) - off) <= f * unit), where
    assert np.all((blocks(np.abs(want) + off) > f * unit / 2) | (unit == 2.0**-117)), where
    per = np.repeat(unit, BLOCK, 1)[:, :cols]
    if ckpt.format == z.ACT8_E4M3:
        half = np.maximum(2.0**-4 * (np.abs(want) + off), 2.0**-10 * per)
    else:
        half = 0.5 * per
    err = np.abs(got - want)
    assert np.all(err <= half + off + 1e-37), (where, float((err - half - off).max()))


def assert_close(got, want, off, where=""):
    """|got - want| <= half a step of got's type + off, all finite."""
    assert tuple(got.shape) == tuple(want.shape), (where, got.shape, want.shape)
    g, w = got.double().cpu(), want.double().cpu()
    bound = HALF_STEP[got.dtype] * w.abs() * (1 + 2.0**-7) + off.double().cpu() * (1 + 2.0**-7) + 1e-37
    assert torch.isfinite(g).all() and torch.isfinite(w).all(), where
    worst = ((g - w).abs() / bound).max().item() if g.numel() else 0.0
    assert worst <= 1.0, (where, worst)


# A row's mean: sums of the differences to a first mean, at most 16 terms in a
# lane, 6 steps of the wave, 16 waves, the difference and the last sum: 40
# roundings, of terms whose sum of magnitudes is at most twice that of x. Its
# squares: the same path, the terms' own 3, and what the mean is off by.
MEAN, XN = 84 * U, 100 * U


def layer_norm_reference(b, x):
    """zero_layer_norm's formulas in 64 bits on the stored rows x: {name: (value, off)}."""
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + float(np.float32(b.eps))).rsqrt()
    xn = c * rstd[:, None]
    # where a row lies far from 0 its first mean is off by more than its spread is worth
    far = 1 + 22 * U * x.abs().mean(1) * rstd
    off = XN * (xn.abs() + far[:, None])
    w = b.w.double() if b.w is not None else torch.ones_like(x[0])
    h = xn * w + (b.b.double() if b.b is not None else 0.0)
    return dict(mean=(mean, MEAN * x.abs().mean(1)), rstd=(rstd, XN * rstd * far), xn=(xn, off),
                h=(h, off * w.abs() + 2 * U * (h.abs() + (xn * w).abs())))


def layer_norm_grad_reference(b, xn):
    """zero_layer_norm_grad's formulas in 64 bits from the rows xn: {name: (value, sum of |terms|)}."""
    dh, r = b.dh.double(), b.rstd.double()[:, None]
    v = dh * b.w.double() if b.w is not None else dh
    d = r * (v - v.mean(1, keepdim=True) - xn * (v * xn).mean(1, keepdim=True))
    mag = r * (v.abs() + v.abs().mean(1, keepdim=True) + xn.abs() * (v * xn).abs().mean(1, keepdim=True))
    if b.dx_out is not None:
        d, mag = d + b.dx_out.double(), mag + b.dx_out.double().abs()
    return dict(dx=(d, mag), dy=(d, mag), dw=((dh * xn).sum(0), (dh * xn).abs().sum(0)), db=(dh.sum(0), dh.abs().sum(0)))


def ffn_reference(b):
    """zero_block_ffn's formulas in 64 bits: {name: (value, off)}. A sum over k
    terms passes through at most k + 64 roundings (the parts of a split one are
    added at the end); the activation's own error is 32 units and 4 |g|."""
    h, k = b.h.double(), b.h.shape[1]
    out = {}
    for name, w in (("gate", b.w_gate.double()), ("up", b.w_up.double())):
        out[name] = (h @ w.t().contiguous(), (k + 64) * U * (h.abs() @ w.abs().t().contiguous()))
    (g, og), (u, ou) = out["gate"], out["up"]
    f = act64(b.act, g)[0]
    out["a"] = (f * u, 1.2 * og * (u.abs() + ou) + f.abs() * ou + (32 + 4 * g.abs()) * U * (g * u).abs())
    return out


def ffn_grad_reference(b, g, u, x):
    """zero_block_ffn_grad's formulas in 64 bits from the saved gate and up and
    the block's input x: {name: (value, sum of |terms|)}; the products are those
    of the stored dgate and dup."""
    da = b.da.double()
    f, d = act64(b.act, g)
    out = dict(dgate=(da * u * d, None), dup=(da * f, None), a=(f * u, (f * u).abs()))
    dg, du = b.dgate.double(), b.dup.double()
    if b.dh is not None:
        wg, wu = b.w_gate.double(), b.w_up.double()
        out["dh"] = (dg @ wg + du @ wu, dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    for name, t in (("dw_gate", dg.t().contiguous()), ("dw_up", du.t().contiguous())):
        if x is not None:
            out[name] = (t @ x, t.abs() @ x.abs())
    return out
