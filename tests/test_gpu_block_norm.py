"""The norms around a block with gate and residual scale, forward and backward,
on the GPU, against the plain 64-bit formulas: every combination of operands,
odd sizes and strides, gates for every row, for some rows and for all, saved
rows in 8 bits and as they are, differences of the forward pass, non-finite
rows, streams and captured graphs."""
import dataclasses
import itertools

import numpy as np
import pytest
import torch

import sharded_optimizer_step_amd as z
from block_cases import (FORMATS, U, assert_saved, assert_within, canary_ok, decode_act8, grad_reference,
                         norm_reference, strided)

pytestmark = pytest.mark.gpu

# Roundings on the longest path of a row's sum: at most 16 terms in a lane (8
# columns, two vectors), 6 steps of the wave, 16 waves, and the terms' own.
# Wide rows sum 16384 columns over 1024 lanes.
ROW = 48 * U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z.lib()
    torch.cuda.set_device(0)
    yield


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, dtype=torch.float32, scale=1.0, mean=0.0):
    return (mean + scale * torch.randn(*shape, device="cuda", generator=g)).to(dtype)


def f64(a):
    return torch.tensor(a, device="cuda")


def forward(rows, cols, *, post=True, pre=True, y=True, gate_rows=0, resid=torch.bfloat16, weights=torch.bfloat16,
            fmt="e4m3", seed=1, saves=True, pad=0, offset=0, eps=1e-6, alpha=0.3):
    """One call with its operands as views of padded buffers; returns the operands and the canaries."""
    g = gen(seed)
    bufs = []

    def place(t):
        if t is None:
            return None
        v, b = strided(t, pad, offset)
        bufs.append((b, t.shape[0], t.shape[1]))
        return v

    new = lambda dtype: torch.zeros(rows, cols, dtype=dtype, device="cuda")  # noqa: E731
    post, gate_rows = post and y, gate_rows if y else 0
    b = z.BlockNorm(
        x=place(rnd(g, rows, cols, dtype=resid, scale=2)), y=place(rnd(g, rows, cols, dtype=torch.bfloat16, scale=3)) if y else None,
        w_post=rnd(g, cols, dtype=weights, scale=0.1, mean=1) if post else None,
        gate=place(rnd(g, -(-rows // gate_rows), cols, dtype=weights)) if gate_rows else None,
        w_pre=rnd(g, cols, dtype=weights, scale=0.1, mean=1) if pre else None,
        x_out=place(new(resid)) if y else None, h=place(new(torch.bfloat16)) if pre else None,
        rstd_post=torch.zeros(rows, device="cuda") if post else None, rstd_pre=torch.zeros(rows, device="cuda") if pre else None,
        ckpt_post=z.new_act8(rows, cols, FORMATS[fmt]) if saves and y else None,
        ckpt_pre=z.new_act8(rows, cols, FORMATS[fmt]) if saves and pre else None,
        gate_rows=gate_rows, residual_scale=alpha, eps=eps)
    z.zero_block_norm(b)
    return b, bufs


def check_forward(b, where=""):
    ref = norm_reference(b, b.x_out if b.y is not None else b.x)
    if b.y is not None:
        # the term: rstd, its row sum, and five products
        assert_within(b.x_out, ref["x_out"], ref["x_out_mag"], ROW + 8 * U, where)
    for name in ("post", "pre"):
        r = getattr(b, "rstd_" + name)
        if r is not None:
            # half a row sum's error, a sum, a root and a quotient
            assert_within(r, ref["rstd_" + name], ref["rstd_" + name], ROW / 2 + 4 * U, where)
        ck = getattr(b, "ckpt_" + name)
        if ck is not None:
            assert_saved(ck, ref["yn" if name == "post" else "xn"].cpu().numpy(), ROW, where)
    if b.w_pre is not None:
        assert_within(b.h, ref["h"], ref["h"].abs(), ROW / 2 + 8 * U, where)


SIZES = [(1, 1), (2, 7), (3, 8), (5, 31), (1, 32), (7, 33), (65, 64), (3, 511), (4, 513), (130, 768), (3, 1025), (2, 2047),
         (5, 2049), (3, 4096), (2, 4097), (33, 5003), (3, 6152), (2, 7001), (2, 8192), (3, 8193), (2, 11008), (2, 16384)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("resid", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, resid, fmt):
    for weights, gate_rows in ((torch.bfloat16, 0), (torch.float32, 1), (torch.bfloat16, 3), (torch.float32, rows + 5)):
        b, _ = forward(rows, cols, gate_rows=gate_rows, resid=resid, weights=weights, fmt=fmt, seed=rows * cols + gate_rows)
        check_forward(b, (weights, gate_rows))


@pytest.mark.parametrize("y,post,pre,gate_rows,saves", [c for c in itertools.product(
    (True, False), (True, False), (True, False), (0, 4), (True, False)) if c[0] or (c[2] and not c[1] and not c[3])])
def test_forward_operands(y, post, pre, gate_rows, saves):
    b, bufs = forward(37, 331, y=y, post=post, pre=pre, gate_rows=gate_rows, saves=saves, pad=3, offset=1, fmt="int8")
    check_forward(b)
    for buf, rows, cols in bufs:
        assert canary_ok(buf, rows, cols, 3, 1)


def integers_of_mean_square(g, count, mean, low, most):
    """count whole numbers, most of them in 0 .. low and none above `most`, whose squares sum to count * mean."""
    squares = {a * a + b * b: (a, b) for a in range(most + 1) for b in range(a + 1)}
    while True:
        n = [int(v) for v in torch.randint(0, low + 1, (count - 4,), generator=g)]
        rest = count * mean - sum(v * v for v in n)
        for half, (a, b) in squares.items():
            if rest - half in squares:
                n += [a, b, *squares[rest - half]]
                return torch.tensor(n)[torch.randperm(count, generator=g)]


@pytest.mark.parametrize("cols", [64, 800])
@pytest.mark.parametrize("fmt", FORMATS)
def test_forward_rounds_the_exact_quotient(fmt, cols):
    # The squares' mean is exactly 1 (and their sums whole numbers below 2^24 of one unit) and eps 2^-24, so the exact factor is 1 - 2^-25, whose nearest fp32 number is 1:
    # the fp32 products are the values themselves, many of them the middle of two codes, and the exact ones a hair
    # below, so each of those goes to the code nearer to zero. e4m3 codes have 4 bits: sixteenths from 16 to 31 have one
    # too many; int8 codes of blocks with a value over 127/128 are multiples of 1/64, the values of 1/128.
    g = torch.Generator().manual_seed(cols)
    unit, low, most = (16, 27, 31) if fmt == "e4m3" else (128, 221, 254)
    n = torch.stack([integers_of_mean_square(g, cols, unit * unit, low, most) for _ in range(5)])
    if fmt == "int8":
        assert bool((n.reshape(5, -1, 32).amax(2) > 127).all())
    sign = torch.where(torch.rand(n.shape, generator=g) < 0.5, -1, 1)
    down = torch.where(n > 16, n - n % 2, n) if fmt == "e4m3" else n - n % 2
    assert int((down != n).sum()) > n.numel() // 8
    want = (sign * down).double() / unit
    v = ((sign * n).double() / unit).to("cuda")
    one, out, h = (torch.ones(cols, device="cuda"), torch.empty(5, cols, device="cuda"),
                   torch.empty(5, cols, dtype=torch.bfloat16, device="cuda"))
    for where in ("pre", "post"):
        ck, rstd = z.new_act8(5, cols, FORMATS[fmt]), torch.empty(5, device="cuda")
        if where == "pre":
            b = z.BlockNorm(x=v.float(), w_pre=one, h=h, rstd_pre=rstd, ckpt_pre=ck, eps=2.0**-24)
        else:
            b = z.BlockNorm(x=torch.zeros(5, cols, device="cuda"), y=v.bfloat16(), w_post=one, x_out=out, rstd_post=rstd,
                            ckpt_post=ck, eps=2.0**-24)
        z.zero_block_norm(b)
        got = torch.empty(5, cols, device="cuda")
        z.zero_act8_load(ck, got)
        assert torch.equal(rstd.cpu(), torch.ones(5)), where
        assert torch.equal(got.double().cpu(), want), where


def test_forward_does_not_depend_on_what_it_saves():
    b, _ = forward(300, 1000, gate_rows=100)
    z.zero_block_norm(b)
    keep = [t.clone() for t in (b.x_out, b.h)]
    z.zero_block_norm(dataclasses.replace(b, ckpt_post=None, ckpt_pre=None, rstd_post=None, rstd_pre=None))
    assert torch.equal(keep[0], b.x_out) and torch.equal(keep[1], b.h)


@pytest.mark.parametrize("cols", [64, 800])
@pytest.mark.parametrize("fmt", FORMATS)
def test_forward_settles_ties_whatever_it_saves(fmt, cols):
    # As above: the fp32 product is the value itself, and the settled one is the
    # next fp32 number towards zero, in nearly every column. An fp32 residual of
    # zeros shows it as it is; h shows it where the product with a weight of
    # 1 + 3/256 is the middle of two bf16 numbers (the values that are powers of two).
    g = torch.Generator().manual_seed(cols)
    unit, low, most = (16, 27, 31) if fmt == "e4m3" else (128, 221, 254)
    n = torch.stack([integers_of_mean_square(g, cols, unit * unit, low, most) for _ in range(5)])
    v = (torch.where(torch.rand(n.shape, generator=g) < 0.5, -1, 1) * n).float() / unit
    settled = torch.nextafter(v, torch.zeros(()))
    assert int((settled != v).sum()) > 0.9 * v.numel()
    weight = 1 + 3.0 / 256
    h = (settled * weight).bfloat16()
    # the middle goes to the even number, 1 + 4/256, and what is below it to 1 + 2/256
    assert int((h != (v * weight).bfloat16()).sum()) >= v.numel() // 50
    x, one, w = v.to("cuda"), torch.ones(cols, device="cuda"), torch.full((cols,), weight, device="cuda")
    new = lambda t=torch.float32: torch.empty(5, cols, dtype=t, device="cuda")  # noqa: E731
    for saves in (True, False):
        ck, rstd = (z.new_act8(5, cols, FORMATS[fmt]), torch.empty(5, device="cuda")) if saves else (None, None)
        b = z.BlockNorm(x=torch.zeros_like(x), y=x.bfloat16(), w_post=one, x_out=new(), rstd_post=rstd, ckpt_post=ck, eps=2.0**-24)
        z.zero_block_norm(b)
        assert torch.equal(b.x_out.cpu(), settled), saves
        b = z.BlockNorm(x=x, w_pre=w, h=new(torch.bfloat16), rstd_pre=rstd, ckpt_pre=ck, eps=2.0**-24)
        z.zero_block_norm(b)
        assert torch.equal(b.h.cpu(), h), saves


def test_forward_in_place_and_nonfinite_rows():
    b, _ = forward(8, 200, resid=torch.float32)
    x = b.x.clone()
    x_out, h = b.x_out.clone(), b.h.clone()
    b.x_out = b.x
    z.zero_block_norm(b)
    assert torch.equal(b.x, x_out) and torch.equal(b.h, h)
    b.x, b.x_out = x, torch.zeros_like(x)
    b.y = b.y.clone()
    b.y[3, 5] = float("nan")
    b.x[6, 150] = float("inf")
    z.zero_block_norm(b)
    fine = [0, 1, 2, 4, 5, 7]
    assert torch.equal(b.h[fine], h[fine]) and torch.equal(b.x_out[fine], x_out[fine])
    assert torch.isnan(b.h[3]).all() and torch.isnan(f64(decode_act8(b.ckpt_pre)[0])[3]).all()
    assert torch.isnan(f64(decode_act8(b.ckpt_post)[0])[3]).all() and torch.isnan(b.h[6, 150])
    assert torch.isnan(f64(decode_act8(b.ckpt_pre)[0])[6, 128:160]).all()
    # rows of zeros, with and without eps
    b.y.zero_()
    b.x.zero_()
    z.zero_block_norm(b)
    assert float(b.h.abs().max()) == 0.0 and float(b.x_out.abs().max()) == 0.0
    assert torch.allclose(b.rstd_pre, torch.full_like(b.rstd_pre, 1e3))


@pytest.mark.parametrize("cols", [40, 700, 9000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_whose_squares_leave_the_range_of_fp32(dtype, cols):
    # rows 0 .. 2: large squares, one infinite element, one NaN; rows 3 and 4: squares that vanish, with a zero among
    # them; row 5: ordinary, near both ends of what a mean of squares can be
    x = torch.ones(6, cols, device="cuda")
    x[0] = -2.0**70
    x[1, 7] = float("inf")
    x[2, 11] = float("nan")
    x[3] = 2.0**-80
    x[4] = -2.0**-80
    x[4, 3] = 0.0
    for size in (2.0**55, 2.0**-55):
        x[5] = size
        x = x.to(dtype)
        r = torch.zeros(6, device="cuda")
        h, ck = torch.zeros(6, cols, dtype=torch.bfloat16, device="cuda"), z.new_act8(6, cols)
        z.zero_block_norm(z.BlockNorm(x=x, w_pre=torch.ones(cols, device="cuda"), h=h, rstd_pre=r, ckpt_pre=ck, eps=0.0))
        inf = float("inf")
        assert torch.equal(r[[0, 1, 3, 4, 5]], torch.tensor([0, 0, inf, inf, 1 / size], device="cuda")) and bool(r[2].isnan())
        assert not h[0].any() and bool(h[2].isnan().all()) and bool((h[3] == inf).all()) and bool((h[5] == 1).all())
        other = torch.arange(cols, device="cuda")
        assert bool(h[1, 7].isnan()) and not h[1][other != 7].any()
        assert bool(h[4, 3].isnan()) and bool((h[4][other != 3] == -inf).all())
        got = f64(decode_act8(ck)[0])
        assert not got[0].any() and bool(got[2:5].isnan().all()) and bool((got[5] == 1).all())
        assert bool(got[1, :32].isnan().all()) and not got[1, 32:].any()


# ------------------------------------------------------------------ backward

def backward(b, *, saved, grad=torch.float32, flags=0, dx_out=True, seed=7, pad=0, offset=0, wants=("dy", "dw_pre", "dw_post", "dgate")):
    """The backward call that belongs to a forward one; saved: which rows come from 8 bits."""
    g = gen(seed)
    rows, cols = b.x.shape
    bufs = []

    def place(t):
        v, buf = strided(t, pad, offset)
        bufs.append((buf, t.shape[0], t.shape[1]))
        return v

    pre, post, y = b.w_pre is not None, b.w_post is not None, b.y is not None
    G = b.gate.shape[0] if b.gate is not None else 0
    new = lambda r, t: place(rnd(g, r, cols, dtype=t))  # noqa: E731
    need = y and (post or (G and "dgate" in wants))
    d = z.BlockNormGrad(
        dx=new(rows, b.x.dtype), dx_out=place(rnd(g, rows, cols, dtype=b.x.dtype, scale=1e-2)) if dx_out or not pre else None,
        dh=place(rnd(g, rows, cols, dtype=torch.bfloat16, scale=1e-2)) if pre else None,
        w_post=b.w_post, gate=b.gate, w_pre=b.w_pre, rstd_pre=b.rstd_pre, rstd_post=b.rstd_post,
        dy=new(rows, torch.bfloat16) if y and "dy" in wants else None,
        dw_pre=new(1, grad) if pre and "dw_pre" in wants else None, dw_post=new(1, grad) if post and "dw_post" in wants else None,
        dgate=new(G, grad) if G and "dgate" in wants else None, gate_rows=b.gate_rows, residual_scale=b.residual_scale)
    xn = yn = None
    if pre:
        if "pre" in saved:
            d.ckpt_pre = b.ckpt_pre
            xn = f64(decode_act8(b.ckpt_pre)[0])
        else:
            d.x_out = b.x_out if y else b.x
            xn = d.x_out.double() * b.rstd_pre.double()[:, None]
    if need:
        if "post" in saved:
            d.ckpt_post = b.ckpt_post
            yn = f64(decode_act8(b.ckpt_post)[0])
        else:
            d.y = b.y
            yn = b.y.double() * (b.rstd_post.double()[:, None] if post else 1.0)
    old = {n: getattr(d, n).double().clone() for n in ("dw_pre", "dw_post", "dgate") if getattr(d, n) is not None}
    ref = grad_reference(d, xn, yn)
    n = z.zero_block_norm_grad_workspace_bytes(rows, cols, b.gate_rows if G else 0)
    ws = z.workspace(n)
    ws.fill_(0xFF)
    z.zero_block_norm_grad(d, flags, ws)
    # a row's three sums, and the products around them
    rel = 2 * ROW + 16 * U
    assert_within(d.dx, *ref["dx"], rel, "dx")
    if d.dy is not None:
        assert_within(d.dy, *ref["dy"], 2 * rel, "dy")
    for name, o in old.items():
        want, mag = ref[name]
        if flags:
            want, mag = want + o, mag + o.abs()
        assert_within(getattr(d, name), want, mag, 2 * rel + (rows + 64) * U, name)
    for buf, r, c in bufs:
        assert canary_ok(buf, r, c, pad, offset)
    return d


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("resid", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, resid, fmt):
    for weights, gate_rows, saved, grad, flags in (
            (torch.bfloat16, 0, ("pre", "post"), torch.bfloat16, 0), (torch.float32, 1, (), torch.float32, 0),
            (torch.bfloat16, 3, ("pre",), torch.float32, z.GRAD_ACCUMULATE),
            (torch.float32, rows + 5, ("post",), torch.bfloat16, 0),
            (torch.bfloat16, 1, ("pre", "post"), torch.float32, z.GRAD_ACCUMULATE)):
        b, _ = forward(rows, cols, gate_rows=gate_rows, resid=resid, weights=weights, fmt=fmt, seed=rows + cols)
        backward(b, saved=saved, grad=grad, flags=flags)


@pytest.mark.parametrize("rows,cols,gate_rows", [
    (5000, 96, 1), (5000, 96, 2), (4099, 96, 4099), (9001, 33, 2), (2000, 520, 7), (3001, 1200, 1), (1500, 2500, 3),
    (1500, 2500, 100), (1030, 4096, 1), (1030, 4096, 400), (700, 8200, 1), (700, 8200, 300), (300, 9000, 2), (2600, 64, 100)])
def test_backward_gates_and_splits(rows, cols, gate_rows):
    # units of a part of a gate row, of one, of several; the last gate row short
    b, _ = forward(rows, cols, gate_rows=gate_rows, seed=rows)
    backward(b, saved=("pre", "post"))
    backward(b, saved=(), grad=torch.bfloat16)


@pytest.mark.parametrize("y,post,pre,gate_rows,dx_out", [c for c in itertools.product(
    (True, False), (True, False), (True, False), (0, 1, 4), (True, False))
    if (c[0] or (c[2] and not c[1] and not c[3])) and (c[2] or c[4])])
def test_backward_operands(y, post, pre, gate_rows, dx_out):
    b, _ = forward(41, 331, y=y, post=post, pre=pre, gate_rows=gate_rows, fmt="int8", resid=torch.float32)
    for saved in (("pre", "post"), ()):
        backward(b, saved=saved, dx_out=dx_out, pad=3, offset=1)


@pytest.mark.parametrize("wants", [(), ("dy",), ("dw_pre",), ("dw_post",), ("dgate",), ("dw_pre", "dgate"), ("dw_post", "dgate")])
@pytest.mark.parametrize("gate_rows", [1, 4, 50])
def test_backward_of_some_gradients(wants, gate_rows):
    b, _ = forward(50, 200, gate_rows=gate_rows)
    backward(b, saved=("pre", "post"), wants=wants)


def test_backward_in_place():
    b, _ = forward(300, 1100, gate_rows=7)
    for cols in (1100,):
        d = backward(b, saved=("pre", "post"))
        want, dy = d.dx.clone(), d.dy.clone()
        d.dx.copy_(d.dx_out)
        d.dx_out = d.dx
        z.zero_block_norm_grad(d, 0, z.workspace(z.zero_block_norm_grad_workspace_bytes(300, cols, 7)))
        assert torch.equal(d.dx, want) and torch.equal(d.dy, dy)


def test_no_rows():
    for dtype in (torch.bfloat16, torch.float32):
        e = lambda t=torch.bfloat16: torch.empty(0, 40, dtype=t, device="cuda")  # noqa: E731
        one = lambda: torch.full((40,), 3.0, dtype=dtype, device="cuda")  # noqa: E731
        r = torch.empty(0, device="cuda")
        z.zero_block_norm(z.BlockNorm(x=e(), y=e(), w_post=one(), w_pre=one(), x_out=e(), h=e(), rstd_post=r, rstd_pre=r))
        d = z.BlockNormGrad(dx=e(), dx_out=e(), dh=e(), w_post=one(), w_pre=one(), x_out=e(), y=e(), rstd_pre=r, rstd_post=r,
                            dy=e(), dw_pre=one(), dw_post=one())
        z.zero_block_norm_grad(d, 0, z.workspace(z.zero_block_norm_grad_workspace_bytes(0, 40, 0)))
        assert float(d.dw_pre.abs().max()) == 0.0 and float(d.dw_post.abs().max()) == 0.0


def test_gradient_against_differences():
    """The directional derivative of L = sum(h * a) + sum(x_out * c) in 64 bits,
    by central differences of the plain formulas, against the kernels' gradients."""
    rows, cols, gate_rows = 6, 200, 2
    b, _ = forward(rows, cols, gate_rows=gate_rows, resid=torch.float32, weights=torch.float32, saves=False, eps=1e-3)
    g = gen(77)
    a, c = rnd(g, rows, cols, dtype=torch.bfloat16), rnd(g, rows, cols)
    new = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    d = z.BlockNormGrad(dx=new(rows, cols), dx_out=c, dh=a, w_post=b.w_post, gate=b.gate, w_pre=b.w_pre, x_out=b.x_out, y=b.y,
                        rstd_pre=b.rstd_pre, rstd_post=b.rstd_post, dy=new(rows, cols, t=torch.bfloat16), dw_pre=new(cols),
                        dw_post=new(cols), dgate=new(3, cols), gate_rows=gate_rows, residual_scale=b.residual_scale)
    z.zero_block_norm_grad(d, 0, z.workspace(z.zero_block_norm_grad_workspace_bytes(rows, cols, gate_rows)))
    alpha, eps = float(np.float32(b.residual_scale)), float(np.float32(b.eps))

    def loss(x, y, wp, gate, w):
        yn = y * (y.square().mean(1, keepdim=True) + eps).rsqrt()
        xo = x + alpha * gate.repeat_interleave(gate_rows, 0) * wp * yn
        h = w * xo * (xo.square().mean(1, keepdim=True) + eps).rsqrt()
        return float((h * a.double()).sum() + (xo * c.double()).sum())

    at = [t.double() for t in (b.x, b.y, b.w_post, b.gate, b.w_pre)]
    grads = [d.dx, d.dy, d.dw_post, d.dgate, d.dw_pre]
    for i, name in enumerate(("x", "y", "w_post", "gate", "w_pre")):
        way = torch.randn(at[i].shape, device="cuda", generator=g, dtype=torch.float64)
        step = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * way, at[i] - step * way
        want = (loss(*up) - loss(*down)) / (2 * step)
        terms = grads[i].double().reshape(at[i].shape) * way
        # dy is bf16: half a step a term; the rest is fp32. The difference itself is off by step^2 of third derivatives
        # of order 1 / cols^0.5 and the losses' own rounding, 2^-52 * 1e3 / step: both below 1e-6 of the terms
        bound = (2.0**-8 if name == "y" else 2.0**-16) * float(terms.abs().sum()) + 1e-6 * float(terms.abs().sum())
        assert abs(float(terms.sum()) - want) <= bound, (name, float(terms.sum()), want)


def test_nonfinite_gradients_stay_in_their_rows():
    b, _ = forward(12, 300, gate_rows=3)
    d = backward(b, saved=("pre", "post"))
    dx, dy, dgate = d.dx.clone(), d.dy.clone(), d.dgate.clone()
    d.dh[4, 17] = float("inf")
    z.zero_block_norm_grad(d, 0, z.workspace(z.zero_block_norm_grad_workspace_bytes(12, 300, 3)))
    keep = [r for r in range(12) if r != 4]
    assert torch.equal(d.dx[keep], dx[keep]) and torch.equal(d.dy[keep], dy[keep])
    assert torch.equal(d.dgate[[0, 2, 3]], dgate[[0, 2, 3]]) and (~torch.isfinite(d.dgate[1])).any()
    assert (~torch.isfinite(d.dx[4])).any() and (~torch.isfinite(d.dw_pre)).any()


def test_two_streams_and_repeats():
    b, _ = forward(900, 700, gate_rows=300)
    d0 = backward(b, saved=("pre", "post"))
    n = z.zero_block_norm_grad_workspace_bytes(900, 700, 300)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    kept = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            d = dataclasses.replace(d0, dx=torch.zeros_like(d0.dx), dy=torch.zeros_like(d0.dy), dw_pre=torch.zeros(700, device="cuda"),
                                    dw_post=torch.zeros(700, device="cuda"), dgate=torch.zeros(3, 700, device="cuda"))
            ws = z.workspace(n)
            z.zero_block_norm_grad(d, 0, ws)
            kept.append((d, ws))
    torch.cuda.synchronize()
    for d, _ in kept:
        for name in ("dx", "dy", "dgate"):
            assert torch.equal(getattr(d, name), getattr(d0, name)), name
        assert torch.equal(d.dw_pre, d0.dw_pre[0]) and torch.equal(d.dw_post, d0.dw_post[0])


@pytest.mark.parametrize("cols", [700, 8200])
def test_captured_and_replayed(cols):
    rows = 200
    b, _ = forward(rows, cols, gate_rows=60)
    d = backward(b, saved=("pre", "post"))
    ws, ws2 = (z.workspace(z.zero_block_norm_grad_workspace_bytes(rows, cols, 60)) for _ in range(2))

    def go(w):
        z.zero_block_norm(b)
        z.zero_block_norm_grad(d, z.GRAD_ACCUMULATE, w)

    go(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(ws)
    names = ("dx", "dy", "dw_pre", "dw_post", "dgate")
    for i in range(4):
        b.x.copy_(rnd(gen(50 + i), rows, cols, dtype=b.x.dtype, scale=2))
        start = {n: getattr(d, n).clone() for n in names}
        graph.replay()
        torch.cuda.synchronize()
        replayed = {n: getattr(d, n).clone() for n in names}
        h = b.h.clone()
        for n in names:
            getattr(d, n).copy_(start[n])
        go(ws2)
        torch.cuda.synchronize()
        assert torch.equal(b.h, h), i
        for n in names:
            assert torch.equal(getattr(d, n), replayed[n]), (n, i)


@pytest.mark.parametrize("resid,rows,cols", [(torch.bfloat16, 9000, 4096), (torch.float32, 6000, 4104), (torch.bfloat16, 1800, 16384)])
def test_large_calls_give_what_small_ones_do(resid, rows, cols):
    # a call that moves more than the caches hold reads and writes past them; its rows are independent of each other
    g = gen(11)
    x, y = rnd(g, rows, cols, dtype=resid), rnd(g, rows, cols, dtype=torch.bfloat16)
    w_post, w_pre = rnd(g, cols, dtype=torch.bfloat16), rnd(g, cols, dtype=torch.bfloat16)

    def go(lo, hi, in_place=False):
        n = hi - lo
        ck = [z.new_act8(n, cols), z.new_act8(n, cols)]
        src = x[lo:hi].clone() if in_place else x[lo:hi]
        out = src if in_place else torch.empty_like(src)
        h = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
        z.zero_block_norm(z.BlockNorm(x=src, y=y[lo:hi], w_post=w_post, w_pre=w_pre, x_out=out, h=h, ckpt_post=ck[0],
                                      ckpt_pre=ck[1], residual_scale=0.7))
        back = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
        z.zero_act8_load(ck[1], back)
        return out, h, back

    assert rows * cols * (2 * x.element_size() + 6) > 256 << 20
    whole = go(0, rows)
    for a, b in zip(whole, go(0, rows, in_place=True)):
        assert torch.equal(a, b)
    step = rows // 5 + 1
    for lo in range(0, rows, step):
        for a, b in zip(whole, go(lo, min(rows, lo + step))):
            assert torch.equal(a[lo:lo + step], b)


def test_offsets_past_32_bits():
    rows, cols, ld = 70, 300, 1 << 25
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    wide = lambda k: big.view(rows, ld)[:, 512 * k:512 * k + cols]  # noqa: E731
    b, _ = forward(rows, cols, gate_rows=9)
    far = z.BlockNorm(**{**b.__dict__, "x": wide(0), "y": wide(1), "x_out": wide(2), "h": wide(3)})
    far.x.copy_(b.x)
    far.y.copy_(b.y)
    z.zero_block_norm(far)
    assert torch.equal(far.x_out, b.x_out) and torch.equal(far.h, b.h)
    d = backward(b, saved=())
    e = z.BlockNormGrad(**{**d.__dict__, "dx": wide(4), "dx_out": wide(5), "dh": wide(6), "dy": wide(7), "x_out": far.x_out, "y": far.y})
    e.dx_out.copy_(d.dx_out)
    e.dh.copy_(d.dh)
    dw = d.dw_pre.clone()
    z.zero_block_norm_grad(e, 0, z.workspace(z.zero_block_norm_grad_workspace_bytes(rows, cols, 9)))
    assert torch.equal(e.dx, d.dx) and torch.equal(e.dy, d.dy) and torch.equal(e.dw_pre, dw)
