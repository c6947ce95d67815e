"""The residual add and the layer norm, forward and backward, on the GPU,
against the plain 64-bit formulas: every combination of operands, odd sizes and
strides, wide rows, rows far from 0, saved rows in 8 bits and as they are,
differences of the forward pass, non-finite rows, streams and captured graphs."""
import itertools

import pytest
import torch

import sharded_optimizer_step_amd as z
from block_cases import FORMATS, U, assert_within, canary_ok, decode_act8, round_act8, strided
from ffn_cases import assert_close, assert_saved_within, layer_norm_grad_reference, layer_norm_reference

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ROW = 64 * U  # roundings of a row's sums and of what is made of them


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


def rnd(g, *shape, dtype=F32, scale=1.0, mean=0.0):
    return (mean + scale * torch.randn(*shape, device="cuda", generator=g)).to(dtype)


class Placed:
    """Operands as views of padded buffers, whose rest must stay as it was."""

    def __init__(self, pad, offset):
        self.pad, self.offset, self.bufs = pad, offset, []

    def __call__(self, t):
        if t is None:
            return None
        v, b = strided(t, self.pad, self.offset)
        self.bufs.append((b, *t.shape))
        return v

    def check(self):
        for buf, rows, cols in self.bufs:
            assert canary_ok(buf, rows, cols, self.pad, self.offset)


def forward(rows, cols, *, add=True, w=True, b=True, resid=BF16, weights=BF16, fmt="e4m3", seed=1, saves=True, pad=0, offset=0,
            eps=1e-5, mean=0.5):
    g, place = gen(seed), Placed(pad, offset)
    new = lambda t: torch.zeros(rows, cols, dtype=t, device="cuda")  # noqa: E731
    n = z.LayerNorm(
        x=place(rnd(g, rows, cols, dtype=resid, scale=2, mean=mean)), y=place(rnd(g, rows, cols, dtype=BF16, scale=3)) if add else None,
        w=rnd(g, cols, dtype=weights, scale=0.1, mean=1) if w else None, b=rnd(g, cols, dtype=weights) if b else None,
        x_out=place(new(resid)) if add else None, h=place(new(BF16)), mean=torch.zeros(rows, device="cuda"),
        rstd=torch.zeros(rows, device="cuda"), ckpt_xn=z.new_act8(rows, cols, FORMATS[fmt]) if saves else None,
        ckpt_h=z.new_act8(rows, cols, FORMATS[fmt]) if saves else None, eps=eps)
    z.zero_layer_norm(n)
    return n, place


def check_forward(n, where=""):
    x = n.x
    if n.y is not None:
        assert_close(n.x_out, n.x.double() + n.y.double(), U * (n.x.double().abs() + n.y.double().abs()), where)
        x = n.x_out
    ref = layer_norm_reference(n, x)
    for name in ("mean", "rstd", "h"):
        if getattr(n, name) is not None:
            assert_close(getattr(n, name), *ref[name], (where, name))
    for ck, name in ((n.ckpt_xn, "xn"), (n.ckpt_h, "h")):
        if ck is not None:
            assert_saved_within(ck, *ref[name], (where, name))


SIZES = [(1, 1), (2, 7), (3, 8), (5, 31), (1, 32), (7, 33), (65, 64), (3, 511), (5, 512), (4, 513), (130, 768), (3, 1025),
         (5, 2049), (3, 4096), (33, 5003), (2, 8192), (3, 8193), (2, 11008), (2, 16384)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("resid", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, resid, fmt):
    for add, weights in itertools.product((True, False), (BF16, F32)):
        check_forward(forward(rows, cols, add=add, resid=resid, weights=weights, fmt=fmt, seed=rows * cols)[0], (add, weights))


@pytest.mark.parametrize("add,w,b,saves", itertools.product((True, False), repeat=4))
def test_forward_operands(add, w, b, saves):
    n, place = forward(37, 331, add=add, w=w, b=b, saves=saves, pad=3, offset=1, fmt="int8")
    check_forward(n)
    place.check()


@pytest.mark.parametrize("cols", [100, 4096, 12000])
@pytest.mark.parametrize("mean", [1e4, -3e5])
def test_rows_far_from_zero_keep_their_variance(cols, mean):
    # a spread of 2 at 1e4 and more: squares summed from 0 would have lost it in fp32
    check_forward(forward(9, cols, resid=F32, add=False, mean=mean, w=False, b=False)[0])


@pytest.mark.parametrize("cols", [64, 1000, 9000])
def test_rows_of_equal_values_give_the_bias(cols):
    g = gen(cols)
    x = torch.full((4, cols), 0.7, device="cuda")
    b, h = rnd(g, cols, dtype=BF16), torch.zeros(4, cols, dtype=BF16, device="cuda")
    mean, rstd = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    z.zero_layer_norm(z.LayerNorm(x=x, b=b, h=h, mean=mean, rstd=rstd, eps=1e-5))
    # a mean that is off by 84 units of 0.7 is taken 1 / sqrt(eps) times
    assert_close(h, b.double().expand(4, cols), torch.full((4, cols), 84 * U * 0.7 * 317, dtype=torch.float64))
    assert_close(mean, torch.full((4,), float(x[0, 0]), dtype=torch.float64), torch.full((4,), 84 * U, dtype=torch.float64))
    assert torch.isfinite(rstd).all() and float(rstd.max()) <= 317


@pytest.mark.parametrize("cols", [40, 700, 9000])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_nonfinite_rows_stay_to_themselves(cols, value):
    n, _ = forward(6, cols, add=False, resid=F32)
    n.x[2, cols // 2] = value
    z.zero_layer_norm(n)
    assert torch.isnan(n.h[2]).all() and torch.isnan(torch.tensor(decode_act8(n.ckpt_xn)[0][2])).all()
    ref = layer_norm_reference(n, n.x)
    keep = [0, 1, 3, 4, 5]
    assert_close(n.h[keep], ref["h"][0][keep], ref["h"][1][keep])


def test_forward_in_place():
    n, _ = forward(50, 600)
    x = n.x.clone()
    want = [t.clone() for t in (n.x_out, n.h, n.mean, n.rstd)]
    n.x, n.x_out = x, x
    z.zero_layer_norm(n)
    for a, b in zip(want, (n.x_out, n.h, n.mean, n.rstd)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ backward

def backward(rows, cols, *, coded=True, dx_out=True, w=True, resid=BF16, weights=BF16, grad=F32, accumulate=True, dy=True, dw=True,
             db=True, fmt="e4m3", seed=1, pad=0, offset=0):
    g, place = gen(seed), Placed(pad, offset)
    new = lambda t: torch.zeros(rows, cols, dtype=t, device="cuda")  # noqa: E731
    x = rnd(g, rows, cols, dtype=resid, scale=2, mean=0.5)
    ck = None
    if coded:
        ck = z.new_act8(rows, cols, FORMATS[fmt])
        z.zero_act8_save(rnd(g, rows, cols), ck)
    n = z.LayerNormGrad(
        dx=place(new(resid)), dh=place(rnd(g, rows, cols, dtype=BF16)), dx_out=place(rnd(g, rows, cols, dtype=resid)) if dx_out else None,
        w=rnd(g, cols, dtype=weights, scale=0.1, mean=1) if w else None, x_out=None if coded else place(x),
        mean=None if coded else x.float().mean(1), rstd=1 / x.float().std(1, correction=0).clamp(min=0.1), ckpt_xn=ck,
        dy=place(new(BF16)) if dy else None, dw=rnd(g, cols, dtype=grad) if dw else None, db=rnd(g, cols, dtype=grad) if db else None)
    xn = torch.tensor(decode_act8(ck)[0], device="cuda") if coded else (x.double() - n.mean.double()[:, None]) * n.rstd.double()[:, None]
    old = {k: getattr(n, k).double().clone() if accumulate else 0.0 for k in ("dw", "db") if getattr(n, k) is not None}
    z.zero_layer_norm_grad(n, z.GRAD_ACCUMULATE if accumulate else 0, z.workspace(z.zero_layer_norm_grad_workspace_bytes(rows, cols)))
    return n, place, xn, old


def check_backward(n, place, xn, old, where=""):
    ref = layer_norm_grad_reference(n, xn)
    rows = xn.shape[0]
    assert_within(n.dx, *ref["dx"], ROW, (where, "dx"))
    if n.dy is not None:
        assert_within(n.dy, *ref["dy"], ROW, (where, "dy"))
    for k, o in old.items():
        want, mag = ref[k]
        assert_within(getattr(n, k), want + o, mag + (o.abs() if torch.is_tensor(o) else 0.0), (rows + 64) * U, (where, k))
    place.check()


@pytest.mark.parametrize("coded", [True, False])
@pytest.mark.parametrize("resid", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES + [(3000, 70), (5001, 520), (700, 9001)])
def test_backward(rows, cols, resid, coded):
    for weights, grad, accumulate, fmt in ((BF16, F32, True, "e4m3"), (F32, BF16, False, "int8"), (BF16, F32, False, "e4m3")):
        check_backward(*backward(rows, cols, coded=coded, resid=resid, weights=weights, grad=grad, accumulate=accumulate, fmt=fmt,
                                 seed=rows + cols), (weights, grad))


@pytest.mark.parametrize("dx_out,w,dy,dw,db", itertools.product((True, False), repeat=5))
def test_backward_operands(dx_out, w, dy, dw, db):
    for coded in (True, False):
        check_backward(*backward(41, 333, coded=coded, dx_out=dx_out, w=w, dy=dy, dw=dw, db=db, pad=3, offset=1))


def test_backward_in_place_and_without_rows():
    n, _, _, _ = backward(50, 600, accumulate=False)
    want = [t.clone() for t in (n.dx, n.dy, n.dw, n.db)]
    n.dx = n.dx_out
    ws = z.workspace(z.zero_layer_norm_grad_workspace_bytes(50, 600))
    z.zero_layer_norm_grad(n, 0, ws)
    for a, b in zip(want, (n.dx, n.dy, n.dw, n.db)):
        assert torch.equal(a, b)
    none = torch.zeros(0, 600, dtype=BF16, device="cuda")
    for flags in (z.GRAD_ACCUMULATE, 0):
        dw, db = torch.ones(600, device="cuda"), torch.ones(600, device="cuda")
        z.zero_layer_norm_grad(z.LayerNormGrad(dx=none, dh=none, rstd=torch.zeros(0, device="cuda"), dw=dw, db=db), flags)
        assert float(dw.sum()) == float(db.sum()) == (600 if flags else 0)


def test_backward_is_the_slope_of_forward():
    """Central differences of the forward formula in 64 bits, along random directions of x, w and b."""
    rows, cols = 5, 75
    g = gen(3)
    x, dh = rnd(g, rows, cols), rnd(g, rows, cols, dtype=BF16)
    w, b = rnd(g, cols, mean=1, scale=0.3), rnd(g, cols)
    h, mean, rstd = torch.zeros(rows, cols, dtype=BF16, device="cuda"), torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    z.zero_layer_norm(z.LayerNorm(x=x, w=w, b=b, h=h, mean=mean, rstd=rstd, eps=1e-5))
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
    z.zero_layer_norm_grad(z.LayerNormGrad(dx=dx, dh=dh, w=w, x_out=x, mean=mean, rstd=rstd, dw=dw, db=db), 0,
                           z.workspace(z.zero_layer_norm_grad_workspace_bytes(rows, cols)))

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return ((c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + b) * dh.double()).sum()

    at = [t.double() for t in (x, w, b)]
    for k, grad in enumerate((dx, dw, db)):
        v = rnd(g, *grad.shape).double()
        step = [v * 1e-4 if i == k else 0.0 for i in range(3)]
        slope = (loss(*(a + s for a, s in zip(at, step))) - loss(*(a - s for a, s in zip(at, step)))) / 2e-4
        # the difference's own error is of the order of step^2, the gradient's that of fp32 sums
        assert abs(float(slope - (grad.double() * v).sum())) <= 1e-5 * float((grad.double() * v).abs().sum())


# ------------------------------------------------------------------ how calls are made

def test_streams_and_two_calls_at_once():
    a, b = backward(300, 900, seed=1, accumulate=False)[0], backward(301, 900, seed=2, accumulate=False)[0]
    want = [t.clone() for n in (a, b) for t in (n.dx, n.dw, n.db)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [z.workspace(z.zero_layer_norm_grad_workspace_bytes(n.dx.shape[0], 900)) for n in (a, b)]
    for n in (a, b):
        for t in (n.dx, n.dw, n.db):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for n, s, ws in zip((a, b), streams, spaces):
            z.zero_layer_norm_grad(n, 0, ws, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(want, [t for n in (a, b) for t in (n.dx, n.dw, n.db)]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("cols", [600, 9000])
def test_captured_graph(cols):
    rows = 200
    n, _ = forward(rows, cols, resid=F32)
    g = z.LayerNormGrad(dx=torch.zeros(rows, cols, device="cuda"), dh=n.h, rstd=n.rstd, w=n.w, ckpt_xn=n.ckpt_xn,
                        dw=torch.zeros(cols, device="cuda"), db=torch.zeros(cols, device="cuda"))
    ws = z.workspace(z.zero_layer_norm_grad_workspace_bytes(rows, cols))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_layer_norm(n)
        z.zero_layer_norm_grad(g, 0, ws)
    for seed in range(4):
        n.x.copy_(rnd(gen(seed), rows, cols))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (n.h, n.mean, n.x_out, g.dx, g.dw, g.db)]
        z.zero_layer_norm(n)
        z.zero_layer_norm_grad(g, 0, ws)
        for a, b in zip(got, (n.h, n.mean, n.x_out, g.dx, g.dw, g.db)):
            assert torch.equal(a, b)
        check_forward(n, seed)


# bf16 rows, whose first means have 16 bits, and rows of all sizes at once
@pytest.mark.parametrize("kind", ["far", "one off", "two values", "tiny among large", "all sizes", "equal"])
@pytest.mark.parametrize("cols", [7, 100, 512, 513, 4096, 5003, 12000])
def test_bf16_rows_far_from_zero_and_of_all_sizes(cols, kind):
    g, rows = gen(cols), 17
    x = rnd(g, rows, cols)
    if kind == "far":
        x = x + 300 * torch.arange(1, rows + 1, device="cuda")[:, None]
    elif kind == "one off":  # the least variance that unequal values have
        x = torch.full((rows, cols), 255.0, device="cuda")
        x[:, cols // 2] = 254.0
    elif kind == "two values":
        x = 1000 + 8 * (x > 0).float()
    elif kind == "tiny among large":
        x = torch.where(x > 1, 1e-6 * x, 77 + x)
    elif kind == "all sizes":
        x = x * 2.0**torch.randint(-30, 30, x.shape, device="cuda", generator=g)
    else:
        x = torch.full((rows, cols), 0.7, device="cuda")
    new = lambda t: torch.zeros(rows, cols, dtype=t, device="cuda")  # noqa: E731
    n = z.LayerNorm(x=x.to(BF16), h=new(BF16), mean=torch.zeros(rows, device="cuda"), rstd=torch.zeros(rows, device="cuda"),
                    ckpt_xn=z.new_act8(rows, cols, z.ACT8_E4M3), eps=1e-5)
    z.zero_layer_norm(n)
    if kind != "equal":
        check_forward(n, kind)
    else:  # the mean's bound is taken 1 / sqrt(eps) times
        assert float(n.h.float().abs().max()) <= 84 * U * 0.71 * 317
        assert_close(n.mean, n.x[:, 0].double(), torch.full((rows,), 84 * U, dtype=torch.float64))


def test_saved_codes_are_those_of_64_bits():
    """A code differs only where the value lies within its error of the middle
    of two codes. That error is taken at 4 units of 2^-24, roundings of fp32 sums
    being spread evenly; the middles of e4m3 lie 2^-4 of the value apart at the
    least, so of evenly spread values at most 2 * 4 * 2^-24 / 2^-4 = 2^-17 have
    another code; and as many again where the largest value of a block of 32 does
    and moves their common unit."""
    rows, cols = 2048, 4096
    n = forward(rows, cols)[0]
    got = torch.tensor(decode_act8(n.ckpt_xn)[0])
    want = torch.tensor(round_act8(layer_norm_reference(n, n.x_out)["xn"][0].cpu().numpy(), z.ACT8_E4M3))
    assert int((got != want).sum()) <= 2.0**-17 * rows * cols * 2
