"""The gated feed-forward block, forward and backward, on the GPU, against the
plain 64-bit formulas: every activation, sizes from one row and column up and
around every tile edge, strides and alignments, saved rows and the input in 8
bits and as they are, absent operands, rounding of the stored gradients,
non-finite values, differences of the forward pass, streams and captured
graphs."""
import pytest
import torch

import sharded_optimizer_step_amd as z
from block_cases import FORMATS, U, assert_within, canary_ok, decode_act8, strided
from ffn_cases import ACTS, act64, assert_close, assert_saved_within, ffn_grad_reference, ffn_reference, nearest_bf16

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


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


def rnd(g, *shape, dtype=BF16, scale=1.0, mean=0.0):
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


def forward(rows, cols, hidden, *, act="silu", saved="raw", fmt="e4m3", seed=1, pad=0, offset=0):
    g, place = gen(seed), Placed(pad, offset)
    new = lambda: place(torch.zeros(rows, hidden, dtype=BF16, device="cuda"))  # noqa: E731
    b = z.BlockFfn(h=place(rnd(g, rows, cols)), w_gate=place(rnd(g, hidden, cols, scale=max(cols, 1)**-0.5)),
                   w_up=place(rnd(g, hidden, cols, scale=max(cols, 1)**-0.5)), a=new(), act=ACTS[act])
    if saved == "raw":
        b.gate, b.up = new(), new()
    elif saved == "8bit":
        b.ckpt_gate, b.ckpt_up = z.new_act8(rows, hidden, FORMATS[fmt]), z.new_act8(rows, hidden, FORMATS[fmt])
    z.zero_block_ffn(b, z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols, hidden)))
    return b, place


def check_forward(b, place, where=""):
    ref = ffn_reference(b)
    assert_close(b.a, *ref["a"], (where, "a"))
    for name in ("gate", "up"):
        if getattr(b, name) is not None:
            assert_close(getattr(b, name), *ref[name], (where, name))
        if getattr(b, "ckpt_" + name) is not None:
            assert_saved_within(getattr(b, "ckpt_" + name), *ref[name], (where, name))
    place.check()


# one row, column and element; around the edges of units, blocks, steps and tiles; split sums; several tiles
SIZES = [(1, 1, 1), (1, 8, 8), (2, 7, 33), (3, 64, 31), (16, 32, 64), (1, 4096, 512), (5, 100, 130), (64, 72, 136), (33, 65, 127),
         (127, 200, 128), (128, 64, 64), (129, 136, 264), (255, 63, 72), (256, 128, 256), (257, 192, 257), (300, 1000, 500),
         (64, 2048, 768), (513, 328, 1032), (1025, 776, 640)]


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 16), (3, 1)])
@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_forward(rows, cols, hidden, pad, offset):
    for k, (act, saved) in enumerate((("silu", "raw"), ("gelu", "8bit"), ("gelu_tanh", "none"))):
        b, place = forward(rows, cols, hidden, act=act, saved=saved, fmt=list(FORMATS)[rows % 2], seed=rows + cols + hidden + k, pad=pad,
                           offset=offset)
        check_forward(b, place, (act, saved))


@pytest.mark.parametrize("rows,cols,hidden", [(2000, 512, 4500), (4200, 264, 2200), (1100, 776, 2048), (4096, 2056, 4360), (50, 4096, 5000)])
def test_forward_of_large_tiles(rows, cols, hidden):
    for saved in ("raw", "8bit"):
        check_forward(*forward(rows, cols, hidden, saved=saved, act="gelu_tanh", fmt="int8"))


def test_forward_without_columns_or_rows():
    b, _ = forward(3, 0, 40)
    assert float(b.a.abs().max()) == float(b.gate.abs().max()) == float(b.up.abs().max()) == 0.0
    forward(0, 16, 40)
    forward(3, 16, 0)


def test_forward_keeps_nonfinite_rows_to_themselves():
    b, _ = forward(140, 96, 200)
    b.h[7, 3], b.h[130, 95] = float("inf"), float("nan")
    z.zero_block_ffn(b, z.workspace(z.zero_block_ffn_workspace_bytes(140, 96, 200)))
    bad = torch.zeros(140, dtype=torch.bool, device="cuda")
    bad[[7, 130]] = True
    assert torch.isfinite(b.a[~bad].float()).all() and torch.isfinite(b.gate[~bad].float()).all()
    assert not torch.isfinite(b.gate[bad].float()).any() and not torch.isfinite(b.up[bad].float()).any()


@pytest.mark.parametrize("act", ACTS)
def test_activation_of_large_and_small_values(act):
    # one column: gate is the weight itself, up is 1
    v = torch.tensor([0.0, 1e-30, -1e-30, 1e-6, -1e-6, 0.5, -0.5, 3, -3, 10, -10, 40, -40, 87, -87, 90, -90, 300, -300, 1e4, -1e4, 1e30, -1e30],
                     device="cuda").to(BF16)
    n = len(v)
    one = torch.ones(1, 1, dtype=BF16, device="cuda")
    a = torch.zeros(1, n, dtype=BF16, device="cuda")
    b = z.BlockFfn(h=one, w_gate=v.view(n, 1), w_up=one.expand(n, 1).contiguous(), a=a, act=ACTS[act])
    z.zero_block_ffn(b, z.workspace(z.zero_block_ffn_workspace_bytes(1, 1, n)))
    want = act64(ACTS[act], v.double())[0]
    # below -9 the exact values of the two forms of gelu, and below -87 those of silu, are of no size beside fp32's steps of |g|
    assert_close(a[0], want, (32 + 4 * v.double().abs().clamp(max=100)) * U * v.double().abs().clamp(max=100) + 1e-30)


# ------------------------------------------------------------------ backward

def backward(rows, cols, hidden, *, act="silu", saved="8bit", input="raw", fmt="e4m3", grad=F32, accumulate=True, dh=True, dw="gu",
             again=False, scale=True, seed=1, pad=0, offset=0, halves=False):
    g, place = gen(seed), Placed(pad, offset)
    new = lambda c: place(torch.zeros(rows, c, dtype=BF16, device="cuda"))  # noqa: E731

    def coded(t):
        ck = z.new_act8(*t.shape, FORMATS[fmt])
        z.zero_act8_save(t, ck)
        return ck, torch.tensor(decode_act8(ck)[0], device="cuda")

    b = z.BlockFfnGrad(da=place(rnd(g, rows, hidden)), dgate=new(hidden), dup=new(hidden), act=ACTS[act])
    if halves:  # of one buffer of rows x 2 hidden
        both = torch.zeros(rows, 2 * hidden, dtype=BF16, device="cuda")
        b.dgate, b.dup = both[:, :hidden], both[:, hidden:]
    gate, up = rnd(g, rows, hidden), rnd(g, rows, hidden)
    if saved == "raw":
        b.gate, b.up = place(gate), place(up)
        gate, up = gate.double(), up.double()
    else:
        (b.ckpt_gate, gate), (b.ckpt_up, up) = coded(gate), coded(up)
    if dh:
        b.w_gate, b.w_up, b.dh = place(rnd(g, hidden, cols)), place(rnd(g, hidden, cols)), new(cols)
    x = None
    if dw:
        x = rnd(g, rows, cols)
        if input == "raw":
            b.h = place(x)
            x = x.double()
        else:
            b.ckpt_h, x = coded(x)
            if scale:
                b.col_scale = rnd(g, cols, mean=1, scale=0.1)
                x = x * b.col_scale.double()
        if "g" in dw:
            b.dw_gate = place(rnd(g, hidden, cols, dtype=grad))
        if "u" in dw:
            b.dw_up = place(rnd(g, hidden, cols, dtype=grad))
    if again:
        b.ckpt_a = z.new_act8(rows, hidden, FORMATS[fmt])
    old = {k: getattr(b, k).double().clone() for k in ("dw_gate", "dw_up") if getattr(b, k) is not None}
    z.zero_block_ffn_grad(b, z.GRAD_ACCUMULATE if accumulate else 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden)))
    return b, place, gate, up, x, old if accumulate else {k: torch.zeros_like(t) for k, t in old.items()}


def check_backward(b, place, gate, up, x, old, where=""):
    ref = ffn_grad_reference(b, gate, up, x)
    rows, hidden = gate.shape
    for k in ("dgate", "dup"):
        # 64-bit formulas differ by a few 2^-52, which does not reach a bf16 border
        wrong = int((getattr(b, k).double() != nearest_bf16(ref[k][0])).sum())
        assert wrong == 0, (where, k, wrong)
    if b.dh is not None:
        assert_within(b.dh, *ref["dh"], (2 * hidden + 64) * U, (where, "dh"))
    for k, o in old.items():
        want, mag = ref[k]
        assert_within(getattr(b, k), want + o, mag + o.abs(), 2 * (rows + 64) * U, (where, k))
    if b.ckpt_a is not None:
        want, mag = ref["a"]
        # the activation within 40 + 2 g^2 units or 8 + 7 |z|, z <= 1.6 (|g| + 0.05 |g|^3)
        assert_saved_within(b.ckpt_a, want, mag * (64 + 16 * gate.abs() + gate.abs()**3) * U, (where, "a"))
    place.check()


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 16), (3, 1)])
@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_backward(rows, cols, hidden, pad, offset):
    for k, (act, saved, inp, grad, acc) in enumerate((("silu", "8bit", "raw", F32, True), ("gelu", "raw", "8bit", F32, False),
                                                      ("gelu_tanh", "raw", "raw", BF16, False))):
        r = backward(rows, cols, hidden, act=act, saved=saved, input=inp, grad=grad, accumulate=acc, fmt=list(FORMATS)[rows % 2],
                     again=k == 1, seed=rows + cols + hidden + k, pad=pad, offset=offset)
        check_backward(*r, (act, saved, inp))


@pytest.mark.parametrize("rows,cols,hidden", [(2000, 2104, 1544), (1100, 1000, 5000), (5000, 72, 136), (3000, 2304, 4360), (700, 4096, 3000),
                                              (4099, 776, 2056), (50, 2048, 6000)])
def test_backward_of_large_tiles(rows, cols, hidden):
    check_backward(*backward(rows, cols, hidden, act="gelu_tanh", halves=True, again=True))
    check_backward(*backward(rows, cols, hidden, saved="raw", grad=BF16, accumulate=False))


@pytest.mark.parametrize("dh,dw", [(True, ""), (False, "gu"), (False, ""), (True, "g"), (False, "u")])
@pytest.mark.parametrize("inp,scale", [("raw", False), ("8bit", True), ("8bit", False)])
def test_backward_operands(dh, dw, inp, scale):
    check_backward(*backward(70, 90, 110, dh=dh, dw=dw, input=inp, scale=scale, again=True, fmt="int8"))


def test_operands_with_strides_of_their_own():
    """Weights and gradients whose two halves lie differently: no common offsets, and one of them unaligned."""
    for other in (16, 3):
        r = backward(300, 264, 520, saved="raw", accumulate=False)
        b, place = r[0], Placed(other, 0)
        b.w_up, b.dup, b.dw_up = place(b.w_up), place(b.dup), place(b.dw_up)
        z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(300, 264, 520)))
        check_backward(b, place, *r[2:])
        f, place = forward(300, 264, 520)
        own = Placed(other, 0)
        f.w_up, f.up = own(f.w_up), own(f.up)
        z.zero_block_ffn(f, z.workspace(z.zero_block_ffn_workspace_bytes(300, 264, 520)))
        check_forward(f, own)


def test_rows_far_apart():
    """Row strides beyond what 32-bit offsets reach over a tile."""
    ld, g = (1 << 22) + 8, gen(2)
    wide = torch.zeros(40, ld, dtype=BF16, device="cuda")
    h = wide[:, :72]
    h.copy_(rnd(g, 40, 72))
    f = z.BlockFfn(h=h, w_gate=rnd(g, 96, 72, scale=0.1), w_up=rnd(g, 96, 72, scale=0.1), a=torch.zeros(40, 96, dtype=BF16, device="cuda"))
    z.zero_block_ffn(f, z.workspace(z.zero_block_ffn_workspace_bytes(40, 72, 96)))
    check_forward(f, Placed(0, 0))
    dw = torch.zeros(96, 72, device="cuda")
    b = z.BlockFfnGrad(da=rnd(g, 40, 96), dgate=torch.zeros(40, 96, dtype=BF16, device="cuda"), dup=torch.zeros(40, 96, dtype=BF16, device="cuda"),
                       gate=rnd(g, 40, 96), up=rnd(g, 40, 96), h=h, dw_gate=dw)
    z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(40, 72, 96)))
    check_backward(b, Placed(0, 0), b.gate.double(), b.up.double(), h.double(), dict(dw_gate=torch.zeros_like(dw).double()))


def test_tensors_of_more_than_32_bits_of_bytes():
    """The last rows of operands of 4.3 GB and more."""
    rows, cols, hidden, g = (1 << 17) + 5, 64, 16640, gen(7)
    last = slice(rows - 5, rows)
    f = z.BlockFfn(h=rnd(g, rows, cols), w_gate=rnd(g, hidden, cols, scale=0.125), w_up=rnd(g, hidden, cols, scale=0.125),
                   a=torch.zeros(rows, hidden, dtype=BF16, device="cuda"), gate=torch.zeros(rows, hidden, dtype=BF16, device="cuda"))
    assert f.a.numel() * 2 > 1 << 32
    z.zero_block_ffn(f, z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols, hidden)))
    few = z.BlockFfn(h=f.h[last], w_gate=f.w_gate, w_up=f.w_up, a=f.a[last], gate=f.gate[last])
    check_forward(few, Placed(0, 0))
    b = z.BlockFfnGrad(da=f.a, dgate=torch.zeros_like(f.a), dup=torch.zeros_like(f.a), gate=f.gate, up=f.gate, w_gate=f.w_gate, w_up=f.w_up,
                       dh=torch.zeros_like(f.h))
    z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden)))
    few = z.BlockFfnGrad(da=b.da[last], dgate=b.dgate[last], dup=b.dup[last], w_gate=b.w_gate, w_up=b.w_up, dh=b.dh[last])
    check_backward(few, Placed(0, 0), f.gate[last].double(), f.gate[last].double(), None, {})


def test_backward_of_empty_sizes():
    for acc in (True, False):
        b = backward(0, 24, 40, accumulate=acc, saved="raw")[0]
        if not acc:
            assert float(b.dw_gate.abs().max()) == float(b.dw_up.abs().max()) == 0.0
    b = backward(5, 24, 0, saved="raw")[0]
    assert float(b.dh.abs().max()) == 0.0
    backward(5, 0, 40, saved="raw")


@pytest.mark.parametrize("act", ACTS)
def test_stored_gradients_are_the_nearest_values(act):
    """Every bf16 gate there is (finite, up to 2^100), so that none is left to the bounds of the fp32 form."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF16)
    gate = bits[torch.isfinite(bits) & (bits.abs() < 2.0**100)]
    n = gate.numel() // 64 * 64
    gate = gate[:n].view(64, -1).cuda()
    g = gen(9)
    up, da = rnd(g, *gate.shape), rnd(g, *gate.shape)
    b = z.BlockFfnGrad(da=da, dgate=torch.zeros_like(gate), dup=torch.zeros_like(gate), gate=gate, up=up, act=ACTS[act])
    z.zero_block_ffn_grad(b)
    f, d = act64(ACTS[act], gate.double())
    for got, want in ((b.dgate, da.double() * up.double() * d), (b.dup, da.double() * f)):
        # below 2^-120 the 64-bit formulas themselves lose digits (erfc's and the exponential's tails)
        sure = (want.abs() > 2.0**-120) | (want == 0)
        w = nearest_bf16(want)
        off = (got.double() != w) & sure
        # two 64-bit forms, each within some 2^-50 of itself and of the two terms of act', may lie on two sides of a border
        step = (got.double() - w).abs()[off] / w.abs()[off]
        assert int(off.sum()) <= 2 and (step.numel() == 0 or float(step.max()) <= 2.0**-7)
        assert (got.double()[~sure].abs() <= 2.0**-119).all()


def test_gradients_of_nothing_are_nothing():
    """Rows whose incoming gradient is 0 have gradients of 0 and add nothing."""
    r = backward(96, 64, 128, accumulate=False)
    b = r[0]
    b.da.zero_()
    z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(96, 64, 128)))
    for t in (b.dgate, b.dup, b.dh, b.dw_gate, b.dw_up):
        assert float(t.abs().max()) == 0.0


def test_nonfinite_gradients_reach_every_result():
    r = backward(96, 64, 128, accumulate=False)
    b = r[0]
    b.da[5, 9] = float("inf")
    z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(96, 64, 128)))
    assert not torch.isfinite(b.dgate[5, 9]) and not torch.isfinite(b.dup[5, 9])
    assert not torch.isfinite(b.dh[5].float()).any() and torch.isfinite(b.dh[4].float()).all()
    assert not torch.isfinite(b.dw_gate[9]).any() and torch.isfinite(b.dw_gate[8]).all()


@pytest.mark.parametrize("act", ACTS)
def test_backward_is_the_slope_of_forward(act):
    """Central differences of the forward formula in 64 bits, along random directions of h and both weights."""
    rows, cols, hidden = 9, 40, 72
    f, _ = forward(rows, cols, hidden, act=act)
    g = gen(4)
    da = rnd(g, rows, hidden)
    b = z.BlockFfnGrad(da=da, dgate=torch.zeros_like(da), dup=torch.zeros_like(da), gate=f.gate, up=f.up, w_gate=f.w_gate, w_up=f.w_up,
                       dh=torch.zeros_like(f.h), h=f.h, dw_gate=torch.zeros(hidden, cols, device="cuda"),
                       dw_up=torch.zeros(hidden, cols, device="cuda"), act=f.act)
    z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden)))

    def loss(h, wg, wu):
        return (act64(f.act, h @ wg.t().contiguous())[0] * (h @ wu.t().contiguous()) * da.double()).sum()

    at = [t.double() for t in (f.h, f.w_gate, f.w_up)]
    for k, grad in enumerate((b.dh, b.dw_gate, b.dw_up)):
        v = rnd(g, *grad.shape, dtype=F32).double()
        step = [v * 1e-4 if i == k else 0.0 for i in range(3)]
        slope = (loss(*(a + s for a, s in zip(at, step))) - loss(*(a - s for a, s in zip(at, step)))) / 2e-4
        # gate, up, dgate, dup and dh are each rounded to bf16 once: 5 half steps of the terms that they make
        wg, wu = f.w_gate.double().abs(), f.w_up.double().abs()
        dg, du = (da.double() * 1.2 * (f.up.double().abs() + 0.1)).abs(), (da.double() * (f.gate.double().abs() + 0.2)).abs()
        mag = (dg @ wg + du @ wu, dg.t().contiguous() @ at[0].abs(), du.t().contiguous() @ at[0].abs())[k]
        assert abs(float(slope - (grad.double() * v).sum())) <= 5 * 2.0**-8 * float((mag * v.abs()).sum())


# ------------------------------------------------------------------ how calls are made

def results(b):
    return [t for t in (b.dgate, b.dup, b.dh, b.dw_gate, b.dw_up) if t is not None]


def test_two_calls_at_once_on_two_streams():
    calls = [backward(500, 300, 700, seed=s, accumulate=False, saved="raw")[0] for s in (1, 2)]
    want = [[t.clone() for t in results(b)] for b in calls]
    spaces = [z.workspace(z.zero_block_ffn_grad_workspace_bytes(500, 300, 700)) for _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for b in calls:
        for t in results(b):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for b, ws, s in zip(calls, spaces, streams):
            z.zero_block_ffn_grad(b, 0, ws, stream=s)
    torch.cuda.synchronize()
    for b, w in zip(calls, want):
        assert all(torch.equal(x, y) for x, y in zip(results(b), w))


@pytest.mark.parametrize("rows,cols,hidden", [(3, 2048, 300), (400, 264, 520)])
def test_captured_graph(rows, cols, hidden):
    f, _ = forward(rows, cols, hidden)
    b = backward(rows, cols, hidden, saved="raw", accumulate=False)[0]
    b.gate, b.up, b.h, b.w_gate, b.w_up = f.gate, f.up, f.h, f.w_gate, f.w_up
    ws = z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols, hidden))
    wsb = z.workspace(z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_block_ffn(f, ws)
        z.zero_block_ffn_grad(b, 0, wsb)
    for seed in range(4):
        f.h.copy_(rnd(gen(seed), rows, cols))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in [f.a, f.gate, f.up] + results(b)]
        z.zero_block_ffn(f, ws)
        z.zero_block_ffn_grad(b, 0, wsb)
        assert all(torch.equal(x, y) for x, y in zip(got, [f.a, f.gate, f.up] + results(b)))


# ------------------------------------------------------------------ columns that are no multiple of 8

ODD = [(300, 767, 2049), (640, 767, 1001), (1000, 4093, 1001), (900, 1003, 1024), (900, 72, 2049), (2011, 1003, 2731), (16, 1003, 2731)]


def among_nans(t):
    """t as a view of rows that NaN follow and that lie at odd addresses."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + 5) + 9,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[1:1 + rows * (cols + 5)].view(rows, cols + 5)[:, :cols]
    v.copy_(t)
    return v


@pytest.mark.parametrize("rows,cols,hidden", ODD)
def test_what_lies_beyond_the_columns_counts_nothing(rows, cols, hidden):
    """Operands among NaN, and a workspace full of them."""
    f, place = forward(rows, cols, hidden)
    f.h, f.w_gate, f.w_up = among_nans(f.h), among_nans(f.w_gate), among_nans(f.w_up)
    ws = z.workspace(max(1, z.zero_block_ffn_workspace_bytes(rows, cols, hidden)))
    ws.fill_(255)
    z.zero_block_ffn(f, ws)
    check_forward(f, place)
    for dw in ("gu", "u"):
        r = backward(rows, cols, hidden, saved="raw", accumulate=False, dw=dw)
        b = r[0]
        for k in ("da", "gate", "up", "h", "w_gate", "w_up"):
            setattr(b, k, among_nans(getattr(b, k)))
        b.dgate, b.dup = among_nans(b.dgate), among_nans(b.dup)
        ws = z.workspace(max(1, z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden)))
        ws.fill_(255)
        z.zero_block_ffn_grad(b, 0, ws)
        check_backward(*r)


def test_odd_columns_in_a_captured_graph():
    test_captured_graph(640, 767, 1001)


def test_an_aligned_call_and_an_odd_one_agree():
    """One column of zeros more changes no sum."""
    rows, cols, hidden = 640, 767, 1000
    f, _ = forward(rows, cols, hidden)
    wide = lambda t: torch.nn.functional.pad(t, (0, 1))  # noqa: E731
    g = z.BlockFfn(h=wide(f.h), w_gate=wide(f.w_gate), w_up=wide(f.w_up), a=torch.zeros_like(f.a), act=f.act)
    z.zero_block_ffn(g, z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols + 1, hidden)))
    ref = ffn_reference(f)
    assert_close(g.a, *ref["a"])
    assert_close(f.a, *ref["a"])


# ------------------------------------------------------------------ what is saved

@pytest.mark.parametrize("saved", ["gate", "up", "ckpt_gate", "ckpt_up", "gate ckpt_up", "up ckpt_gate", "gate up ckpt_gate ckpt_up"])
@pytest.mark.parametrize("rows,cols,hidden", [(5, 100, 130), (257, 192, 257)])
def test_forward_saves_what_is_asked(rows, cols, hidden, saved):
    b, place = forward(rows, cols, hidden, saved="none")
    for k in saved.split():
        setattr(b, k, z.new_act8(rows, hidden) if "ckpt" in k else torch.zeros(rows, hidden, dtype=BF16, device="cuda"))
    z.zero_block_ffn(b, z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols, hidden)))
    check_forward(b, place, saved)
