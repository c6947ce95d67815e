"""The layer norm and the gated feed-forward block used together, as a training
step uses them: a residual block forward with 8-bit checkpoints, backward over
two micro-batches into fp32 accumulators (the down projection's weight gradient
too), and the framework's own step from those gradients. Every stage is held to
its 64-bit formula on the tensors that it was given, and the new weights to the
CPU oracle on the same gradients. And a workspace that serves a step and these
calls in turn."""
import pytest
import torch

import oracle
import sharded_optimizer_step_amd as z
from block_cases import U, assert_within, decode_act8
from cases import assert_state_matches, hp_oracle, to_np_f32, to_np_u16
from ffn_cases import (assert_close, assert_saved_within, ffn_grad_reference, ffn_reference, layer_norm_grad_reference,
                       layer_norm_reference, nearest_bf16)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z.lib()
    torch.cuda.set_device(0)
    yield


def decoded(ck):
    return torch.tensor(decode_act8(ck)[0], device="cuda")


@pytest.mark.parametrize("fmt", [z.ACT8_E4M3, z.ACT8_INT8])
@pytest.mark.parametrize("resid", [BF16, F32])
@pytest.mark.parametrize("act,rows,cols,hidden", [(z.FFN_SILU, 70, 96, 264), (z.FFN_GELU, 513, 330, 700), (z.FFN_GELU_TANH, 300, 1000, 328)])
def test_a_block_and_a_step(act, rows, cols, hidden, resid, fmt):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    rnd = lambda *s, scale=1.0, mean=0.0, t=BF16: (mean + scale * torch.randn(*s, device="cuda", generator=g)).to(t)  # noqa: E731
    p = dict(w=rnd(cols, scale=0.1, mean=1), b=rnd(cols, scale=0.1), w_gate=rnd(hidden, cols, scale=cols**-0.5),
             w_up=rnd(hidden, cols, scale=cols**-0.5), w_down=rnd(cols, hidden, scale=hidden**-0.5))
    acc = {k: torch.zeros(v.shape, device="cuda") for k, v in p.items()}
    new = lambda c, t=BF16: torch.zeros(rows, c, dtype=t, device="cuda")  # noqa: E731
    ws = z.workspace(max(z.zero_layer_norm_grad_workspace_bytes(rows, cols), z.zero_block_ffn_workspace_bytes(rows, cols, hidden),
                         z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden), z.zero_act8_wgrad_workspace_bytes(rows, cols, hidden)))
    for _ in range(2):  # micro-batches
        x, y0 = rnd(rows, cols, t=resid), rnd(rows, cols)
        # forward: residual add and norm, block
        n = z.LayerNorm(x=x, y=y0, w=p["w"], b=p["b"], x_out=new(cols, resid), h=new(cols), rstd=torch.zeros(rows, device="cuda"),
                        ckpt_xn=z.new_act8(rows, cols, fmt), ckpt_h=z.new_act8(rows, cols, fmt))
        z.zero_layer_norm(n)
        ref = layer_norm_reference(n, n.x_out)
        assert_close(n.h, *ref["h"], "h")
        assert_saved_within(n.ckpt_xn, *ref["xn"], "xn")
        assert_saved_within(n.ckpt_h, *ref["h"], "saved h")
        f = z.BlockFfn(h=n.h, w_gate=p["w_gate"], w_up=p["w_up"], a=new(hidden), ckpt_gate=z.new_act8(rows, hidden, fmt),
                       ckpt_up=z.new_act8(rows, hidden, fmt), act=act)
        z.zero_block_ffn(f, ws)
        ref = ffn_reference(f)
        assert_close(f.a, *ref["a"], "a")
        assert_saved_within(f.ckpt_gate, *ref["gate"], "gate")
        # backward from the gradient of the stream and of the block's output
        d, dy = rnd(rows, cols, scale=1e-2, t=resid), rnd(rows, cols, scale=1e-2)
        da = (dy.float() @ p["w_down"].float()).bfloat16()
        old = {k: v.double().clone() for k, v in acc.items()}
        b = z.BlockFfnGrad(da=da, dgate=new(hidden), dup=new(hidden), ckpt_gate=f.ckpt_gate, ckpt_up=f.ckpt_up, w_gate=p["w_gate"],
                           w_up=p["w_up"], dh=new(cols), ckpt_h=n.ckpt_h, dw_gate=acc["w_gate"], dw_up=acc["w_up"],
                           ckpt_a=z.new_act8(rows, hidden, fmt), act=act)
        z.zero_block_ffn_grad(b, z.GRAD_ACCUMULATE, ws)
        ref = ffn_grad_reference(b, decoded(f.ckpt_gate), decoded(f.ckpt_up), decoded(n.ckpt_h))
        for k in ("dgate", "dup"):
            assert int((getattr(b, k).double() != nearest_bf16(ref[k][0])).sum()) == 0, k
        assert_within(b.dh, *ref["dh"], (2 * hidden + 64) * U, "dh")
        for k in ("dw_gate", "dw_up"):
            o = old[k.replace("dw", "w")]
            assert_within(getattr(b, k), ref[k][0] + o, ref[k][1] + o.abs(), 2 * (rows + 64) * U, k)
        z.zero_act8_wgrad(dy, b.ckpt_a, acc["w_down"], z.GRAD_ACCUMULATE, ws)
        a8, dyt, o = decoded(b.ckpt_a), dy.double().t().contiguous(), old["w_down"]
        assert_within(acc["w_down"], dyt @ a8 + o, dyt.abs() @ a8.abs() + o.abs(), 2 * (rows + 8) * U, "dw_down")
        r = z.LayerNormGrad(dx=new(cols, resid), dh=b.dh, rstd=n.rstd, dx_out=d, w=p["w"], ckpt_xn=n.ckpt_xn,
                            dy=new(cols), dw=acc["w"], db=acc["b"])
        z.zero_layer_norm_grad(r, z.GRAD_ACCUMULATE, ws)
        ref = layer_norm_grad_reference(r, decoded(n.ckpt_xn))
        assert_within(r.dx, *ref["dx"], 64 * U, "dx")
        assert_within(r.dy, *ref["dy"], 64 * U, "dy")
        for k in ("w", "b"):
            want, mag = ref["d" + k]
            assert_within(acc[k], want + old[k], mag + old[k].abs(), (rows + 64) * U, k)
    # the step: AdamW on each parameter from its fp32 gradient, and the same from the oracle
    hp = z.HParams(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3, max_grad_norm=1.0, grad_scale=1.0)
    for k, a in acc.items():
        master, m, v = p[k].float().flatten(), torch.zeros(a.numel(), device="cuda"), torch.zeros(a.numel(), device="cuda")
        start = [to_np_f32(t).copy() for t in (master, m, v)]
        res = z.new_result()
        z.zero_grad_check_norm(a.flatten(), hp, 0.0, z.workspace(z.zero_grad_check_norm_workspace_bytes(a.numel())), res)
        z.zero_adamw_step(master, m, v, a.flatten(), p[k].view(-1), hp, res)
        r = z.read_result(res)
        norm = float(a.double().norm())
        assert r["found_inf"] == 0 and abs(r["grad_norm"] - norm) <= 1e-5 * norm
        after = oracle.adamw(*start, to_np_f32(a.flatten()), hp_oracle(hp), r["clip_coef"])
        assert_state_matches(to_np_f32(master), to_np_f32(m), to_np_f32(v), to_np_u16(p[k].view(-1)), *after, where=k)


def test_nonfinite_rows_skip_the_step():
    """An inf in the stream reaches the weight gradient, its flag and the skip, and no other row's gradients."""
    rows, cols, hidden = 64, 96, 128
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    x[9, 40] = float("inf")
    new = lambda c: torch.zeros(rows, c, dtype=BF16, device="cuda")  # noqa: E731
    h, w = new(cols), [torch.randn(hidden, cols, device="cuda").bfloat16() for _ in range(2)]
    z.zero_layer_norm(z.LayerNorm(x=x, h=h))
    f = z.BlockFfn(h=h, w_gate=w[0], w_up=w[1], a=new(hidden), gate=new(hidden), up=new(hidden))
    z.zero_block_ffn(f, z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols, hidden)))
    replica = torch.zeros(hidden, cols, dtype=BF16, device="cuda")
    b = z.BlockFfnGrad(da=torch.randn(rows, hidden, device="cuda").bfloat16(), dgate=new(hidden), dup=new(hidden), gate=f.gate, up=f.up,
                       w_gate=w[0], w_up=w[1], dh=new(cols), h=h, dw_gate=replica)
    z.zero_block_ffn_grad(b, 0, z.workspace(z.zero_block_ffn_grad_workspace_bytes(rows, cols, hidden)))
    keep = torch.arange(rows, device="cuda") != 9
    assert torch.isfinite(b.dh[keep].float()).all() and not torch.isfinite(b.dh[9].float()).any()
    state = [torch.randn(hidden * cols, device="cuda") for _ in range(3)]
    state[2].abs_()
    before = [t.clone() for t in state]
    out = torch.zeros(hidden * cols, dtype=BF16, device="cuda")
    ts = [z.ZeroTensor([replica.view(-1)], *state, out)]
    hp = z.HParams(step=2, skip_on_nonfinite=1)
    res = z.new_result()
    z.zero_step(ts, hp, 0.0, z.workspace(z.zero_step_workspace_bytes(ts, 1, hp)), res)
    r = z.read_result(res)
    assert r["found_inf"] == 1 and r["skipped"] == 1
    assert all(torch.equal(a, b) for a, b in zip(state, before)) and float(out.abs().max()) == 0.0


# ------------------------------------------------------------------ one workspace for a step and these calls

HP = dict(lr=1e-3, step=2)


def tensors():
    """A list whose table is longer than what the calls below sum at the least."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    return [z.ZeroTensor([rnd(640).bfloat16() for _ in range(4)], rnd(640), rnd(640), rnd(640).abs(),
                         torch.zeros(640, dtype=BF16, device="cuda")) for _ in range(300)]


def state_of(ts):
    return [t.clone() for x in ts for t in (x.master, x.exp_avg, x.exp_avg_sq, x.param_out)]


def step(ts, ws):
    res = z.new_result()
    z.zero_step(ts, z.HParams(**HP), 0.0, ws, res)
    return z.read_result(res)


def norm_call(wants, cols, ws):
    rnd = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    one = torch.ones(64, device="cuda")
    new = lambda k: torch.zeros(cols, device="cuda") if k in wants else None  # noqa: E731
    z.zero_layer_norm_grad(z.LayerNormGrad(dx=rnd(64, cols), dh=rnd(64, cols), rstd=one, x_out=rnd(64, cols), mean=one, dw=new("dw"),
                                           db=new("db")), 0, ws)


def forward_call(rows, cols, hidden, ws):
    rnd = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    z.zero_block_ffn(z.BlockFfn(h=rnd(rows, cols), w_gate=rnd(hidden, cols), w_up=rnd(hidden, cols), a=rnd(rows, hidden)), ws)


def backward_call(wants, rows, cols, hidden, ws):
    rnd = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    dh, dw = "dh" in wants, [torch.zeros(hidden, cols, device="cuda") if k in wants else None for k in ("dw_gate", "dw_up")]
    z.zero_block_ffn_grad(z.BlockFfnGrad(
        da=rnd(rows, hidden), dgate=rnd(rows, hidden), dup=rnd(rows, hidden), gate=rnd(rows, hidden), up=rnd(rows, hidden),
        w_gate=rnd(hidden, cols) if dh else None, w_up=rnd(hidden, cols) if dh else None, dh=rnd(rows, cols) if dh else None,
        h=rnd(rows, cols) if any(t is not None for t in dw) else None, dw_gate=dw[0], dw_up=dw[1]), 0, ws)


# sums over long axes into small results: their parts are in the workspace
CALLS = [(norm_call, w, c) for c in (512, 8200) for w in ((), ("dw",), ("db",), ("dw", "db"))]
CALLS += [(forward_call, 8, 20000, 64), (backward_call, ("dh",), 8, 64, 20000)]
CALLS += [(backward_call, w, 20000, 64, 64) for w in (("dw_gate",), ("dw_up",), ("dw_gate", "dw_up"))]
# odd columns: copies of the operands
CALLS += [(forward_call, 640, 767, 1001)] + [(backward_call, w, 640, 767, 1001) for w in (("dh",), ("dw_gate",), ("dw_up",))]


@pytest.mark.parametrize("case", CALLS)
def test_a_step_after_a_call_on_its_workspace(case):
    want = tensors()
    own = z.workspace(z.zero_step_workspace_bytes(want, 4, z.HParams(**HP)))
    for _ in range(3):
        assert step(want, own)["status"] == 0
    ts, ws = tensors(), z.workspace(64 << 20)
    for _ in range(2):
        assert step(ts, ws)["status"] == 0
    case[0](*case[1:], ws)
    assert step(ts, ws)["status"] == 0
    assert all(torch.equal(a, b) for a, b in zip(state_of(ts), state_of(want)))


@pytest.mark.parametrize("case", CALLS)
def test_a_captured_step_knows_that_its_table_is_gone(case):
    ts, ws, res = tensors(), z.workspace(64 << 20), z.new_result()
    hp = z.HParams(**HP)
    z.zero_step(ts, hp, 0.0, ws, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_step(ts, hp, 0.0, ws, res)  # the table is in place: the graph holds the step alone
    graph.replay()
    assert z.read_result(res)["status"] == 0
    before = state_of(ts)
    case[0](*case[1:], ws)
    if case[0] is norm_call and case[1] == () and case[2] <= 8192:
        return  # no sums: it writes nothing to its workspace
    for _ in range(2):
        graph.replay()
        r = z.read_result(res)
        assert r["status"] == z.ZERO_ERR_STALE_WORKSPACE and r["skipped"] == 1
        assert all(torch.equal(a, b) for a, b in zip(state_of(ts), before))
    z.zero_step(ts, hp, 0.0, ws, res)  # uploads the table again, for the graph too
    assert z.read_result(res)["status"] == 0
    for _ in range(2):
        graph.replay()
        assert z.read_result(res)["status"] == 0
