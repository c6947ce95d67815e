"""The calls around a training block used together, as a training step uses
them: two residual blocks forward with 8-bit checkpoints, backward through the
norms and the weight gradients over two micro-batches, and the framework's own
step from those gradients. Every stage is held to its 64-bit formula on the
tensors that it was given, the weight gradients also to what unrounded
activations give, and the new weights to the CPU oracle on the same gradients."""
import pytest
import torch

import oracle
import sharded_optimizer_step_amd as z
from block_cases import U, assert_within, decode_act8, grad_reference, norm_reference
from cases import assert_state_matches, hp_oracle, to_np_f32, to_np_u16

pytestmark = pytest.mark.gpu

ROW = 48 * U  # roundings of a row's sum, as in the norms' own tests


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z.lib()
    torch.cuda.set_device(0)
    yield


class Block:
    """x -> x + alpha * gate * n(W n(x)): its bf16 parameters and what a micro-batch saves."""

    def __init__(self, cols, gates, g):
        near_one = lambda: (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).bfloat16()  # noqa: E731
        self.w = (torch.randn(cols, cols, device="cuda", generator=g) * cols**-0.5).bfloat16()
        self.w_pre, self.w_post = near_one(), near_one()
        self.gate = (0.5 * torch.randn(gates, cols, device="cuda", generator=g)).bfloat16()
        self.names = ("w", "w_pre", "w_post", "gate")


def boundary(x, block, y, after, gate_rows, alpha, fmt):
    """The boundary after `block` (None: the stream's start) and before `after` (None: its end)."""
    rows, cols = x.shape
    new = lambda t: torch.zeros(rows, cols, dtype=t, device="cuda")  # noqa: E731
    b = z.BlockNorm(x=x, y=y, w_post=block.w_post if block else None, gate=block.gate if block else None,
                    w_pre=after.w_pre if after else None, x_out=new(x.dtype) if block else None,
                    h=new(torch.bfloat16) if after else None,
                    rstd_post=torch.zeros(rows, device="cuda") if block else None,
                    rstd_pre=torch.zeros(rows, device="cuda") if after else None,
                    ckpt_post=z.new_act8(rows, cols, fmt) if block else None,
                    ckpt_pre=z.new_act8(rows, cols, fmt) if after else None,
                    gate_rows=gate_rows if block else 0, residual_scale=alpha)
    z.zero_block_norm(b)
    ref = norm_reference(b, b.x_out if block else b.x)
    if block:
        assert_within(b.x_out, ref["x_out"], ref["x_out_mag"], ROW + 8 * U, "x_out")
    if after:
        assert_within(b.h, ref["h"], ref["h"].abs(), ROW / 2 + 8 * U, "h")
        b.exact_xn = ref["xn"]
    return b


@pytest.mark.parametrize("fmt", [z.ACT8_E4M3, z.ACT8_INT8])
@pytest.mark.parametrize("resid", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,gate_rows", [(70, 96, 35), (513, 328, 200), (130, 1000, 130)])
def test_two_blocks_and_a_step(rows, cols, gate_rows, resid, fmt):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    alpha, gates = 0.5, -(-rows // gate_rows)
    blocks = [Block(cols, gates, g) for _ in range(2)]
    acc = {(i, n): torch.zeros_like(getattr(b, n), dtype=torch.float32) for i, b in enumerate(blocks) for n in b.names}
    ws_w = z.workspace(z.zero_act8_wgrad_workspace_bytes(rows, cols, cols))
    ws_n = z.workspace(z.zero_block_norm_grad_workspace_bytes(rows, cols, gate_rows))
    for micro in range(2):
        x = torch.randn(rows, cols, device="cuda", generator=g).to(resid)
        # forward
        edges, y = [boundary(x, None, None, blocks[0], 0, alpha, fmt)], None
        for i, blk in enumerate(blocks):
            y = (edges[-1].h.float() @ blk.w.float().t()).bfloat16()
            after = blocks[i + 1] if i + 1 < len(blocks) else None
            edges.append(boundary(edges[-1].x_out if edges[-1].x_out is not None else x, blk, y, after, gate_rows, alpha, fmt))
        # backward from a gradient of the stream's end
        d = (torch.randn(rows, cols, device="cuda", generator=g) * 1e-2).to(resid)
        dh = None
        for i in (1, 0):
            blk, after, e = blocks[i], blocks[i + 1] if i == 0 else None, edges[i + 1]
            gr = z.BlockNormGrad(
                dx=torch.zeros_like(d), dx_out=d, dh=dh, w_post=blk.w_post, gate=blk.gate, w_pre=after.w_pre if after else None,
                ckpt_pre=e.ckpt_pre, ckpt_post=e.ckpt_post, rstd_pre=e.rstd_pre, rstd_post=e.rstd_post,
                dy=torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"),
                dw_pre=acc[1, "w_pre"] if after else None, dw_post=acc[i, "w_post"], dgate=acc[i, "gate"],
                gate_rows=gate_rows, residual_scale=alpha)
            old = {n: t.double().clone() for n, t in (("dw_pre", gr.dw_pre), ("dw_post", gr.dw_post), ("dgate", gr.dgate)) if t is not None}
            yn = torch.tensor(decode_act8(e.ckpt_post)[0], device="cuda")
            xn = torch.tensor(decode_act8(e.ckpt_pre)[0], device="cuda") if after else None
            z.zero_block_norm_grad(gr, z.GRAD_ACCUMULATE, ws_n)
            ref = grad_reference(gr, xn, yn)
            rel = 2 * ROW + 16 * U
            assert_within(gr.dx, *ref["dx"], rel, "dx")
            assert_within(gr.dy, *ref["dy"], 2 * rel, "dy")
            for n, o in old.items():
                got = getattr(gr, n).reshape(o.shape)
                want, mag = (t.reshape(o.shape) for t in ref[n])
                assert_within(got, want + o, mag + o.abs(), 2 * rel + (rows + 64) * U, n)
            # the block's matrix, from its 8-bit input rows before their weight
            before = edges[i]
            o = acc[i, "w"].double().clone()
            z.zero_act8_wgrad(gr.dy, before.ckpt_pre, acc[i, "w"], z.GRAD_ACCUMULATE, ws_w, col_scale=blk.w_pre)
            rows8 = torch.tensor(decode_act8(before.ckpt_pre)[0], device="cuda")
            scale = blk.w_pre.double()
            dyt = gr.dy.double().t().contiguous()
            want, mag = (dyt @ rows8) * scale, (dyt.abs() @ rows8.abs()) * scale.abs()
            assert_within(acc[i, "w"], want + o, mag + o.abs(), 2 * (rows + 8) * U, "dw")
            # against the rows that were saved: half a step of e4m3, or half of a
            # block's unit, at most 1/127 of its largest value, an element
            half = (2.0**-4 * before.exact_xn.abs() + 2.0**-10 if fmt == z.ACT8_E4M3 else
                    torch.nn.functional.max_pool1d(before.exact_xn.abs()[:, None], 32, 32, ceil_mode=True).repeat_interleave(32, 2)[:, 0, :cols] / 127)
            off = (acc[i, "w"].double() - o - (dyt @ before.exact_xn) * scale).abs()
            assert (off <= (dyt.abs() @ half) * scale.abs() * (1 + 2.0**-7) + 2 * (rows + 8) * U * mag + U * o.abs()).all()
            dh = (gr.dy.float() @ blk.w.float()).bfloat16()
            d = gr.dx
        # the stream's start: the first block's norm alone
        e = edges[0]
        gr = z.BlockNormGrad(dx=torch.zeros_like(d), dx_out=d, dh=dh, w_pre=blocks[0].w_pre, ckpt_pre=e.ckpt_pre, rstd_pre=e.rstd_pre,
                             dw_pre=acc[0, "w_pre"])
        o = acc[0, "w_pre"].double().clone()
        z.zero_block_norm_grad(gr, z.GRAD_ACCUMULATE, z.workspace(z.zero_block_norm_grad_workspace_bytes(rows, cols, 0)))
        ref = grad_reference(gr, torch.tensor(decode_act8(e.ckpt_pre)[0], device="cuda"), None)
        assert_within(gr.dx, *ref["dx"], 2 * ROW + 16 * U, "dx")
        assert_within(acc[0, "w_pre"], ref["dw_pre"][0][0] + o, ref["dw_pre"][1][0] + o.abs(), 4 * ROW + (rows + 96) * U, "dw_pre")
    # the step: AdamW on each parameter from its fp32 gradient, and the same from the oracle
    hp = z.HParams(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3, max_grad_norm=1.0, grad_scale=1.0)
    for (i, n), a in acc.items():
        p = getattr(blocks[i], n)
        master, m, v = p.float().flatten(), torch.zeros(p.numel(), device="cuda"), torch.zeros(p.numel(), device="cuda")
        start = [to_np_f32(t).copy() for t in (master, m, v)]
        res = z.new_result()
        ws = z.workspace(z.zero_grad_check_norm_workspace_bytes(p.numel()))
        z.zero_grad_check_norm(a.flatten(), hp, 0.0, ws, res)
        z.zero_adamw_step(master, m, v, a.flatten(), p.view(-1), hp, res)
        r = z.read_result(res)
        norm = float(a.double().norm())
        assert r["found_inf"] == 0 and abs(r["grad_norm"] - norm) <= 1e-5 * norm
        new = oracle.adamw(*start, to_np_f32(a.flatten()), hp_oracle(hp), r["clip_coef"])
        assert_state_matches(to_np_f32(master), to_np_f32(m), to_np_f32(v), to_np_u16(p.view(-1)), *new, where=(i, n))


def test_nonfinite_activations_skip_the_step():
    """An inf in a saved row reaches the weight gradient, its flag and the skip."""
    rows, cols = 64, 96
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    x[9, 40] = float("inf")
    ck = z.new_act8(rows, cols)
    z.zero_act8_save(x, ck)
    dy = torch.randn(rows, cols, device="cuda").bfloat16()
    replica = torch.zeros(cols, cols, dtype=torch.bfloat16, device="cuda")
    z.zero_act8_wgrad(dy, ck, replica)
    state = [torch.randn(cols * cols, device="cuda") for _ in range(3)]
    state[2].abs_()
    out = torch.zeros(cols * cols, dtype=torch.bfloat16, device="cuda")
    keep = [t.clone() for t in state]
    ts = [z.ZeroTensor([replica.view(-1)], *state, out)]
    hp = z.HParams(step=2, skip_on_nonfinite=1)
    res = z.new_result()
    z.zero_step(ts, hp, 0.0, z.workspace(z.zero_step_workspace_bytes(ts, 1, hp)), res)
    r = z.read_result(res)
    assert r["found_inf"] == 1 and r["skipped"] == 1
    assert all(torch.equal(a, b) for a, b in zip(state, keep)) and float(out.abs().max()) == 0.0
