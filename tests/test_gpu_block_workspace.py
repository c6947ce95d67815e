"""A workspace that serves a step and a call around a training block in turn, on
the GPU: the step after the call is, bit for bit, the step with a workspace of
its own."""
import pytest
import torch

import sharded_optimizer_step_amd as z

pytestmark = pytest.mark.gpu

ROWS, COLS = 64, 512
HP = dict(lr=1e-3, step=2)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z.lib()
    torch.cuda.set_device(0)
    yield


def tensors():
    """A list whose table is longer than a unit's sums."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    return [z.ZeroTensor([rnd(640).bfloat16() for _ in range(4)], rnd(640), rnd(640), rnd(640).abs(),
                         torch.zeros(640, dtype=torch.bfloat16, device="cuda")) for _ in range(300)]


def state(ts):
    return [t.clone() for x in ts for t in (x.master, x.exp_avg, x.exp_avg_sq, x.param_out)]


def step(ts, ws):
    res = z.new_result()
    z.zero_step(ts, z.HParams(**HP), 0.0, ws, res)
    return z.read_result(res)


def norm_grad(wants, gate_rows, cols, ws):
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    new = lambda n, name: torch.zeros(n, cols, device="cuda") if name in wants else None  # noqa: E731
    gates = -(-ROWS // gate_rows) if gate_rows else 0
    b = z.BlockNormGrad(dx=rnd(ROWS, cols), dx_out=rnd(ROWS, cols), dh=rnd(ROWS, cols), w_post=rnd(cols), w_pre=rnd(cols),
                        gate=rnd(gates, cols) if gates else None, x_out=rnd(ROWS, cols), y=rnd(ROWS, cols),
                        rstd_pre=torch.ones(ROWS, device="cuda"), rstd_post=torch.ones(ROWS, device="cuda"), dy=rnd(ROWS, cols),
                        dw_pre=new(1, "dw_pre"), dw_post=new(1, "dw_post"), dgate=new(gates, "dgate"), gate_rows=gate_rows)
    z.zero_block_norm_grad(b, 0, ws)


def wgrad(ws):
    rows, outs, cols = 20000, 64, 64
    assert 0 < z.zero_act8_wgrad_workspace_bytes(rows, outs, cols) <= ws.numel()
    ck = z.new_act8(rows, cols)
    z.zero_act8_save(torch.randn(rows, cols, device="cuda"), ck)
    z.zero_act8_wgrad(torch.randn(rows, outs, device="cuda").bfloat16(), ck, torch.zeros(outs, cols, device="cuda"), 0, ws)


CALLS = [("wgrad",)] + [(w, gate_rows, cols) for cols in (COLS, 8200) for w, gate_rows in (
    ((), 0), (("dw_pre",), 0), (("dw_post",), 0), (("dgate",), 1), (("dw_post", "dgate"), 1), (("dgate",), ROWS),
    (("dw_post", "dgate"), ROWS))]


def call(case, ws):
    if case[0] == "wgrad":
        wgrad(ws)
    else:
        norm_grad(*case, ws)


@pytest.mark.parametrize("case", CALLS)
def test_a_step_after_a_call_on_its_workspace(case):
    want = tensors()
    own = z.workspace(z.zero_step_workspace_bytes(want, 4, z.HParams(**HP)))
    for _ in range(3):
        assert step(want, own)["status"] == 0
    ts, ws = tensors(), z.workspace(16 << 20)
    for _ in range(2):
        assert step(ts, ws)["status"] == 0
    call(case, ws)
    assert step(ts, ws)["status"] == 0
    assert all(torch.equal(a, b) for a, b in zip(state(ts), state(want)))


@pytest.mark.parametrize("case", CALLS)
def test_a_captured_step_knows_that_its_table_is_gone(case):
    ts, ws, res = tensors(), z.workspace(16 << 20), z.new_result()
    hp = z.HParams(**HP)
    z.zero_step(ts, hp, 0.0, ws, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_step(ts, hp, 0.0, ws, res)  # the table is in place: the graph holds the step alone
    graph.replay()
    assert z.read_result(res)["status"] == 0
    before = state(ts)
    call(case, ws)
    if case[0] == () and case[2] == COLS:
        return  # no sums: it writes nothing to its workspace
    for _ in range(2):
        graph.replay()
        r = z.read_result(res)
        assert r["status"] == z.ZERO_ERR_STALE_WORKSPACE and r["skipped"] == 1
        assert all(torch.equal(a, b) for a, b in zip(state(ts), before))
    z.zero_step(ts, hp, 0.0, ws, res)  # uploads the table again, for the graph too
    assert z.read_result(res)["status"] == 0
    for _ in range(2):
        graph.replay()
        assert z.read_result(res)["status"] == 0
    want = tensors()
    own = z.workspace(z.zero_step_workspace_bytes(want, 4, hp))
    for _ in range(5):
        step(want, own)
    assert all(torch.equal(a, b) for a, b in zip(state(ts), state(want)))
