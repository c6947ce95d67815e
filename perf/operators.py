"""Timing cases of the operators around a training block: 8-bit activation
checkpoints, the weight gradient taken from one, and the norms before and
after a block with its gate and residual scale, forward and backward.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes a case's inputs on the GPU from a seed, ``run()`` makes one
pass: the plain PyTorch form, or with ``own`` set the library's entry points.
``exact()`` computes the same outputs in binary64, ``work()`` counts what a
pass has to move and compute.

The 8-bit form: each row is cut into blocks of 32 columns (the last may be
short); a block is stored as 8-bit codes and a power of two 2^k, the smallest
with max|x| <= F * 2^k (F = 448 for e4m3, 127 for int8) and k >= -117; a code
is x / 2^k rounded to nearest even. A block that holds an inf or NaN decodes
to NaN. In memory: rows x P codes (P = columns rounded up to 32, the rest 0),
then rows x P/32 bytes k + 127 (255: NaN).
"""
import math

import torch

own = False

BLOCK = 32
KMIN = -117


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short sequence of a small model, saved and read back: the latency of two small launches
        dict(name="checkpoint short", op="checkpoint", rows=129, cols=771, pad=5, dtype="fp32", fmt="e4m3"),
        # a long micro-batch's block boundary of a 4096-wide model
        dict(name="checkpoint long", op="checkpoint", rows=16384, cols=4096, pad=0, dtype="bf16", fmt="int8"),
        # a 768-wide projection, one short sequence
        dict(name="wgrad short", op="wgrad", rows=192, outs=768, cols=768, fmt="e4m3", grad="bf16", scaled=False),
        # the 4096 x 4096 attention projections: one micro-batch of several, added to the fp32 accumulator;
        # the checkpoint holds normalised rows, so the norm's weight scales the columns
        dict(name="wgrad attention", op="wgrad", rows=8192, outs=4096, cols=4096, fmt="int8", grad="fp32", scaled=True),
        # the 11008 x 4096 gate and up projections, one bf16 gradient replica
        dict(name="wgrad mlp", op="wgrad", rows=8192, outs=11008, cols=4096, fmt="e4m3", grad="bf16", scaled=True),
        # a small odd matrix under very many tokens: the work has to be split over the tokens
        dict(name="wgrad tokens", op="wgrad", rows=30011, outs=200, cols=333, fmt="int8", grad="fp32", scaled=False),
        # between two blocks of a small model, a learned gate per channel
        dict(name="norm short", op="norm", rows=128, cols=768, post=True, pre=True, gate_rows=128, resid="bf16",
             weights="bf16", fmt="e4m3"),
        # a long micro-batch of 4096-wide rows, a gate for each 2048-token sequence, both checkpoints written
        dict(name="norm long", op="norm", rows=16384, cols=4096, post=True, pre=True, gate_rows=2048, resid="bf16",
             weights="bf16", fmt="e4m3"),
        # odd rows and columns, an fp32 residual stream, no norm after the block, a gate for every token
        dict(name="norm odd", op="norm", rows=3001, cols=5003, post=False, pre=True, gate_rows=1, resid="fp32",
             weights="fp32", fmt="int8"),
        # the same boundaries backwards
        dict(name="norm grad short", op="grad", rows=128, cols=768, post=True, pre=True, gate_rows=128, resid="bf16",
             weights="bf16", fmt="e4m3", saved="8bit", grad="bf16"),
        dict(name="norm grad long", op="grad", rows=16384, cols=4096, post=True, pre=True, gate_rows=2048,
             resid="bf16", weights="bf16", fmt="e4m3", saved="8bit", grad="bf16"),
        # odd sizes, fp32 residual gradient, the saved rows in their own types, fp32 gradients added to
        dict(name="norm grad odd", op="grad", rows=3001, cols=5003, post=True, pre=True, gate_rows=700, resid="fp32",
             weights="fp32", fmt="int8", saved="raw", grad="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["checkpoint", "wgrad", "norm", "grad"])
    fmt = rng.choice(["e4m3", "int8"])
    if op == "wgrad":
        while True:
            rows, outs, cols = _log(rng, 1, 32768), _log(rng, 64, 11008), _log(rng, 64, 11008)
            if rng.random() < 0.5:
                outs, cols = -(-outs // 64) * 64, -(-cols // 64) * 64
            if rows * outs * cols <= 8192 * 11008 * 4096:
                break
        return dict(op=op, rows=rows, outs=outs, cols=cols, fmt=fmt, grad=rng.choice(["bf16", "fp32"]),
                    scaled=rng.random() < 0.5)
    while True:
        rows, cols = _log(rng, 1, 32768), _log(rng, 64, 11008)
        if rng.random() < 0.5:
            cols = -(-cols // 64) * 64
        if rows * cols <= 16384 * 4096:
            break
    if op == "checkpoint":
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 3, 64]), dtype=rng.choice(["bf16", "fp32"]),
                    fmt=fmt)
    post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
    gate_rows = rng.choice([0, 1, rows, _log(rng, 1, rows)])
    case = dict(op=op, rows=rows, cols=cols, post=post, pre=pre, gate_rows=gate_rows,
                resid=rng.choice(["bf16", "fp32"]), weights=rng.choice(["bf16", "fp32"]), fmt=fmt)
    if op == "grad":
        case.update(saved=rng.choice(["8bit", "raw"]), grad=rng.choice(["bf16", "fp32"]))
    return case


# ------------------------------------------------------------------ the 8-bit form, in 32 bits

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _pow2(n):
    return ((n + 127) << 23).view(torch.float32)


def _blocks(x):
    """The rows of x in whole blocks of 32 columns, the last one filled with zeros."""
    short = -x.shape[1] % BLOCK
    if short:
        x = torch.cat([x, x.new_zeros(x.shape[0], short)], 1)
    return x.view(x.shape[0], -1, BLOCK)


def _quantise(x, fmt):
    """(values on the code grid, k, whether the block is finite) of fp32 rows."""
    b = _blocks(x)
    top = b.abs().amax(2, keepdim=True)
    fine = torch.isfinite(top)
    # the exponent of top, one more where its mantissa is over F's
    over, emax = (0x1FFFFF, 8) if fmt == "e4m3" else (0x01FFFF, 6)
    k = (((top.view(torch.int32) + over) >> 23) - (127 + emax)).clamp(min=KMIN)
    k = torch.where(fine, k, torch.zeros_like(k))
    v = torch.where(fine, b, torch.zeros_like(b)) * _pow2(-k)
    if fmt == "e4m3":
        step = torch.frexp(v)[1].clamp(min=-5) - 4
        v = torch.round(v * _pow2(-step)) * _pow2(step)
    else:
        v = torch.round(v)
    return v, k, fine


def _rounded(x, fmt):
    """What a checkpoint of the fp32 rows x decodes to, in fp32."""
    v, k, fine = _quantise(x, fmt)
    out = torch.where(fine, v * _pow2(k), torch.full_like(v, math.nan))
    return out.view(x.shape[0], -1)[:, :x.shape[1]]


def _encode(x, fmt):
    """The checkpoint of fp32 rows, as the bytes of its layout."""
    v, k, fine = _quantise(x, fmt)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else v.to(torch.int8).view(torch.uint8)
    scales = torch.where(fine, k + 127, torch.full_like(k, 255)).to(torch.uint8)
    return torch.cat([codes.reshape(-1), scales.reshape(-1)])


def _decode(buf, rows, cols, fmt):
    pitch = -(-cols // BLOCK) * BLOCK
    codes = buf[:rows * pitch].view(rows, -1, BLOCK)
    k = buf[rows * pitch:].view(rows, -1, 1).to(torch.int32) - 127
    if fmt == "e4m3":
        c = codes.to(torch.int32)
        e, m = (c >> 3) & 15, (c & 7).float()
        v = torch.where(e > 0, (8 + m) * _pow2((e - 10).clamp(min=-9)), m * 2.0**-9)
        v = torch.where(c > 127, -v, v)
    else:
        v = codes.view(torch.int8).float()
    v = torch.where(k == 128, torch.full_like(v, math.nan), v * _pow2(k.clamp(max=127)))
    return v.view(rows, pitch)[:, :cols]


# ------------------------------------------------------------------ inputs

def _activations(rows, cols, g, dev):
    """Rows as a transformer's: a few channels are ten times the others."""
    x = torch.randn(rows, cols, device=dev, generator=g)
    loud = torch.rand(cols, device=dev, generator=g) < 0.01
    return x * torch.where(loud, 10.0, 1.0)


def _gates(case, g, dev):
    if not case["gate_rows"]:
        return None
    n = -(-case["rows"] // case["gate_rows"])
    return (torch.randn(n, case["cols"], device=dev, generator=g) * 0.5).to(_TYPES[case["weights"]])


def _normalised(x, eps):
    rstd = torch.rsqrt((x * x).mean(1) + eps)
    return x * rstd[:, None], rstd


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows, cols = case["rows"], case["cols"]
    s = dict(case)
    new = lambda r, c, t: torch.empty(r, c, dtype=t, device=dev)  # noqa: E731
    if case["op"] == "checkpoint":
        t = _TYPES[case["dtype"]]
        s["x"] = new(rows, cols + case["pad"], t)[:, :cols]
        s["x"].copy_(_activations(rows, cols, g, dev))
        s["saved"] = torch.empty(rows * (-(-cols // BLOCK)) * (BLOCK + 1), dtype=torch.uint8, device=dev)
        s["out"] = new(rows, cols, torch.bfloat16)
    elif case["op"] == "wgrad":
        x = _activations(rows, cols, g, dev)
        s["saved_x"] = _encode(_normalised(x, 1e-6)[0] if case["scaled"] else x, case["fmt"])
        s["dy"] = (torch.randn(rows, case["outs"], device=dev, generator=g) * 1e-3).to(torch.bfloat16)
        s["scale"] = (1 + 0.1 * torch.randn(cols, device=dev, generator=g)).to(torch.bfloat16) if case["scaled"] else None
        s["dw"] = new(case["outs"], cols, _TYPES[case["grad"]])
        if case["grad"] == "fp32":  # the sum of the micro-batches before this one
            s["dw"].normal_(0, 1e-2, generator=g)
    else:
        rt, wt, pt = _TYPES[case["resid"]], _TYPES[case["weights"]], torch.bfloat16
        near_one = lambda: (1 + 0.1 * torch.randn(cols, device=dev, generator=g)).to(wt)  # noqa: E731
        s["alpha"], s["eps"] = 0.125, 1e-6  # 1 / sqrt(2 * 32 layers)
        s["w_post"] = near_one() if case["post"] else None
        s["w_pre"] = near_one() if case["pre"] else None
        s["gate"] = _gates(case, g, dev)
        y = (_activations(rows, cols, g, dev) * 3).to(pt)
        if case["op"] == "norm":
            s["x"] = (_activations(rows, cols, g, dev) * 2).to(rt)
            s["y"] = y
            s["x_out"] = new(rows, cols, rt)
            for name in (("post", "pre") if case["pre"] else ("post",)):
                s["rstd_" + name] = torch.empty(rows, device=dev)
                s["saved_" + name] = torch.empty(rows * (-(-cols // BLOCK)) * (BLOCK + 1), dtype=torch.uint8, device=dev)
                s["read_" + name] = new(rows, cols, pt)
            s["h"] = new(rows, cols, pt) if case["pre"] else None
        else:
            x_out = (_activations(rows, cols, g, dev) * 2).to(rt)
            xhat, s["rstd_pre"] = _normalised(x_out.float(), s["eps"])
            yhat, s["rstd_post"] = _normalised(y.float(), s["eps"])
            if not case["post"]:
                yhat = y.float()
            if case["saved"] == "raw":
                s["x_out"], s["y"] = x_out, y
            else:
                s["saved_pre"], s["saved_post"] = _encode(xhat, case["fmt"]), _encode(yhat, case["fmt"])
            s["dh"] = (torch.randn(rows, cols, device=dev, generator=g) * 1e-3).to(pt) if case["pre"] else None
            s["dx_out"] = (torch.randn(rows, cols, device=dev, generator=g) * 1e-3).to(rt)
            s["dx"], s["dy"] = new(rows, cols, rt), new(rows, cols, pt)
            gt = _TYPES[case["grad"]]
            for name, n in (("dw_pre", 1 if case["pre"] else 0), ("dw_post", 1 if case["post"] else 0),
                            ("dgate", 0 if s["gate"] is None else s["gate"].shape[0])):
                s[name] = new(n, cols, gt) if n else None
                if n and case["grad"] == "fp32":
                    s[name].normal_(0, 1e-2, generator=g)
    if own:  # the workspace that a program keeps beside its buffers
        import sharded_optimizer_step_amd as z
        if case["op"] == "wgrad":
            s["ws"] = z.workspace(z.zero_act8_wgrad_workspace_bytes(rows, case["outs"], cols))
        elif case["op"] == "grad":
            s["ws"] = z.workspace(z.zero_block_norm_grad_workspace_bytes(rows, cols, case["gate_rows"]))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _sum_into(s, name, value):
    """A gradient as its buffer takes it: added to an fp32 accumulator, or one bf16 replica."""
    if s["grad"] == "fp32":
        s[name] += value
        return s[name]
    return value.to(torch.bfloat16)


def _plain_checkpoint(s):
    return _rounded(s["x"].float(), s["fmt"]).to(torch.bfloat16)


def _plain_wgrad(s):
    dw = s["dy"].float().t() @ _decode(s["saved_x"], s["rows"], s["cols"], s["fmt"])
    if s["scale"] is not None:
        dw = dw * s["scale"].float()
    return _sum_into(s, "dw", dw)


def _by_row(s):
    """The gate's row for each row, times the residual scale."""
    if s["gate"] is None:
        return s["alpha"]
    at = torch.arange(s["rows"], device=s["gate"].device) // s["gate_rows"]
    return s["alpha"] * s["gate"].float()[at]


def _plain_norm(s):
    out = {}
    y = s["y"].float()
    if s["post"]:
        y, out["rstd_post"] = _normalised(y, s["eps"])
        u = y * s["w_post"].float()
    else:
        u = y
    out["read_post"] = _rounded(y, s["fmt"]).to(torch.bfloat16)
    out["x_out"] = (s["x"].float() + _by_row(s) * u).to(s["x"].dtype)
    if s["pre"]:
        xhat, out["rstd_pre"] = _normalised(out["x_out"].float(), s["eps"])
        out["h"] = (xhat * s["w_pre"].float()).to(torch.bfloat16)
        out["read_pre"] = _rounded(xhat, s["fmt"]).to(torch.bfloat16)
    return out


def _saved(s, name, raw):
    if s["saved"] == "8bit":
        return _decode(s["saved_" + name], s["rows"], s["cols"], s["fmt"])
    x = s[raw].float()
    return x * s["rstd_" + name][:, None] if s[name] else x


def _plain_grad(s):
    out = {}
    dx = s["dx_out"].float()
    if s["pre"]:
        xhat, dh = _saved(s, "pre", "x_out"), s["dh"].float()
        v = dh * s["w_pre"].float()
        dx = dx + s["rstd_pre"][:, None] * (v - xhat * (v * xhat).mean(1, keepdim=True))
        out["dw_pre"] = _sum_into(s, "dw_pre", (dh * xhat).sum(0, keepdim=True))
    out["dx"] = dx.to(s["dx_out"].dtype)
    du = dx * _by_row(s)
    if s["post"] or s["gate"] is not None:
        yhat = _saved(s, "post", "y")
    if s["post"]:
        w = s["w_post"].float()
        v = du * w
        out["dy"] = (s["rstd_post"][:, None] * (v - yhat * (v * yhat).mean(1, keepdim=True))).to(torch.bfloat16)
        out["dw_post"] = _sum_into(s, "dw_post", (du * yhat).sum(0, keepdim=True))
    else:
        w = 1.0
        out["dy"] = du.to(torch.bfloat16)
    if s["gate"] is not None:
        each = s["alpha"] * dx * yhat * w
        # rows of one gate are next to each other: a padded view sums them without atomics
        short = -s["rows"] % s["gate_rows"]
        if short:
            each = torch.cat([each, each.new_zeros(short, s["cols"])])
        out["dgate"] = _sum_into(s, "dgate", each.view(int(s["gate"].shape[0]), s["gate_rows"], -1).sum(1))
    return out


_plain = dict(checkpoint=_plain_checkpoint, wgrad=_plain_wgrad, norm=_plain_norm, grad=_plain_grad)


def _format(z, s):
    return z.ACT8_E4M3 if s["fmt"] == "e4m3" else z.ACT8_INT8


def _own_checkpoint(s):
    import sharded_optimizer_step_amd as z
    ck = z.Act8(s["rows"], s["cols"], _format(z, s), s["saved"])
    z.zero_act8_save(s["x"], ck)
    z.zero_act8_load(ck, s["out"])
    return s["out"]


def _own_wgrad(s):
    import sharded_optimizer_step_amd as z
    ck = z.Act8(s["rows"], s["cols"], _format(z, s), s["saved_x"])
    z.zero_act8_wgrad(s["dy"], ck, s["dw"], z.GRAD_ACCUMULATE if s["grad"] == "fp32" else 0, s["ws"],
                      col_scale=s["scale"])
    return s["dw"]


def _own_norm(s):
    import sharded_optimizer_step_amd as z
    act = lambda n: z.Act8(s["rows"], s["cols"], _format(z, s), s["saved_" + n])  # noqa: E731
    post, pre = act("post"), act("pre") if s["pre"] else None
    z.zero_block_norm(z.BlockNorm(
        x=s["x"], y=s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], x_out=s["x_out"], h=s["h"],
        rstd_post=s["rstd_post"] if s["post"] else None, rstd_pre=s["rstd_pre"] if s["pre"] else None,
        ckpt_post=post, ckpt_pre=pre, gate_rows=s["gate_rows"], residual_scale=s["alpha"], eps=s["eps"]))
    out = dict(x_out=s["x_out"], read_post=s["read_post"])
    z.zero_act8_load(post, s["read_post"])
    if s["post"]:
        out["rstd_post"] = s["rstd_post"]
    if s["pre"]:
        z.zero_act8_load(pre, s["read_pre"])
        out.update(rstd_pre=s["rstd_pre"], h=s["h"], read_pre=s["read_pre"])
    return out


def _own_grad(s):
    import sharded_optimizer_step_amd as z
    b = z.BlockNormGrad(
        dx_out=s["dx_out"], dh=s["dh"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], dx=s["dx"], dy=s["dy"],
        dw_post=s["dw_post"], dgate=s["dgate"], dw_pre=s["dw_pre"],
        rstd_post=s["rstd_post"] if s["post"] else None, rstd_pre=s["rstd_pre"] if s["pre"] else None,
        gate_rows=s["gate_rows"], residual_scale=s["alpha"])
    need = s["post"] or s["gate"] is not None
    if s["saved"] == "8bit":
        b.ckpt_pre = z.Act8(s["rows"], s["cols"], _format(z, s), s["saved_pre"]) if s["pre"] else None
        b.ckpt_post = z.Act8(s["rows"], s["cols"], _format(z, s), s["saved_post"]) if need else None
    else:
        b.x_out = s["x_out"] if s["pre"] else None
        b.y = s["y"] if need else None
    z.zero_block_norm_grad(b, z.GRAD_ACCUMULATE if s["grad"] == "fp32" else 0, s["ws"])
    out = dict(dx=s["dx"], dy=s["dy"])
    for name in ("dw_pre", "dw_post", "dgate"):
        if s[name] is not None:
            out[name] = s[name]
    return out


_own = dict(checkpoint=_own_checkpoint, wgrad=_own_wgrad, norm=_own_norm, grad=_own_grad)


# ------------------------------------------------------------------ work

def work(case):
    rows, cols = case["rows"], case["cols"]
    size = {"bf16": 2, "fp32": 4}
    packed = rows * (-(-cols // BLOCK)) * (BLOCK + 1)
    n = rows * cols
    if case["op"] == "checkpoint":  # saved and read back: two calls, so the 8 bits are written and read
        return dict(bytes=n * size[case["dtype"]] + 2 * packed + 2 * n, flops=0)
    if case["op"] == "wgrad":
        dw = case["outs"] * cols * (2 if case["grad"] == "bf16" else 8)
        return dict(bytes=packed + 2 * rows * case["outs"] + dw + (2 * cols if case["scaled"] else 0),
                    flops=2 * rows * case["outs"] * cols)
    r, w = size[case["resid"]], size[case["weights"]]
    gates = -(-rows // case["gate_rows"]) * cols if case["gate_rows"] else 0
    small = (case["post"] + case["pre"]) * (cols * w + 4 * rows) + gates * w
    if case["op"] == "norm":
        byts = n * (2 * r + 2) + 2 * packed + 2 * n + small
        if case["pre"]:
            byts += 2 * n + 2 * packed + 2 * n
        return dict(bytes=byts, flops=n * (14 if case["pre"] else 7))
    need = case["post"] or gates
    byts = n * (2 * r + 2) + small
    byts += ((packed if case["saved"] == "8bit" else n * r) + 2 * n) if case["pre"] else 0
    byts += (packed if case["saved"] == "8bit" else 2 * n) if need else 0
    byts += ((case["post"] + case["pre"]) * cols + gates) * (2 if case["grad"] == "bf16" else 8)
    return dict(bytes=byts, flops=n * 20)


# ------------------------------------------------------------------ in 64 bits

def _grid64(fmt):
    """The non-negative values that a code can stand for, in order."""
    if fmt == "int8":
        return [float(i) for i in range(128)]
    return [m * 2.0**-9 for m in range(8)] + [(1 + m / 8) * 2.0**(e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest64(x, fmt):
    """Rows through the 8-bit form, by looking for the nearest code; ties go to the even one."""
    rows, cols = x.shape
    out = torch.empty_like(x)
    grid = torch.tensor(_grid64(fmt), dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    whole = cols // BLOCK * BLOCK
    parts = [x[:, :whole].reshape(rows, -1, BLOCK)] + ([x[:, whole:].reshape(rows, 1, -1)] if whole < cols else [])
    done = []
    for p in parts:
        if p.numel() == 0:
            continue
        top = p.abs().amax(2, keepdim=True)
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0**-140) / grid[-1])) - 1)
        for _ in range(3):  # up from below to the first power of two that reaches
            unit = torch.where(top > grid[-1] * unit, unit * 2, unit)
        unit = unit.clamp(min=2.0**KMIN)
        a = (p.abs() / unit).clamp(max=grid[-1].item())
        i = torch.searchsorted(middle, a.contiguous())
        tie = (a == middle[i.clamp(max=middle.numel() - 1)]) & (i % 2 == 1)
        done.append((torch.sign(p) * grid[i + tie.to(i.dtype)] * unit).reshape(rows, -1))
    torch.cat(done, 1, out=out)
    return out


def _read64(buf, rows, cols, fmt):
    pitch = -(-cols // BLOCK) * BLOCK
    codes = buf[:rows * pitch].view(rows, pitch)
    half = torch.tensor(_grid64(fmt), dtype=torch.float64, device=buf.device)
    if fmt == "e4m3":
        both = torch.cat([half, half.new_tensor([math.nan]), -half, half.new_tensor([math.nan])])
    else:
        both = torch.cat([half, half.new_tensor([math.nan]), -half[1:].flip(0)])
    unit = torch.exp2(buf[rows * pitch:].view(rows, -1).double() - 127).repeat_interleave(BLOCK, 1)
    return (both[codes.long()] * unit)[:, :cols]


def _gain64(s, dev):
    """residual scale times the gate of each row, [rows, cols] or [1, 1]."""
    if s["gate"] is None:
        return torch.full((1, 1), s["alpha"], dtype=torch.float64, device=dev)
    return s["alpha"] * s["gate"].double().repeat_interleave(s["gate_rows"], 0)[:s["rows"]]


def exact(case, seed):
    s = prepare(case, seed)
    rows, cols, fmt = case["rows"], case["cols"], case["fmt"]
    if case["op"] == "checkpoint":
        return _nearest64(s["x"].double(), fmt)
    if case["op"] == "wgrad":
        x = _read64(s["saved_x"], rows, cols, fmt)
        if s["scale"] is not None:
            x *= s["scale"].double()
        dw = torch.mm(s["dy"].double().t().contiguous(), x)
        return s["dw"].double() + dw if case["grad"] == "fp32" else dw
    gain = _gain64(s, s["gate"].device if s["gate"] is not None else torch.device("cuda"))
    if case["op"] == "norm":
        out = {}
        y = s["y"].double()
        if case["post"]:
            out["rstd_post"] = (y.square().sum(1) / cols + s["eps"]) ** -0.5
            y = y * out["rstd_post"].unsqueeze(1)
        out["read_post"] = _nearest64(y, fmt)
        x = s["x"].double() + gain * (y * s["w_post"].double() if case["post"] else y)
        out["x_out"] = x
        if case["pre"]:
            # the norm is that of the stored residual stream, so it is taken from the rounded values
            x = x.to(s["x"].dtype).double()
            out["rstd_pre"] = (x.square().sum(1) / cols + s["eps"]) ** -0.5
            x = x * out["rstd_pre"].unsqueeze(1)
            out["h"] = x * s["w_pre"].double()
            out["read_pre"] = _nearest64(x, fmt)
        return out
    old = lambda n: s[n].double() if case["grad"] == "fp32" else 0.0  # noqa: E731
    kept = {}
    for name, raw in (("pre", "x_out"), ("post", "y")):
        if case["saved"] == "8bit":
            kept[name] = _read64(s["saved_" + name], rows, cols, fmt)
        else:
            kept[name] = s[raw].double() * (s["rstd_" + name].double().unsqueeze(1) if case[name] else 1.0)
    out = {}
    total = s["dx_out"].double()
    if case["pre"]:
        dh, xh = s["dh"].double(), kept["pre"]
        wd = dh * s["w_pre"].double()
        along = (wd * xh).sum(1, keepdim=True) / cols
        total = total + (wd - along * xh) * s["rstd_pre"].double().unsqueeze(1)
        out["dw_pre"] = old("dw_pre") + (dh * xh).sum(0, keepdim=True)
    out["dx"] = total
    du, yh = gain * total, kept["post"]
    if case["post"]:
        wd = du * s["w_post"].double()
        along = (wd * yh).sum(1, keepdim=True) / cols
        out["dy"] = (wd - along * yh) * s["rstd_post"].double().unsqueeze(1)
        out["dw_post"] = old("dw_post") + (du * yh).sum(0, keepdim=True)
        yh = yh * s["w_post"].double()
    else:
        out["dy"] = du.expand(rows, cols)
    if s["gate"] is not None:
        sums = torch.stack([p.sum(0) for p in (s["alpha"] * total * yh).split(case["gate_rows"])])
        out["dgate"] = old("dgate") + sums
    return out
