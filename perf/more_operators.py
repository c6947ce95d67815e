"""Timing cases of the layer norm and the gated feed-forward block, forward and
backward, as a training block runs them between the residual stream and the
gradients that the optimizer step reads.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes a case's inputs on the GPU from a seed, ``run()`` makes one
pass: the plain PyTorch form, or with ``own`` set the library's entry points.
``exact()`` computes the same outputs in binary64, ``work()`` counts what a
pass has to move and compute.

Layer norm, per row of C columns:
  x_out = x + y (stored in x's type; x itself without y)
  mean = sum(x_out) / C, rstd = 1 / sqrt(sum((x_out - mean)^2) / C + eps)
  xn = (x_out - mean) * rstd,  h = w * xn + b
backward, with v = w * dh:
  dx = dx_out + rstd * (v - mean(v) - xn * mean(v * xn))
  dw = sum over rows of dh * xn,  db = sum over rows of dh

Gated feed-forward block, h: R x C, weights F x C:
  g = h Wg^T,  u = h Wu^T,  a = act(g) * u
backward, from the saved g and u:
  dg = da * u * act'(g),  du = da * act(g)       (stored in bf16)
  dh = dg Wg + du Wu,  dWg = dg^T h,  dWu = du^T h   of dg and du as stored

Saved rows may be held in 8 bits: blocks of 32 columns (the last may be short)
of e4m3 or int8 codes with a power of two 2^k, the smallest with
max|x| <= F * 2^k (F = 448 or 127) and k >= -117; a code is x / 2^k rounded to
nearest even. In memory: rows x P codes (P = columns rounded up to 32, the rest
0), then rows x P/32 bytes k + 127.
"""
import math

import torch

own = False

BLOCK = 32
KMIN = -117


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short sequence of a small model: the latency of a small launch
        dict(name="layer norm short", op="norm", rows=128, cols=768, add=True, resid="bf16", weights="bf16", bias=True,
             save="", fmt="e4m3", pad=0),
        # a long micro-batch of 4096-wide rows, the normalised rows saved in 8 bits
        dict(name="layer norm long", op="norm", rows=16384, cols=4096, add=True, resid="bf16", weights="bf16", bias=True,
             save="xn", fmt="e4m3", pad=0),
        # the same backwards
        dict(name="layer norm grad short", op="norm_grad", rows=128, cols=768, resid="bf16", weights="bf16", bias=True,
             saved="raw", fmt="e4m3", grad="bf16", pad=0),
        dict(name="layer norm grad long", op="norm_grad", rows=16384, cols=4096, resid="bf16", weights="bf16", bias=True,
             saved="8bit", fmt="e4m3", grad="bf16", pad=0),
        # odd rows and columns, an fp32 residual stream, fp32 gradients added to
        dict(name="layer norm grad odd", op="norm_grad", rows=3001, cols=5003, resid="fp32", weights="fp32", bias=True,
             saved="raw", fmt="int8", grad="fp32", pad=5),
        # one token through the 11008 x 4096 gate and up projections: the weights have to be read
        dict(name="ffn token", op="ffn", rows=1, cols=4096, hidden=11008, act="silu", saved="", fmt="e4m3", pad=0),
        # one short sequence of a small model
        dict(name="ffn short", op="ffn", rows=192, cols=768, hidden=2048, act="gelu_tanh", saved="raw", fmt="e4m3", pad=0),
        # a micro-batch of 8192 tokens through the 11008 x 4096 projections, gate and up rows saved in bf16
        dict(name="ffn long", op="ffn", rows=8192, cols=4096, hidden=11008, act="silu", saved="raw", fmt="e4m3", pad=0),
        # odd sizes, rows that start anywhere, gate and up rows saved in 8 bits
        dict(name="ffn odd", op="ffn", rows=2011, cols=1003, hidden=2731, act="gelu", saved="8bit", fmt="int8", pad=3),
        # one short sequence backwards, one bf16 gradient replica
        dict(name="ffn grad short", op="ffn_grad", rows=192, cols=768, hidden=2048, act="gelu_tanh", saved="raw",
             input="raw", again=False, fmt="e4m3", grad="bf16", pad=0),
        # the micro-batch of 8192 tokens backwards from 8-bit gate and up rows, added to the fp32 accumulator
        dict(name="ffn grad long", op="ffn_grad", rows=8192, cols=4096, hidden=11008, act="silu", saved="8bit",
             input="raw", again=False, fmt="e4m3", grad="fp32", pad=0),
        # odd sizes; the block's input and a itself in 8 bits too, the input as the norm before it saves it
        dict(name="ffn grad odd", op="ffn_grad", rows=2011, cols=1003, hidden=2731, act="gelu", saved="8bit",
             input="8bit", again=True, fmt="int8", grad="fp32", pad=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "ffn", "ffn_grad"])
    fmt, pad = rng.choice(["e4m3", "int8"]), rng.choice([0, 0, 3, 64])
    if op.startswith("norm"):
        while True:
            rows, cols = _log(rng, 1, 32768), _log(rng, 64, 11008)
            if rng.random() < 0.5:
                cols = -(-cols // 64) * 64
            if rows * cols <= 16384 * 4096:
                break
        case = dict(op=op, rows=rows, cols=cols, resid=rng.choice(["bf16", "fp32"]), weights=rng.choice(["bf16", "fp32"]),
                    bias=rng.random() < 0.75, fmt=fmt, pad=pad)
        if op == "norm":
            case.update(add=rng.random() < 0.7, save=rng.choice(["", "xn", "h", "both"]))
        else:
            case.update(saved=rng.choice(["8bit", "raw"]), grad=rng.choice(["bf16", "fp32"]))
        return case
    while True:
        rows, cols, hidden = _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 64, 11008)
        if rng.random() < 0.6:
            cols, hidden = -(-cols // 64) * 64, -(-hidden // 64) * 64
        if rows * cols * hidden <= 8192 * 4096 * 11008 and rows * max(cols, hidden) <= 8192 * 11008:
            break
    case = dict(op=op, rows=rows, cols=cols, hidden=hidden, act=rng.choice(["silu", "gelu", "gelu_tanh"]), fmt=fmt, pad=pad)
    if op == "ffn":
        case.update(saved=rng.choice(["", "raw", "8bit"]))
    else:
        case.update(saved=rng.choice(["raw", "8bit"]), input=rng.choice(["raw", "8bit"]), again=rng.random() < 0.3,
                    grad=rng.choice(["bf16", "fp32"]))
    return case


# ------------------------------------------------------------------ the 8-bit form, in 32 bits

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _packed(rows, cols):
    return rows * (-(-cols // BLOCK)) * (BLOCK + 1)


def _pow2(n):
    return ((n + 127) << 23).view(torch.float32)


def _quantise(x, fmt):
    """(values on the code grid, k) of fp32 rows, in whole blocks."""
    short = -x.shape[1] % BLOCK
    if short:
        x = torch.cat([x, x.new_zeros(x.shape[0], short)], 1)
    b = x.view(x.shape[0], -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    # the exponent of top, one more where its mantissa is over F's
    over, emax = (0x1FFFFF, 8) if fmt == "e4m3" else (0x01FFFF, 6)
    k = (((top.view(torch.int32) + over) >> 23) - (127 + emax)).clamp(min=KMIN)
    v = b * _pow2(-k)
    if fmt == "e4m3":
        step = torch.frexp(v)[1].clamp(min=-5) - 4
        v = torch.round(v * _pow2(-step)) * _pow2(step)
    else:
        v = torch.round(v)
    return v, k


def _rounded(x, fmt):
    """What 8-bit rows of the fp32 rows x stand for; exact in bf16."""
    v, k = _quantise(x, fmt)
    return (v * _pow2(k)).view(x.shape[0], -1)[:, :x.shape[1]].to(torch.bfloat16)


def _encode(x, fmt):
    """The 8-bit rows of fp32 rows, as the bytes of their layout."""
    v, k = _quantise(x, fmt)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else v.to(torch.int8).view(torch.uint8)
    return torch.cat([codes.reshape(-1), (k + 127).to(torch.uint8).reshape(-1)])


def _decode(buf, rows, cols, fmt):
    pitch = -(-cols // BLOCK) * BLOCK
    codes = buf[:rows * pitch].view(rows, -1, BLOCK)
    k = buf[rows * pitch:].view(rows, -1, 1).to(torch.int32) - 127
    v = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()
    return (v * _pow2(k)).view(rows, pitch)[:, :cols]


# ------------------------------------------------------------------ inputs

def _activations(rows, cols, g, dev):
    """Rows as a transformer's: a few channels are ten times the others, and each has a mean of its own."""
    x = torch.randn(rows, cols, device=dev, generator=g) + 0.3 * torch.randn(cols, device=dev, generator=g)
    loud = torch.rand(cols, device=dev, generator=g) < 0.01
    return x * torch.where(loud, 10.0, 1.0)


def _held(x, dtype, pad):
    """x in its own type, in rows that may lie further apart."""
    out = torch.empty(x.shape[0], x.shape[1] + pad, dtype=dtype, device=x.device)[:, :x.shape[1]]
    out.copy_(x)
    return out


def _statistics(x, eps):
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + eps)
    return mean, rstd, c * rstd[:, None]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    (_prepare_norm if case["op"].startswith("norm") else _prepare_ffn)(case, s, g, dev)
    if own:  # the workspace that a program keeps beside its buffers
        import sharded_optimizer_step_amd as z
        rows, cols = case["rows"], case["cols"]
        if case["op"] == "norm_grad":
            s["ws"] = z.workspace(z.zero_layer_norm_grad_workspace_bytes(rows, cols))
        elif case["op"] == "ffn":
            s["ws"] = z.workspace(z.zero_block_ffn_workspace_bytes(rows, cols, case["hidden"]))
        elif case["op"] == "ffn_grad":
            s["ws"] = z.workspace(z.zero_block_ffn_grad_workspace_bytes(rows, cols, case["hidden"]))
    return s


def _grads(s, case, names, g, dev):
    for name, shape in names:
        s[name] = torch.empty(shape, dtype=_TYPES[case["grad"]], device=dev)
        if case["grad"] == "fp32":  # the sum of the micro-batches before this one
            s[name].normal_(0, 1e-2, generator=g)


def _prepare_norm(case, s, g, dev):
    rows, cols, pad = case["rows"], case["cols"], case["pad"]
    rt, wt, bf = _TYPES[case["resid"]], _TYPES[case["weights"]], torch.bfloat16
    new = lambda t: torch.empty(rows, cols + pad, dtype=t, device=dev)[:, :cols]  # noqa: E731
    s["eps"] = 1e-5
    s["w"] = (1 + 0.1 * torch.randn(cols, device=dev, generator=g)).to(wt)
    s["b"] = (0.1 * torch.randn(cols, device=dev, generator=g)).to(wt) if case["bias"] else None
    x = _activations(rows, cols, g, dev) * 2
    if case["op"] == "norm":
        s["x"] = _held(x, rt, pad)
        s["y"] = _held(_activations(rows, cols, g, dev), bf, pad) if case["add"] else None
        s["x_out"] = new(rt) if case["add"] else None
        s["h"] = new(bf)
        s["mean"], s["rstd"] = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        for n in ("xn", "h"):
            if case["save"] in (n, "both"):
                s["saved_" + n] = torch.empty(_packed(rows, cols), dtype=torch.uint8, device=dev)
                s["read_" + n] = torch.empty(rows, cols, dtype=bf, device=dev)
        return
    s["x_out"] = _held(x, rt, pad)
    s["mean"], s["rstd"], xn = _statistics(s["x_out"].float(), s["eps"])
    if case["saved"] == "8bit":
        s["saved_xn"] = _encode(xn, case["fmt"])
        s["x_out"] = s["mean"] = None
    s["dh"] = _held(torch.randn(rows, cols, device=dev, generator=g) * 1e-3, bf, pad)
    s["dx_out"] = _held(torch.randn(rows, cols, device=dev, generator=g) * 1e-3, rt, pad)
    s["dx"] = new(rt)
    s["dy"] = new(bf) if case["resid"] == "fp32" else None
    _grads(s, case, [("dw", cols)] + ([("db", cols)] if case["bias"] else []), g, dev)


def _prepare_ffn(case, s, g, dev):
    rows, cols, hidden, pad = case["rows"], case["cols"], case["hidden"], case["pad"]
    bf = torch.bfloat16
    new = lambda c: torch.empty(rows, c + pad, dtype=bf, device=dev)[:, :c]  # noqa: E731
    for n in ("w_gate", "w_up"):
        s[n] = _held(torch.randn(hidden, cols, device=dev, generator=g) * (cols ** -0.5), bf, 0)
    x = torch.randn(rows, cols, device=dev, generator=g)
    if case["op"] == "ffn":
        s["h"] = _held(x, bf, pad)
        s["a"] = new(hidden)
        if case["saved"] == "raw":
            s["gate"], s["up"] = new(hidden), new(hidden)
        elif case["saved"] == "8bit":
            for n in ("gate", "up"):
                s["saved_" + n] = torch.empty(_packed(rows, hidden), dtype=torch.uint8, device=dev)
                s["read_" + n] = torch.empty(rows, hidden, dtype=bf, device=dev)
        return
    for n in ("gate", "up"):
        v = torch.randn(rows, hidden, device=dev, generator=g)
        if case["saved"] == "raw":
            s[n] = _held(v, bf, pad)
        else:
            s["saved_" + n] = _encode(v, case["fmt"])
    s["da"] = _held(torch.randn(rows, hidden, device=dev, generator=g) * 1e-3, bf, pad)
    s["scale"] = None
    if case["input"] == "raw":
        s["h"] = _held(x, bf, pad)
    else:  # a norm's rows before their weight, which the products' columns then take
        s["saved_h"] = _encode(x, case["fmt"])
        s["scale"] = (1 + 0.1 * torch.randn(cols, device=dev, generator=g)).to(bf)
    s["dgate"], s["dup"], s["dh"] = new(hidden), new(hidden), new(cols)
    if case["again"]:
        s["saved_a"] = torch.empty(_packed(rows, hidden), dtype=torch.uint8, device=dev)
        s["read_a"] = torch.empty(rows, hidden, dtype=bf, device=dev)
    _grads(s, case, [("dw_gate", (hidden, cols)), ("dw_up", (hidden, cols))], g, dev)


# ------------------------------------------------------------------ one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _sum_into(s, name, value):
    """A gradient as its buffer takes it: added to an fp32 accumulator, or one bf16 replica."""
    if s["grad"] == "fp32":
        s[name] += value
        return s[name]
    return value.to(torch.bfloat16)


def _plain_norm(s):
    out = {}
    x = s["x"].float()
    if s["add"]:
        out["x_out"] = (x + s["y"].float()).to(s["x"].dtype)
        x = out["x_out"].float()
    out["mean"], out["rstd"], xn = _statistics(x, s["eps"])
    h = xn * s["w"].float()
    if s["bias"]:
        h = h + s["b"].float()
    out["h"] = h.to(torch.bfloat16)
    if s["save"] in ("xn", "both"):
        out["read_xn"] = _rounded(xn, s["fmt"])
    if s["save"] in ("h", "both"):
        out["read_h"] = _rounded(h, s["fmt"])
    return out


def _plain_norm_grad(s):
    if s["saved"] == "8bit":
        xn = _decode(s["saved_xn"], s["rows"], s["cols"], s["fmt"])
    else:
        xn = (s["x_out"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dh = s["dh"].float()
    v = dh * s["w"].float()
    dx = s["dx_out"].float() + s["rstd"][:, None] * (v - v.mean(1, keepdim=True) - xn * (v * xn).mean(1, keepdim=True))
    out = dict(dx=dx.to(s["dx_out"].dtype), dw=_sum_into(s, "dw", (dh * xn).sum(0)))
    if s["dy"] is not None:
        out["dy"] = dx.to(torch.bfloat16)
    if s["bias"]:
        out["db"] = _sum_into(s, "db", dh.sum(0))
    return out


def _act(g, kind):
    """(act(g), act'(g))"""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    h = s["h"].float()
    g, u = h @ s["w_gate"].float().t(), h @ s["w_up"].float().t()
    out = dict(a=(_act(g, s["act"])[0] * u).to(torch.bfloat16))
    if s["saved"] == "raw":
        out.update(gate=g.to(torch.bfloat16), up=u.to(torch.bfloat16))
    elif s["saved"] == "8bit":
        out.update(read_gate=_rounded(g, s["fmt"]), read_up=_rounded(u, s["fmt"]))
    return out


def _bf16(x):
    """64-bit values to the nearest bf16. By way of fp32, so one that this moves
    onto the middle of two bf16 values is moved back off it first."""
    f = x.float()
    bits = f.view(torch.int32)
    middle = ((bits & 0xFFFF) == 0x8000) & (f.double() != x)
    toward = torch.where(f.double().abs() > x.abs(), -1, 1).to(torch.int32)
    return torch.where(middle, bits + toward, bits).view(torch.float32).to(torch.bfloat16)


def _plain_ffn_grad(s):
    rows, hidden, cols = s["rows"], s["hidden"], s["cols"]
    if s["saved"] == "raw":
        g, u = s["gate"].float(), s["up"].float()
    else:
        g, u = _decode(s["saved_gate"], rows, hidden, s["fmt"]), _decode(s["saved_up"], rows, hidden, s["fmt"])
    # in 64 bits: fp32 sums are taken from these two after their rounding to bf16, where a
    # last bit next to the border of two values would count for 2^-8
    da, g, u = s["da"].double(), g.double(), u.double()
    f, df = _act(g, s["act"])
    out = dict(dgate=_bf16(da * u * df), dup=_bf16(da * f))
    dg, du = out["dgate"].float(), out["dup"].float()  # the products are those of the stored gradients
    out["dh"] = (dg @ s["w_gate"].float() + du @ s["w_up"].float()).to(torch.bfloat16)
    x = s["h"].float() if s["input"] == "raw" else _decode(s["saved_h"], rows, cols, s["fmt"]) * s["scale"].float()
    out["dw_gate"], out["dw_up"] = _sum_into(s, "dw_gate", dg.t() @ x), _sum_into(s, "dw_up", du.t() @ x)
    if s["again"]:
        out["read_a"] = _rounded((f * u).float(), s["fmt"])
    return out


_plain = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, ffn=_plain_ffn, ffn_grad=_plain_ffn_grad)


def _act8(z, s, name, cols):
    if "saved_" + name not in s:
        return None
    return z.Act8(s["rows"], cols, z.ACT8_E4M3 if s["fmt"] == "e4m3" else z.ACT8_INT8, s["saved_" + name])


def _kind(z, s):
    return {"silu": z.FFN_SILU, "gelu": z.FFN_GELU, "gelu_tanh": z.FFN_GELU_TANH}[s["act"]]


def _own_norm(s):
    import sharded_optimizer_step_amd as z
    xn, h = _act8(z, s, "xn", s["cols"]), _act8(z, s, "h", s["cols"])
    z.zero_layer_norm(z.LayerNorm(x=s["x"], y=s["y"], w=s["w"], b=s["b"], x_out=s["x_out"], h=s["h"], mean=s["mean"],
                                  rstd=s["rstd"], ckpt_xn=xn, ckpt_h=h, eps=s["eps"]))
    out = dict(mean=s["mean"], rstd=s["rstd"], h=s["h"])
    if s["add"]:
        out["x_out"] = s["x_out"]
    if xn is not None:
        z.zero_act8_load(xn, s["read_xn"])
        out["read_xn"] = s["read_xn"]
    if h is not None:
        z.zero_act8_load(h, s["read_h"])
        out["read_h"] = s["read_h"]
    return out


def _own_norm_grad(s):
    import sharded_optimizer_step_amd as z
    z.zero_layer_norm_grad(z.LayerNormGrad(
        dx=s["dx"], dh=s["dh"], dx_out=s["dx_out"], w=s["w"], x_out=s["x_out"], mean=s["mean"], rstd=s["rstd"],
        ckpt_xn=_act8(z, s, "xn", s["cols"]), dy=s["dy"], dw=s["dw"], db=s["db"] if s["bias"] else None),
        z.GRAD_ACCUMULATE if s["grad"] == "fp32" else 0, s["ws"])
    out = dict(dx=s["dx"], dw=s["dw"])
    if s["dy"] is not None:
        out["dy"] = s["dy"]
    if s["bias"]:
        out["db"] = s["db"]
    return out


def _own_ffn(s):
    import sharded_optimizer_step_amd as z
    gate, up = _act8(z, s, "gate", s["hidden"]), _act8(z, s, "up", s["hidden"])
    z.zero_block_ffn(z.BlockFfn(h=s["h"], w_gate=s["w_gate"], w_up=s["w_up"], a=s["a"], gate=s.get("gate"), up=s.get("up"),
                                ckpt_gate=gate, ckpt_up=up, act=_kind(z, s)), s["ws"])
    out = dict(a=s["a"])
    if s["saved"] == "raw":
        out.update(gate=s["gate"], up=s["up"])
    elif s["saved"] == "8bit":
        z.zero_act8_load(gate, s["read_gate"])
        z.zero_act8_load(up, s["read_up"])
        out.update(read_gate=s["read_gate"], read_up=s["read_up"])
    return out


def _own_ffn_grad(s):
    import sharded_optimizer_step_amd as z
    a = _act8(z, s, "a", s["hidden"])
    z.zero_block_ffn_grad(z.BlockFfnGrad(
        da=s["da"], dgate=s["dgate"], dup=s["dup"], w_gate=s["w_gate"], w_up=s["w_up"], gate=s.get("gate"), up=s.get("up"),
        ckpt_gate=_act8(z, s, "gate", s["hidden"]), ckpt_up=_act8(z, s, "up", s["hidden"]), dh=s["dh"], h=s.get("h"),
        ckpt_h=_act8(z, s, "h", s["cols"]), col_scale=s["scale"], dw_gate=s["dw_gate"], dw_up=s["dw_up"], ckpt_a=a,
        act=_kind(z, s)), z.GRAD_ACCUMULATE if s["grad"] == "fp32" else 0, s["ws"])
    out = dict(dgate=s["dgate"], dup=s["dup"], dh=s["dh"], dw_gate=s["dw_gate"], dw_up=s["dw_up"])
    if a is not None:
        z.zero_act8_load(a, s["read_a"])
        out["read_a"] = s["read_a"]
    return out


_own = dict(norm=_own_norm, norm_grad=_own_norm_grad, ffn=_own_ffn, ffn_grad=_own_ffn_grad)


# ------------------------------------------------------------------ work

def work(case):
    rows, cols = case["rows"], case["cols"]
    size = {"bf16": 2, "fp32": 4}
    n = rows * cols
    if case["op"] in ("norm", "norm_grad"):
        r, vector = size[case["resid"]], cols * size[case["weights"]]
        if case["op"] == "norm":
            byts = n * (r + 2) + vector * (1 + case["bias"]) + 8 * rows + (n * (r + 2) if case["add"] else 0)
            saves = {"": 0, "xn": 1, "h": 1, "both": 2}[case["save"]]
            # saved and read back: the 8 bits are written and read
            return dict(bytes=byts + saves * (2 * _packed(rows, cols) + 2 * n), flops=n * 10)
        byts = n * (2 + 2 * r) + vector + 4 * rows + (2 * n if case["resid"] == "fp32" else 0)
        byts += _packed(rows, cols) if case["saved"] == "8bit" else n * r + 4 * rows
        byts += (1 + case["bias"]) * cols * (2 if case["grad"] == "bf16" else 8)
        return dict(bytes=byts, flops=n * 14)
    hidden = case["hidden"]
    m, weights, saved = rows * hidden, 2 * hidden * cols, _packed(rows, hidden)
    if case["op"] == "ffn":
        extra = {"": 0, "raw": 4 * m, "8bit": 4 * saved + 4 * m}[case["saved"]]
        return dict(bytes=2 * n + 2 * weights + 2 * m + extra, flops=4 * m * cols)
    byts = 2 * m + (4 * m if case["saved"] == "raw" else 2 * saved) + 4 * m + 2 * weights + 2 * n
    byts += 2 * n if case["input"] == "raw" else _packed(rows, cols) + 2 * cols
    byts += 2 * hidden * cols * (2 if case["grad"] == "bf16" else 8) + (2 * saved + 2 * m if case["again"] else 0)
    return dict(bytes=byts, flops=8 * m * cols)


# ------------------------------------------------------------------ in 64 bits

def _grid64(fmt):
    """The non-negative values that a code can stand for, in order."""
    if fmt == "int8":
        return [float(i) for i in range(128)]
    return [m * 2.0**-9 for m in range(8)] + [(1 + m / 8) * 2.0**(e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest64(x, fmt):
    """Rows through the 8-bit form, by looking for the nearest code; ties go to the even one."""
    grid = torch.tensor(_grid64(fmt), dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    done = []
    for p in x.split(64 * BLOCK, 1):
        cols = p.shape[1]
        p = torch.nn.functional.pad(p, (0, -cols % BLOCK)).reshape(x.shape[0], -1, BLOCK)
        top = p.abs().amax(2, keepdim=True)
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0**-140) / grid[-1])) - 1)
        for _ in range(3):  # up from below to the first power of two that reaches
            unit = torch.where(top > grid[-1] * unit, unit * 2, unit)
        unit = unit.clamp(min=2.0**KMIN)
        a = (p.abs() / unit).clamp(max=grid[-1].item())
        i = torch.searchsorted(middle, a.contiguous())
        tie = (a == middle[i.clamp(max=middle.numel() - 1)]) & (i % 2 == 1)
        done.append((torch.sign(p) * grid[i + tie.to(i.dtype)] * unit).reshape(x.shape[0], -1)[:, :cols])
    return torch.cat(done, 1)


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


def _act64(kind, x):
    """The activation as x times a distribution function P with derivative D: (x P, P + x D)."""
    if kind == "silu":
        p = torch.special.expit(x)
        d = p * torch.special.expit(-x)
    elif kind == "gelu":
        p = torch.special.ndtr(x)
        d = torch.exp(-x.square() / 2) / (2 * math.pi) ** 0.5
    else:
        z = (8 / math.pi) ** 0.5 * (x + 0.044715 * x.pow(3))  # (1 + tanh(z / 2)) / 2 is the logistic function of z
        p = torch.special.expit(z)
        d = p * torch.special.expit(-z) * (8 / math.pi) ** 0.5 * (1 + 0.134145 * x.square())
    return x * p, p + x * d


def exact(case, seed):
    s = prepare(case, seed)
    rows, cols, fmt = case["rows"], case["cols"], case["fmt"]
    old = lambda n: s[n].double() if case["grad"] == "fp32" else 0.0  # noqa: E731
    if case["op"] == "norm":
        out = {}
        x = s["x"].double()
        if case["add"]:
            out["x_out"] = x + s["y"].double()
            # the norm is that of the stored residual stream, so it is taken from the rounded values
            x = out["x_out"].to(s["x"].dtype).double()
        out["mean"] = x.sum(1) / cols
        out["rstd"] = ((x - out["mean"].unsqueeze(1)).square().sum(1) / cols + s["eps"]) ** -0.5
        xn = (x - out["mean"].unsqueeze(1)) * out["rstd"].unsqueeze(1)
        out["h"] = torch.addcmul(s["b"].double() if case["bias"] else torch.zeros_like(xn), xn, s["w"].double())
        if case["save"] in ("xn", "both"):
            out["read_xn"] = _nearest64(xn, fmt)
        if case["save"] in ("h", "both"):
            out["read_h"] = _nearest64(out["h"], fmt)
        return out
    if case["op"] == "norm_grad":
        if case["saved"] == "8bit":
            xn = _read64(s["saved_xn"], rows, cols, fmt)
        else:
            xn = (s["x_out"].double() - s["mean"].double().unsqueeze(1)) * s["rstd"].double().unsqueeze(1)
        dh = s["dh"].double()
        v = s["w"].double() * dh
        along = (v * xn).sum(1, keepdim=True) / cols
        dx = s["dx_out"].double() + (v - v.sum(1, keepdim=True) / cols - along * xn) * s["rstd"].double().unsqueeze(1)
        out = dict(dx=dx, dw=old("dw") + torch.einsum("rc,rc->c", dh, xn))
        if s["dy"] is not None:
            out["dy"] = dx
        if case["bias"]:
            out["db"] = old("db") + dh.sum(0)
        return out
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    if case["op"] == "ffn":
        x = s["h"].double()
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        out = dict(a=u * _act64(case["act"], g)[0])
        if case["saved"] == "raw":
            out.update(gate=g, up=u)
        elif case["saved"] == "8bit":
            out.update(read_gate=_nearest64(g, fmt), read_up=_nearest64(u, fmt))
        return out
    if case["saved"] == "raw":
        g, u = s["gate"].double(), s["up"].double()
    else:
        g, u = (_read64(s["saved_" + n], rows, case["hidden"], fmt) for n in ("gate", "up"))
    f, df = _act64(case["act"], g)
    out = dict(dgate=s["da"].double() * df * u, dup=s["da"].double() * f)
    if case["again"]:
        out["read_a"] = _nearest64(f * u, fmt)
    # the gradients are stored in bf16, and what follows is taken from them
    dg, du = (torch.ldexp(torch.round(torch.frexp(out[n])[0] * 256) / 256, torch.frexp(out[n])[1]) for n in ("dgate", "dup"))
    out["dh"] = torch.mm(dg, wg).addmm_(du, wu)
    x = s["h"].double() if case["input"] == "raw" else _read64(s["saved_h"], rows, cols, fmt) * s["scale"].double()
    out["dw_gate"], out["dw_up"] = old("dw_gate") + torch.mm(dg.t(), x), old("dw_up") + torch.mm(du.t(), x)
    return out
