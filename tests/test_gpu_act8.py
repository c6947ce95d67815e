"""8-bit activation checkpoints and the weight gradient taken from one, on the
GPU, against plain 64-bit forms: codes and scales bit for bit, every format,
type, odd size, stride and alignment; every code of both formats through the
decoder; blocks with inf and NaN; buffers past 2^32 bytes; streams, captured
graphs and repeated calls."""
import numpy as np
import pytest
import torch

import sharded_optimizer_step_amd as z
from block_cases import FORMATS, U, assert_within, canary_ok, decode_act8, round_act8, strided

pytestmark = pytest.mark.gpu


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


def randn(rows, cols, seed, dtype=torch.float32):
    x = torch.randn(rows, cols, device="cuda", generator=gen(seed))
    return (x * torch.exp2(torch.randint(-3, 4, (cols,), device="cuda", generator=gen(seed + 1)))).to(dtype)


def save(x, fmt):
    ck = z.new_act8(x.shape[0], x.shape[1], fmt)
    ck.buf.fill_(0xAB)
    z.zero_act8_save(x, ck)
    return ck


SIZES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 31), (4, 32), (7, 33), (1, 64), (63, 65), (129, 771), (33, 1000), (2, 4096),
         (257, 513), (1000, 40), (3, 11008)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_save_is_nearest_code_and_load_is_exact(rows, cols, dtype, fmt):
    x = randn(rows, cols, 11 * rows + cols, dtype)
    ck = save(x, FORMATS[fmt])
    want = round_act8(x.double().cpu().numpy(), FORMATS[fmt])
    got, _ = decode_act8(ck)
    assert np.array_equal(got, want)
    for out_type in (torch.bfloat16, torch.float32):
        out = torch.full((rows, cols), 5.0, dtype=out_type, device="cuda")
        z.zero_act8_load(ck, out)
        assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 3), (8, 0), (64, 5)])
def test_strides_and_alignments(fmt, dtype, pad, offset):
    rows, cols = 19, 203
    x = randn(rows, cols, 5, dtype)
    v, _ = strided(x, pad, offset)
    ck, flat = save(v, FORMATS[fmt]), save(x, FORMATS[fmt])
    assert torch.equal(ck.buf, flat.buf)
    out, buf = strided(torch.zeros_like(x), pad, offset)
    z.zero_act8_load(ck, out)
    want = torch.zeros_like(x)
    z.zero_act8_load(flat, want)
    assert torch.equal(out, want) and canary_ok(buf, rows, cols, pad, offset)


@pytest.mark.parametrize("fmt", FORMATS)
def test_scales_over_the_whole_range(fmt):
    # one block for every exponent of fp32, its largest value on both sides of F * 2^k
    f = 448.0 if fmt == "e4m3" else 127.0
    e = np.arange(-149, 120)
    tops = np.concatenate([np.ldexp(1.0, e), np.ldexp(f / 256, e), np.nextafter(np.ldexp(f / 256, e).astype(np.float32), np.float32(np.inf))])
    x = (tops[:, None] * np.linspace(-1, 1, 32)[None, :]).astype(np.float32)
    x[:, 0] = tops
    ck = save(torch.tensor(x, device="cuda"), FORMATS[fmt])
    got, _ = decode_act8(ck)
    assert np.array_equal(got, round_act8(x.astype(np.float64), FORMATS[fmt]))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_and_nonfinite_blocks(fmt, dtype):
    x = randn(6, 100, 3, dtype)
    x[0] = 0
    x[1, 40] = float("inf")
    x[2, 99] = float("-inf")
    x[3, 0] = float("nan")
    x[4, 31], x[4, 32] = torch.finfo(dtype).max, torch.finfo(dtype).min
    x[5, 64:96] = 0
    ck = save(x, FORMATS[fmt])
    want = round_act8(x.double().cpu().numpy(), FORMATS[fmt])
    out = torch.zeros(6, 100, device="cuda")
    z.zero_act8_load(ck, out)
    assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[1, 32:64]).all() and np.isfinite(want[1, :32]).all() and np.isfinite(want[1, 64:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_and_scale_decodes(fmt):
    # one row for each scale byte that a save writes (and NaN), every code in 8 blocks
    scales = list(range(10, 250)) + [255]
    codes = np.tile(np.arange(256, dtype=np.uint8), (len(scales), 1))
    if fmt == "e4m3":
        codes[:, [127, 255]] = 0
    else:
        codes[:, 128] = 0
    buf = np.concatenate([codes.reshape(-1), np.repeat(np.array(scales, np.uint8), 8)])
    ck = z.Act8(len(scales), 256, FORMATS[fmt], torch.tensor(buf, device="cuda"))
    want, _ = decode_act8(ck)
    want = np.where(np.abs(want) >= 2.0**128, np.copysign(np.inf, want), want)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.zeros(len(scales), 256, dtype=dtype, device="cuda")
        z.zero_act8_load(ck, out)
        assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)
    # and through the weight gradient: dy picks one row, so dw is that row, exactly
    rows = [i for i, s in enumerate(scales) if 40 <= s <= 220]
    dy = torch.zeros(len(scales), len(rows), dtype=torch.bfloat16, device="cuda")
    for j, r in enumerate(rows):
        dy[r, j] = 1.0
    dw = torch.zeros(len(rows), 256, device="cuda")
    n = sum(s <= 240 for s in scales)  # up to 2^113, so that nothing in a column is infinite
    keep = z.Act8(n, 256, FORMATS[fmt], torch.tensor(
        np.concatenate([codes[:n].reshape(-1), np.repeat(np.array(scales[:n], np.uint8), 8)]), device="cuda"))
    ws = z.workspace(z.zero_act8_wgrad_workspace_bytes(n, len(rows), 256))
    z.zero_act8_wgrad(dy[:n], keep, dw, 0, ws)
    assert np.array_equal(dw.double().cpu().numpy(), want[rows])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,outs,cols", [(70, 40, 96), (300, 300, 300)])
def test_wgrad_of_the_largest_and_smallest_blocks(rows, outs, cols, fmt):
    # finite values up to 1.75 * 2^127, and as small as a block's smallest scale
    # holds: every decoded value is finite, and with dy near 1 / max so are the sums
    for top, size in ((127, 2.0**-100), (-110, 2.0**60)):
        sign = torch.sign(randn(rows, cols, 5))
        mant = 1 + torch.rand(rows, cols, device="cuda", generator=gen(6)) * 0.75
        x = (sign.double() * mant.double() * 2.0**top).to(torch.float32)
        ck = save(x, FORMATS[fmt])
        dy = (torch.randn(rows, outs, device="cuda", generator=gen(7)).double() * size).to(torch.bfloat16)
        xs = torch.tensor(decode_act8(ck)[0], device="cuda")
        assert bool(xs.abs().max() < 2.0**128)
        wgrad_check(ck, dy, xs, torch.empty(outs, cols, device="cuda"), 0, None, (fmt, top))


def wgrad_case(rows, outs, cols, fmt, seed, dy_pad=0, dy_offset=0):
    x = randn(rows, cols, seed)
    ck = save(x, fmt)
    dy, _ = strided((torch.randn(rows, outs, device="cuda", generator=gen(seed + 2)) * 1e-3).to(torch.bfloat16), dy_pad, dy_offset)
    return ck, dy, torch.tensor(decode_act8(ck)[0], device="cuda")


def wgrad_check(ck, dy, xs, dw, flags, scale=None, where=""):
    rows, outs, cols = ck.rows, dy.shape[1], ck.cols
    old = dw.double().clone()
    ws = z.workspace(z.zero_act8_wgrad_workspace_bytes(rows, outs, cols))
    if ws is not None:
        ws.fill_(0xFF)
    z.zero_act8_wgrad(dy, ck, dw, flags, ws, col_scale=scale)
    want = dy.double().t().contiguous() @ xs
    mag = dy.double().abs().t().contiguous() @ xs.abs()
    if scale is not None:
        want, mag = want * scale.double(), mag * scale.double().abs()
    if flags:
        want, mag = want + old, mag + old.abs()
    # a chain of at most `rows` fp32 additions in the matrix unit, which may
    # drop the bits below a step where a rounding would keep half of one
    assert_within(dw, want, mag, 2 * (rows + 8) * U, where)
    # and without a bias: far less than that in the 2-norm, sqrt(rows) steps
    off = (dw.double() - want).norm() / want.norm().clamp(min=1e-300)
    assert off <= (2.0**-8 if dw.dtype == torch.bfloat16 else 0) + 2 * U * (rows**0.5 + 8), (where, off)


WGRAD = [(1, 1, 1), (1, 40, 33), (2, 8, 64), (31, 16, 16), (32, 17, 15), (33, 128, 128), (64, 129, 127), (65, 127, 130),
         (100, 200, 333), (192, 768, 768), (257, 300, 100), (1537, 1000, 771), (9000, 130, 70), (640, 1408, 1152)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,outs,cols", WGRAD)
def test_wgrad(rows, outs, cols, fmt):
    ck, dy, xs = wgrad_case(rows, outs, cols, FORMATS[fmt], rows + 3 * cols)
    g = gen(9)
    for dtype, flags, scaled in ((torch.bfloat16, 0, None), (torch.float32, 0, torch.bfloat16),
                                 (torch.float32, z.GRAD_ACCUMULATE, torch.float32)):
        dw = torch.randn(outs, cols, device="cuda", generator=g).to(dtype)
        scale = None if scaled is None else (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(scaled)
        wgrad_check(ck, dy, xs, dw, flags, scale, (dtype, flags, scaled))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,outs,cols,pad,offset", [(70, 131, 65, 1, 1), (300, 260, 300, 3, 5), (64, 128, 256, 8, 0),
                                                       (2100, 33, 47, 5, 2)])
def test_wgrad_strides_alignments_and_what_lies_beyond(rows, outs, cols, pad, offset, dtype):
    ck, dy, xs = wgrad_case(rows, outs, cols, z.ACT8_E4M3, 21, pad, offset)
    dw, buf = strided(torch.zeros(outs, cols, dtype=dtype, device="cuda"), pad, offset)
    wgrad_check(ck, dy, xs, dw, 0)
    assert canary_ok(buf, outs, cols, pad, offset)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("outs,cols", [(4097, 4097), (4103, 4072)])
def test_wgrad_of_whole_and_split_tiles(outs, cols, fmt):
    # more tiles than fit the chip at once: the ones left over are split over the rows
    rows = 2048
    n = z.zero_act8_wgrad_workspace_bytes(rows, outs, cols)
    assert 0 < n < 4 * outs * cols
    ck, dy, xs = wgrad_case(rows, outs, cols, FORMATS[fmt], 3)
    for dtype, flags in ((torch.bfloat16, 0), (torch.float32, z.GRAD_ACCUMULATE)):
        dw = torch.randn(outs, cols, device="cuda", generator=gen(4)).to(dtype)
        scale = (1 + 0.1 * torch.randn(cols, device="cuda", generator=gen(5))).bfloat16()
        wgrad_check(ck, dy, xs, dw, flags, scale, dtype)


def test_wgrad_of_no_rows_writes_zeros_or_nothing():
    ck = z.new_act8(0, 40, z.ACT8_INT8)
    dy = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        dw = torch.full((24, 40), 3.0, dtype=dtype, device="cuda")
        z.zero_act8_wgrad(dy, ck, dw)
        assert torch.equal(dw, torch.zeros_like(dw))
        dw.fill_(3.0)
        z.zero_act8_wgrad(dy, ck, dw, col_scale=torch.full((40,), float("inf"), device="cuda"))
        assert torch.equal(dw, torch.zeros_like(dw))
    dw = torch.full((24, 40), 3.0, device="cuda")
    z.zero_act8_wgrad(dy, ck, dw, z.GRAD_ACCUMULATE)
    assert torch.equal(dw, torch.full_like(dw, 3.0))


def test_empty_sizes_are_no_ops():
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        ck = z.new_act8(rows, cols)
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        z.zero_act8_save(x, ck)
        z.zero_act8_load(ck, x)
    ck = save(randn(4, 8, 1), z.ACT8_E4M3)
    z.zero_act8_wgrad(torch.empty(4, 0, dtype=torch.bfloat16, device="cuda"), ck, torch.empty(0, 8, device="cuda"))


def test_wgrad_nonfinite_activations_reach_their_columns_only():
    ck0, dy, xs = wgrad_case(300, 140, 200, z.ACT8_E4M3, 4)
    x = randn(300, 200, 4)
    x[17, 70] = float("nan")
    ck = save(x, z.ACT8_E4M3)
    dw = torch.zeros(140, 200, device="cuda")
    ws = z.workspace(z.zero_act8_wgrad_workspace_bytes(300, 140, 200))
    z.zero_act8_wgrad(dy, ck, dw, 0, ws)
    assert torch.isnan(dw[:, 64:96]).all() and torch.isfinite(dw[:, :64]).all() and torch.isfinite(dw[:, 96:]).all()
    dy = dy.clone()
    dy[5, 9] = float("inf")
    z.zero_act8_wgrad(dy, ck0, dw, 0, ws)
    assert (~torch.isfinite(dw[9])).all() and torch.isfinite(dw[:9]).all() and torch.isfinite(dw[10:]).all()


def test_offsets_past_32_bits():
    # x and dy are the last rows of buffers of more than 2^32 bytes, reached by a long row stride
    rows, cols, ld = 70, 96, 1 << 25
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = big.view(rows, ld)[:, :cols]
    x.copy_(randn(rows, cols, 8))
    ck = save(x, z.ACT8_INT8)
    assert np.array_equal(decode_act8(ck)[0], round_act8(x.double().cpu().numpy(), z.ACT8_INT8))
    out = big.view(rows, ld)[:, 128:128 + cols]
    z.zero_act8_load(ck, out)
    assert np.array_equal(out.double().cpu().numpy(), decode_act8(ck)[0])
    dw = torch.zeros(cols, cols, device="cuda")
    wgrad_check(ck, x, torch.tensor(decode_act8(ck)[0], device="cuda"), dw, 0)
    del big, x, out
    # a checkpoint of more than 2^32 bytes: its first and last rows
    rows, cols = 140000, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in (0, 1, rows // 2, rows - 2, rows - 1):
        x[r] = randn(1, cols, r, torch.bfloat16)[0]
    ck = save(x, z.ACT8_E4M3)
    x.fill_(9.0)
    z.zero_act8_load(ck, x)
    for r in (0, 1, rows // 2, rows - 2, rows - 1):
        want = round_act8(randn(1, cols, r, torch.bfloat16).double().cpu().numpy(), z.ACT8_E4M3)
        assert np.array_equal(x[r:r + 1].double().cpu().numpy(), want)
    assert float(x[2:rows // 2].abs().max()) == 0.0


def test_calls_are_repeatable_and_streams_are_honoured():
    ck, dy, xs = wgrad_case(5000, 200, 300, z.ACT8_INT8, 6)
    n = z.zero_act8_wgrad_workspace_bytes(5000, 200, 300)
    assert n > 0  # split over the rows
    want = torch.zeros(200, 300, device="cuda")
    z.zero_act8_wgrad(dy, ck, want, 0, z.workspace(n))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):  # two calls at once, each with a workspace of its own
        s = streams[i % 2]
        with torch.cuda.stream(s):
            o = torch.zeros(200, 300, device="cuda")
            ws = z.workspace(n)
            z.zero_act8_wgrad(dy, ck, o, 0, ws)
            outs.append((o, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o, _ in outs)


def test_captured_and_replayed():
    rows, outs, cols = 3000, 150, 260
    x = randn(rows, cols, 1, torch.bfloat16)
    dy = (randn(rows, outs, 2) * 1e-3).to(torch.bfloat16)
    ck, ck2 = z.new_act8(rows, cols), z.new_act8(rows, cols)
    out = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(outs, cols, device="cuda")
    ws, ws2 = (z.workspace(z.zero_act8_wgrad_workspace_bytes(rows, outs, cols)) for _ in range(2))
    assert ws is not None

    def go(ck, out, dw, ws):
        z.zero_act8_save(x, ck)
        z.zero_act8_load(ck, out)
        z.zero_act8_wgrad(dy, ck, dw, z.GRAD_ACCUMULATE, ws)

    go(ck, out, dw, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(ck, out, dw, ws)
    dw.zero_()
    eager = torch.zeros_like(dw)
    eager_out = torch.zeros_like(out)
    for i in range(4):
        x.copy_(randn(rows, cols, 30 + i, torch.bfloat16))
        graph.replay()
        go(ck2, eager_out, eager, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, eager_out) and torch.equal(dw, eager) and torch.equal(ck.buf, ck2.buf), i
