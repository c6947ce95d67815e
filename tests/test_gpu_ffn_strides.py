"""The feed-forward block's gradients on the GPU where the columns of some
operands are a multiple of 8 and those of others are not, so that some are
copied to the workspace and others read where they are, and the two of a pair
lie at strides and addresses of their own: against the 64-bit formulas, and bit
for bit what packed operands give, whose sums have the same order."""
import pytest
import torch

import sharded_optimizer_step_amd as z
from test_gpu_block_ffn import Placed, backward, check_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    z.lib()
    torch.cuda.set_device(0)
    yield


SIZES = [(300, 767, 520), (900, 1003, 1024), (300, 520, 767), (2011, 1024, 2731)]
RESULTS = ("dgate", "dup", "dh", "dw_gate", "dw_up")


def again(b, sizes):
    ws = z.workspace(max(1, z.zero_block_ffn_grad_workspace_bytes(*sizes)))
    ws.fill_(255)
    z.zero_block_ffn_grad(b, 0, ws)


# (columns more than there are, elements before the first row) of the first and the second of a pair
@pytest.mark.parametrize("first,second", [((0, 0), (8, 0)), ((8, 0), (0, 0)), ((24, 0), (8, 8)), ((8, 0), (8, 1)), ((8, 3), (16, 0)),
                                          ((0, 0), (3, 0))])
@pytest.mark.parametrize("pair", [("dgate", "dup"), ("w_gate", "w_up")])
@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_pairs_of_operands_that_lie_differently(rows, cols, hidden, pair, first, second):
    r = backward(rows, cols, hidden, saved="raw", accumulate=False)
    b = r[0]
    want = [getattr(b, k).clone() for k in RESULTS]
    places = [Placed(*first), Placed(*second)]
    for k, place in zip(pair, places):
        setattr(b, k, place(getattr(b, k)))
    for k in ("dh", "dw_gate", "dw_up"):
        getattr(b, k).zero_()
    again(b, (rows, cols, hidden))
    check_backward(*r)
    for place in places:
        place.check()
    for k, w in zip(RESULTS, want):
        assert torch.equal(getattr(b, k), w), k


def far_apart(t, ld):
    """t in rows of `ld` elements."""
    v = torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=t.dtype, device="cuda").as_strided(t.shape, (ld, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("names,rows,cols,hidden,ld", [(("dgate", "dup"), 300, 767, 520, 1 << 22), (("dgate",), 300, 767, 520, 1 << 23),
                                                       (("w_gate", "w_up"), 300, 520, 767, 1 << 22), (("h",), 300, 520, 767, 1 << 25)])
def test_rows_that_32_bit_offsets_do_not_reach(names, rows, cols, hidden, ld):
    r = backward(rows, cols, hidden, saved="raw", accumulate=False)
    b = r[0]
    want = [getattr(b, k).clone() for k in RESULTS]
    for k in names:
        setattr(b, k, far_apart(getattr(b, k), ld + 8))
    again(b, (rows, cols, hidden))
    check_backward(*r)
    for k, w in zip(RESULTS, want):
        assert torch.equal(getattr(b, k), w), k
