"""The norm gradient for rows above 2048 columns at many rows: every stage of a thread block's ring used several times over (six
or eight of them), and more than 32 rows for a thread block or cluster, whose scalars come 32 rows at a time.  Tolerances are
those of the fewer rows' tests: they grow with the rows."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from test_block_norm import backward, check_grad, forward, gen, inputs, normal

pytestmark = pytest.mark.gpu

SIZES = [(10000, 2056), (8001, 3000), (6000, 4096), (7777, 4104), (1700, 9000), (1501, 20000), (1100, 32768)]


@pytest.mark.parametrize("post,token,channel", [(True, True, True), (False, True, True), (True, False, False)])
@pytest.mark.parametrize("b,H", SIZES)
def test_gradients(b, H, post, token, channel):
    g = gen(b)
    d = inputs(g, b, H, post, token, channel)
    d_y, d_out = normal(g, b, H), normal(g, b, H, std=0.5)
    rstd = forward(d)[2]
    got = backward(d, d_y, d_out, rstd)
    check_grad(d, d_y, d_out, got)
    again = backward(d, d_y, d_out, rstd)
    assert all(torch.equal(got[k], again[k]) for k in got)  # the same bits every time
    none = backward(d, d_y, None, rstd)
    check_grad(d, d_y, None, none)
    # in place
    work = torch.empty(mt.moe_tail_block_norm_grad_workspace_bytes(b, H), dtype=torch.uint8, device="cuda")
    mt.moe_tail_block_norm_grad(d_y, d_out, d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], rstd, d_y, d_out, work,
                                token_gate=d["token_gate"], channel_gate=d["channel_gate"])
    assert torch.equal(d_y, got["d_x"]) and torch.equal(d_out, got["d_residual"])
    assert mt.moe_tail_take_device_error() == 0
