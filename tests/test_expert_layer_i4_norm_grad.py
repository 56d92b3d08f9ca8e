"""The 4-bit layer's norm() in a training step: the rstd it leaves is the direct call's, and the gradients taken with it are the
formulas'."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300.expert_layer import ExpertLayerI4
from test_block_norm import BF, backward, check_forward, check_grad, gen, inputs, normal

pytestmark = pytest.mark.gpu


def layer(H, b, post_gamma, gamma):
    E, I, group = 2, 16, 128

    def weight(N, D):
        return (torch.zeros((E, N, -(-D // 128) * 64), dtype=torch.uint8, device="cuda"),
                torch.ones((E, N, -(-(-(-D // group)) // 4) * 4), device="cuda").to(torch.float8_e4m3fn),
                torch.ones((E, N), device="cuda"))

    return ExpertLayerI4(gamma, weight(2 * I, H), weight(H, I), max_tokens=b, top_k=1, post_gamma=post_gamma, residual_scale=0.5)


@pytest.mark.parametrize("post,token,channel", [(True, True, True), (False, True, False)])
@pytest.mark.parametrize("H", [264, 2056, 4104])
def test_gradients_with_the_rstd_of_the_layer(H, post, token, channel):
    g = gen(H)
    for b in (1, 37):
        d = inputs(g, b, H, post, token, channel)
        m = layer(H, 40, d["post_gamma"], d["pre_gamma"])
        out, rstd = torch.full((b, H), 77.0, dtype=BF, device="cuda"), torch.full((b, 2), 77.0, device="cuda")
        before = d["x"].clone(), d["residual"].clone()
        got, rows = m.norm(d["x"], d["residual"], residual_out=out, token_gate=d["token_gate"], channel_gate=d["channel_gate"],
                           rstd=rstd)
        assert got is out and torch.equal(d["x"], before[0]) and torch.equal(d["residual"], before[1])
        check_forward(d, (out, rows, rstd), residual_scale=0.5)
        d_y, d_out = normal(g, b, H), normal(g, b, H)
        check_grad(d, d_y, d_out, backward(d, d_y, d_out, rstd, residual_scale=0.5), residual_scale=0.5)
        with pytest.raises(ValueError, match="rstd"):
            m.norm(d["x"], d["residual"], residual_out=out, rstd=torch.empty((b, 1), device="cuda"))
        with pytest.raises(ValueError, match="norm"):  # the refused one left no rows to route
            m.experts(torch.zeros((b, 1), dtype=torch.int32, device="cuda"), torch.ones((b, 1), device="cuda"), out)
    assert mt.moe_tail_take_device_error() == 0
