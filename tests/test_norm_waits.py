"""The norm gradient for rows above 2048 columns when its waits run out: with a limit shorter than a memory trip a call gives up,
says so, leaves what surrounds its outputs as it was and the device usable.  What a call that gave up wrote is undefined."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from test_block_norm import BF, backward, check_grad, forward, gen, inputs, normal

pytestmark = pytest.mark.gpu

# one thread block a row (eight and six rows ahead), and clusters of two, four, six and eight; more rows than a block has ahead
SIZES = [(3000, 2056), (2000, 4096), (1, 4096), (900, 4104), (600, 9000), (500, 20000), (1, 32768), (300, 32768)]


@pytest.mark.parametrize("b,H", SIZES)
def test_waits_that_run_out(b, H):
    g = gen(H)
    d = inputs(g, b, H, True, True, True)
    d_y, d_out = normal(g, b, H), normal(g, b, H)
    rstd = forward(d)[2]
    assert mt.moe_tail_take_device_error() == 0
    for limit in (1, 1, 100, 400, 1000, 3000):  # nanoseconds: 1 gives up in any case, the others here and there
        mt.moe_tail_set_stage_wait_limit(limit)
        try:
            for _ in range(3):
                backward(d, d_y, d_out, rstd)
            torch.cuda.synchronize()
        finally:
            mt.moe_tail_set_stage_wait_limit(0)
        bits = mt.moe_tail_take_device_error()
        assert bits in ((1,) if limit == 1 else (0, 1)), (limit, bits)
        got = backward(d, d_y, d_out, rstd)
        check_grad(d, d_y, d_out, got)
        assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("b,H", [(1000, 3000), (400, 9000)])
def test_a_call_that_gave_up_writes_nothing_outside_its_outputs(b, H):
    g, buffers = gen(H), []

    def new(dtype, *shape):
        n = torch.empty(0, dtype=dtype).element_size() * torch.Size(shape).numel()
        whole = torch.full((n + (1 << 16),), 0xA5, dtype=torch.uint8, device="cuda")
        buffers.append((whole, n))
        return whole[1 << 15:(1 << 15) + n].view(dtype).view(shape)

    d = inputs(g, b, H, True, True, False)
    d_y, rstd = normal(g, b, H), forward(d)[2]
    for limit in (1, 500):
        mt.moe_tail_set_stage_wait_limit(limit)
        try:
            mt.moe_tail_block_norm_grad(d_y, None, d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], rstd, new(BF, b, H),
                                        new(BF, b, H), new(torch.uint8, mt.moe_tail_block_norm_grad_workspace_bytes(b, H)),
                                        token_gate=d["token_gate"], d_token_gate=new(torch.float32, b))
            torch.cuda.synchronize()
        finally:
            mt.moe_tail_set_stage_wait_limit(0)
    assert mt.moe_tail_take_device_error() == 1
    for whole, n in buffers:
        assert (whole[:1 << 15] == 0xA5).all() and (whole[(1 << 15) + n:] == 0xA5).all()
