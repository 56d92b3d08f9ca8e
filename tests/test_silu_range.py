"""silu(gate) * up in 8 bits over the whole range of gates, against the definition in 64 bits.

Tolerances: an exponential of half the gate (2 units in the last place) enters twice, four products and an addition are
rounded (half a unit each) and the quotient is within 2 units: under 10 * 2^-23 = 1.2e-6 of the value.  The scale adds a
division, so 2e-6 is asked of it, and of a value half a step of the rounding plus twice that of its magnitude.
"""
import pytest
import torch

import moe_decode_tail_gb300 as mt

pytestmark = pytest.mark.gpu

BF, I8, F32, F64, E4 = torch.bfloat16, torch.int8, torch.float32, torch.float64, torch.float8_e4m3fn
MOST = {I8: 127.0, E4: 448.0}


def check(q, scale, v, group):
    rows, width = v.shape
    size = group or width
    for g in range(-(-width // size)):
        part, got = v[:, g * size:(g + 1) * size], q[:, g * size:(g + 1) * size].to(F32).to(F64)
        sc = (scale[:, g] if group else scale).to(F64)
        want = part.abs().amax(1) / MOST[q.dtype]
        assert (want > 1e-36).all()
        assert ((sc - want).abs() <= 2e-6 * want).all(), ((sc - want).abs() / want).max()
        ratio = part / want[:, None]
        if q.dtype == I8:
            half = torch.full_like(ratio, 0.5)
        else:  # three bits after the leading one, down to 2^-9
            half = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp_min(1e-30))).clamp_min(-6.0) - 4)
        off = (got - ratio).abs()
        assert (off <= half * (1 + 1e-6) + 4e-6 * ratio.abs() + 1e-9).all(), (off - half).max()


# gate, and a size of up at which the products stay in FP32's normal range
GATES = [(-0.01, 1.0), (-5.0, 1.0), (-20.0, 1e10), (-60.0, 1e10), (-85.0, 1e10), (-87.0, 1e10), (-87.5, 1e10), (-88.0, 1e30),
         (-88.5, 1e30), (-89.0, 1e30), (-100.0, 1e37), (-120.0, 1e37), (-150.0, 1e37), (0.01, 1.0), (20.0, 1.0), (87.5, 1e30),
         (88.5, 1e30), (150.0, 1e-20), (1e20, 1e10)]


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("gate,size", GATES)
def test_rows_of_one_gate(gate, size, group, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(abs(gate) * 10) % 1000)
    rows, width = 5, 520
    gate_up = torch.empty((rows, 2 * width), dtype=BF, device="cuda")
    gate_up[:, :width] = gate
    gate_up[:, width:] = torch.randn((rows, width), generator=g, device="cuda").clamp(-3, 3) * size
    q = torch.empty((rows, width), dtype=dtype, device="cuda")
    scale = torch.empty((rows, 5) if group else (rows,), device="cuda")
    mt.moe_tail_silu_quant(gate_up, q, scale, group=group)
    z, up = gate_up[:, :width].to(F64), gate_up[:, width:].to(F64)
    check(q, scale, z / (1 + torch.exp(-z)) * up, group)


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
def test_every_gate_below_which_a_factor_leaves_the_range(group, dtype):
    # all BF16 gates from -128 to -16, one to a row, up chosen so that the largest product of the row is about 1
    gates = torch.arange(-128.0, -16.0, 0.5, device="cuda").to(BF)
    rows, width = len(gates), 128
    z = gates.to(F64)
    silu = z / (1 + torch.exp(-z))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    up = torch.randn((rows, width), generator=g, device="cuda", dtype=F64) * (1 / silu.abs()).clamp(max=1e37)[:, None]
    gate_up = torch.cat([gates[:, None].expand(rows, width), up.clamp(-3e38, 3e38).to(BF)], dim=1).contiguous()
    q = torch.empty((rows, width), dtype=dtype, device="cuda")
    scale = torch.empty((rows, 1) if group else (rows,), device="cuda")
    mt.moe_tail_silu_quant(gate_up, q, scale, group=group)
    check(q, scale, silu[:, None] * gate_up[:, width:].to(F64), group)
