"""The 4-bit products where a row, a sum or a gate is near the ends of FP32's range although the result is an ordinary number.

Tolerances: a row with one column, or with a whole number of equal ones, has sums that are exact in FP32 and results that are
BF16 numbers: equal bits are asked.  silu's results round once (2^-8 of the value), and the exponential of half a gate, of
which two are multiplied, is off by up to half of 2^-149 where it is below 2^-126: 2^-18 of itself for the gates here."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300.expert_layer import pack_int4

pytestmark = pytest.mark.gpu

BF, I8, F64, E4 = torch.bfloat16, torch.int8, torch.float64, torch.float8_e4m3fn
# rows and channels: the kernel for few rows; tiles of 16, 32 and 64 rows; wide tiles
FORMS = [(1, 8), (8, 24), (16, 24), (30, 136), (64, 8), (2600, 5136)]


def product(x, q, gs, cs, group, gated=False):
    """x [R, D] by one weight q [channels, D] with scales gs [channels, groups] and cs [channels]."""
    channels = q.shape[0]
    padded = torch.nn.functional.pad(gs, (0, -gs.shape[1] % 4)).to(E4)
    out = torch.full((x.shape[0], channels // 2 if gated else channels), 77.0, dtype=BF, device="cuda")
    fn = mt.moe_tail_gated_product_i4 if gated else mt.moe_tail_expert_product_i4
    return fn(x, pack_int4(q)[None], padded[None].contiguous(), cs[None], out, group=group)


# x, q, group scale, channel scale; columns of the row that are x
CASES = [(2.0 ** 123, 7, 448.0, 2.0 ** -120, 1), (2.0 ** 126, 7, 2.0 ** -9, 2.0 ** -116, 128), (-2.0 ** 127, -8, 0.25, 2.0 ** -126, 4),
         (2.0 ** 120, 7, 448.0, 2.0 ** -120, 128), (2.0 ** -100, 1, 2.0 ** -9, 2.0 ** 100, 1), (2.0 ** -100, -8, 448.0, 2.0 ** 90, 64)]


@pytest.mark.parametrize("R,N", FORMS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size,q,gs,cs,columns", CASES)
def test_rows_near_the_ends_of_the_range(size, q, gs, cs, columns, group, R, N):
    D = 256
    x = torch.zeros((R, D), dtype=BF, device="cuda")
    x[:, 128 - columns:128] = size
    out = product(x, torch.full((N, D), q, dtype=I8, device="cuda"), torch.full((N, D // group), gs, device="cuda"),
                  torch.full((N,), cs, device="cuda"), group)
    want = torch.tensor(size * q * gs * cs * columns, dtype=F64).to(BF).item()
    assert want == size * q * gs * cs * columns  # a BF16 number
    assert (out == want).all(), (out.flatten()[0].item(), want)


@pytest.mark.parametrize("R,N", FORMS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gates_whose_silu_only_a_large_up_brings_into_range(sign, R, N):
    gates = torch.tensor([-100.0, -150.0, -170.0, -174.0, -175.0, -176.0, -178.0, -180.0], device="cuda").repeat(N // 8)
    q = torch.zeros((2 * N, 128), dtype=I8, device="cuda")
    q[:N, 0], q[N:, 1] = 1, 1
    x = torch.zeros((R, 128), dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = 1.0, sign * 2.0 ** 100
    out = product(x, q, torch.ones((2 * N, 1), device="cuda"), torch.cat([gates, torch.full((N,), 2.0 ** 27, device="cuda")]), 128,
                  gated=True)
    z = gates.to(F64)
    want = z / (1 + torch.exp(-z)) * (sign * 2.0 ** 127)
    assert (want.abs() > 2.0 ** -126).all()
    assert ((out.to(F64) - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs()).all(), (out[0, :8], want[:8])
