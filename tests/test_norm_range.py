"""Residual, norm and 8-bit rows where a square, a sum of squares or a product with a gain leaves FP32's range although
the result does not, against the definition in 64 bits.

Tolerances: an FP32 sum of squares by threads and warps (under 100 additions in a row), root, division and products,
under 100 * 2^-24 = 6e-6 of the value; 1e-5 is asked of scales, half a step and twice that of values.
"""
import pytest
import torch

import moe_decode_tail_gb300 as mt

pytestmark = pytest.mark.gpu

BF, I8, F32, F64, E4 = torch.bfloat16, torch.int8, torch.float32, torch.float64, torch.float8_e4m3fn
MOST = {I8: 127.0, E4: 448.0}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").clamp(-3.0, 3.0)


def quantised(x, residual, gamma, dtype, group, **more):
    b, H = x.shape
    q = torch.full((b, H), 77.0, device="cuda").to(dtype)
    scale = torch.full((b, -(-H // 128)) if group else (b,), 77.0, device="cuda")
    out, y = torch.empty_like(x), torch.empty_like(x)
    mt.moe_tail_norm_quant(x, residual, gamma, q, scale, residual_out=out, y=y, group=group, **more)
    return q, scale, out, y


def check(got, x, residual, gamma, group, gain_center, eps):
    q, scale, out, y = got
    h = x.to(F64) + (0.0 if residual is None else residual.to(F64))
    v = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * (gamma.to(F64) + gain_center)
    assert ((out.to(F64) - h).abs() <= h.abs() * 2.0 ** -8 + 1e-40).all()
    assert ((y.to(F64) - v).abs() <= v.abs() * (2.0 ** -8 + 1e-5) + 1e-40).all()
    size = group or x.shape[1]
    for g in range(-(-x.shape[1] // size)):
        part, values = v[:, g * size:(g + 1) * size], q[:, g * size:(g + 1) * size].to(F32).to(F64)
        sc = (scale[:, g] if group else scale).to(F64)
        want = part.abs().amax(1) / MOST[q.dtype]
        assert ((sc - want).abs() <= 1e-5 * want + 1e-44).all(), (sc, want)
        ratio = torch.where(want[:, None] > 0, part / want.clamp_min(1e-300)[:, None], 0.0)
        if q.dtype == I8:
            half = torch.full_like(ratio, 0.5)
        else:
            half = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp_min(1e-30))).clamp_min(-6.0) - 4)
        off = (values - ratio).abs()
        assert (off <= half * (1 + 1e-5) + 2e-5 * ratio.abs() + 1e-9).all(), (off - half).max()


SIZES = [8, 136, 4096, 16384, 32768]


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("H", SIZES)
def test_rows_whose_squares_overflow(H, group, dtype):
    g = gen(H)
    b = 400
    gamma = (normal(g, H) * 0.1).to(BF)
    for size in (1e17, 1e19, 1e25, 1e30, 5e37):
        x, residual = normal(g, b, H), normal(g, b, H)
        x[::3] *= size          # every third row; the others are ordinary
        residual[::3] *= size
        x[1], residual[1] = 0, 0
        x, residual = x.to(BF), residual.to(BF)
        for rows in (b, 3):     # many rows and a few
            got = quantised(x[:rows], residual[:rows], gamma, dtype, group, gain_center=1.0, eps=1e-6)
            check(got, x[:rows], residual[:rows], gamma, group, 1.0, 1e-6)
    # one huge value in a row of ordinary ones
    x = normal(g, 4, H).to(BF)
    x[2, H // 2] = 3e38
    check(quantised(x, None, gamma, dtype, group, gain_center=1.0, eps=1e-6), x, None, gamma, group, 1.0, 1e-6)


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("H", SIZES)
def test_rows_whose_squares_vanish(H, group, dtype):
    g = gen(H + 1)
    gamma = (normal(g, H) * 0.1).to(BF)
    for size in (1e-17, 1e-19, 1e-23, 1e-30):
        for eps in (0.0, size * size, 1e-38):
            x = (normal(g, 5, H) * size).to(BF)
            x[3] = normal(g, H).to(BF)
            check(quantised(x, None, gamma, dtype, group, gain_center=1.0, eps=eps), x, None, gamma, group, 1.0,
                  float(torch.tensor(eps, dtype=F32)))


def test_rows_without_a_norm():
    # what has no finite norm is NaN: an infinity or a NaN in the row, an infinite sum, 0 / 0
    H = 256
    gamma = torch.zeros(H, dtype=BF, device="cuda")
    x, residual = torch.ones((4, H), dtype=BF, device="cuda"), torch.ones((4, H), dtype=BF, device="cuda")
    x[0, 3], x[1, 4] = float("inf"), float("nan")
    x[2, 5], residual[2, 5] = 3e38, 3e38
    for group in (0, 128):
        _, scale, _, _ = quantised(x, residual, gamma, I8, group)
        s = scale.view(4, -1)
        assert s[:3, 0].isnan().all() and s[3].isfinite().all()
    _, scale, _, _ = quantised(torch.zeros_like(x), None, gamma, I8, 0, eps=0.0)
    assert scale.isnan().all()


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("H", SIZES)
@pytest.mark.parametrize("size,gain,eps", [(1e18, 1e25, 1e-6), (1e3, 1e36, 1e-6), (1e30, 1e20, 1e-6), (1e-14, 1e-28, 1e-38),
                                           (1e-3, 1e-34, 1e-9), (1.0, 1e-34, 1e-6), (1e-14, 1e30, 1e-38)])
def test_products_with_gains_that_leave_the_range(size, gain, eps, H, group, dtype):
    g = gen(H + 2)
    x = (normal(g, 5, H) * size).to(BF)
    x[2] = normal(g, H).to(BF)
    gamma = (normal(g, H) * gain).to(BF)
    check(quantised(x, None, gamma, dtype, group, gain_center=0.0, eps=eps), x, None, gamma, group, 0.0,
          float(torch.tensor(eps, dtype=F32)))


@pytest.mark.parametrize("dtype", [I8, E4])
def test_a_row_and_its_only_group_agree(dtype):
    # up to 128 columns a group is the row: whatever rounds on the way, both forms round the same values
    g = gen(3)
    H = 128
    x, gamma = torch.full((3, H), 2.0 ** -87, device="cuda"), torch.full((H,), 2.0 ** 120, device="cuda")
    x *= 1 + torch.rand((3, H), generator=g, device="cuda")
    x[:, 0], gamma[0] = 2.0 ** 60, 0.0
    x[1] *= 2.0 ** -40
    x[2] *= 2.0 ** 40
    x, gamma = x.to(BF), gamma.to(BF)
    a = quantised(x, None, gamma, dtype, 0, gain_center=0.0, eps=1e-6)
    b = quantised(x, None, gamma, dtype, 128, gain_center=0.0, eps=1e-6)
    assert torch.equal(a[0].view(I8), b[0].view(I8)) and torch.equal(a[1], b[1][:, 0]) and torch.equal(a[3], b[3])
