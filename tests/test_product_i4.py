"""The 4-bit products on a GPU, against plain implementations in 64 bits.

Tolerances, from the formulas: half a unit in the last place of the BF16 result (2^-8 of its binade's lower end), and the
FP32 sum's error before it.  Every term x * (gs * q) is exact, so that error is at most one rounding or truncation (2^-23)
of the sum of magnitudes for each of the D additions, the groups' and the splits'.  Where all terms are small whole
numbers the sum is exact, and so is the result up to its rounding.
silu(g) * u with g and u off by dg and du: at most 1.1 |u| dg + |silu(g)| du + 1.1 dg du, and 2^-19 of itself for the
exponential (2 units), the division (2) and four products.
"""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300.expert_layer import pack_int4, quantise_groups

pytestmark = pytest.mark.gpu

BF, I8, I32, F32, F64, E4 = torch.bfloat16, torch.int8, torch.int32, torch.float32, torch.float64, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


class Weight:
    """A 4-bit weight [E, channels, D] and the numbers it stands for; what the layout leaves open is filled with the worst."""

    def __init__(self, g, E, channels, D, group, exact=False):
        self.q = torch.randint(-8, 8, (E, channels, D), generator=g, device="cuda").to(I8)
        groups = -(-D // group)
        if exact:  # powers of two
            gs = torch.exp2(torch.randint(-2, 3, (E, channels, groups), generator=g, device="cuda").float())
            self.cs = torch.exp2(torch.randint(-3, 3, (E, channels), generator=g, device="cuda").float())
        else:
            gs = torch.rand((E, channels, groups), generator=g, device="cuda") * 400 + 1
            self.cs = torch.rand((E, channels), generator=g, device="cuda") * 1e-4
        full = torch.full((E, channels, -(-groups // 4) * 4), float("nan"), device="cuda")
        full[:, :, :groups] = gs
        self.gs, self.group, self.D = full.to(E4), group, D
        pad = torch.randint(-8, 8, (E, channels, -D % 128), generator=g, device="cuda").to(I8)
        self.w = pack_int4(torch.cat([self.q, pad], -1))

    def value(self, e):  # FP64 [channels, D], without the channels' scales
        gs = self.gs[e].to(F32).to(F64).repeat_interleave(self.group, 1)[:, :self.D]
        return self.q[e].to(F64) * gs


def expected(x, weight, offsets, gated):
    """(FP64 result, its bound before the rounding, rows with an expert)."""
    E, channels, D = weight.q.shape
    R = x.shape[0]
    N = channels // 2 if gated else channels
    want, slack = torch.zeros((R, N), dtype=F64, device="cuda"), torch.zeros((R, N), dtype=F64, device="cuda")
    live = torch.zeros(R, dtype=torch.bool, device="cuda")
    ends = [0, R] if offsets is None else offsets.tolist()
    for e in range(E):
        i, j = ends[e], ends[e + 1]
        if j <= i:
            continue
        w, cs = weight.value(e), weight.cs[e].to(F64)
        p = (x[i:j].to(F64) @ w.T) * cs
        size = (x[i:j].to(F64).abs() @ w.abs().T) * cs.abs()
        dp = (D + 256) * 2.0 ** -23 * size
        if gated:
            g, u, dg, du = p[:, :N], p[:, N:], dp[:, :N], dp[:, N:]
            s = g * torch.sigmoid(g)
            want[i:j] = s * u
            slack[i:j] = 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + 2.0 ** -19 * (s * u).abs()
        else:
            want[i:j], slack[i:j] = p, dp + 2.0 ** -23 * p.abs()
        live[i:j] = True
    return want, slack, live


def call(x, weight, offsets, gated, out=None):
    channels = weight.q.shape[1]
    if out is None:
        out = torch.full((x.shape[0], channels // 2 if gated else channels), 77.0, dtype=BF, device="cuda")
    fn = mt.moe_tail_gated_product_i4 if gated else mt.moe_tail_expert_product_i4
    assert fn(x, weight.w, weight.gs, weight.cs, out, group=weight.group, expert_offsets=offsets) is out
    return out


def check(out, x, weight, offsets, gated):
    want, slack, live = expected(x, weight, offsets, gated)
    off = (out.to(F64) - want).abs()
    bound = want.abs() * 2.0 ** -8 * (1 + 2.0 ** -10) + slack + 1e-40
    assert (off <= bound)[live].all(), (off - bound)[live].max()
    assert (out[~live] == 77).all()  # rows of no expert are not written
    assert not (out.view(torch.int16) == -32768).any()


def offsets_of(counts):
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.as_tensor(counts).cumsum(0)]).to(I32).cuda()


SIZES = [(8, 8), (16, 24), (128, 128), (136, 40), (72, 200), (256, 512), (1032, 136), (2056, 264), (3584, 1024), (4096, 72)]  # D, N


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("D,N", SIZES)
def test_dense(D, N, group, gated):
    g = gen(D + N + group)
    for exact in (True, False):
        weight = Weight(g, 1, 2 * N if gated else N, D, group, exact)
        for R in (1, 2, 8, 9, 16, 17, 33, 64, 65, 130):
            x = torch.randint(-3, 4, (R, D), generator=g, device="cuda").to(BF) if exact else normal(g, R, D)
            out = call(x, weight, None, gated)
            check(out, x, weight, None, gated)
            if exact and not gated:
                want, _, _ = expected(x, weight, None, False)
                assert torch.equal(out, want.to(F32).to(BF) + 0.0)  # the sums are exact in FP32
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["few", "uneven", "one", "none", "many"])
@pytest.mark.parametrize("E,D,N,group", [(1, 256, 64, 128), (5, 392, 136, 32), (60, 520, 72, 64), (128, 128, 256, 128), (1024, 64, 16, 32)])
def test_by_expert(E, D, N, group, kind, gated):
    g = gen(E + D)
    torch.manual_seed(E)
    weight = Weight(g, E, 2 * N if gated else N, D, group)
    counts = torch.zeros(E, dtype=torch.long)
    if kind == "few":
        counts = torch.randint(0, 4, (E,))
    elif kind == "uneven":
        counts = torch.arange(E) * 7 % 41
    elif kind == "one":
        counts[E // 2] = 333
    elif kind == "many":
        counts = torch.randint(0, 2 + 3000 // E, (E,)) + (torch.arange(E) == 1) * 300
    offsets = offsets_of(counts)
    R = int(offsets[-1]) + 5  # rows of no expert at the end
    x = normal(g, R, D)
    x[-5:] = float("nan")
    out = call(x, weight, offsets, gated)
    check(out, x, weight, offsets, gated)
    again = call(x, weight, offsets, gated)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,E,D,N", [(1, 1, 7168, 4096), (512, 128, 2048, 1024), (2048, 64, 1544, 520), (3000, 8, 1024, 776),
                                     (400, 1, 4104, 2056), (1, 1, 65536, 24)])
def test_weights_that_stream(R, E, D, N, gated):
    # many tiles for every thread block, the reduction longer than the rings, several calls in flight
    g = gen(R + E)
    weight = Weight(g, E, 2 * N if gated else N, D, 128)
    ids = (torch.rand((R, E), generator=g, device="cuda") * torch.linspace(1.0, 3.0, E, device="cuda")).argmax(1)
    offsets = offsets_of(torch.bincount(ids, minlength=E).cpu()) if E > 1 else None
    x = normal(g, R, D)
    out = call(x, weight, offsets, gated)
    again = [call(x, weight, offsets, gated) for _ in range(6)]
    check(out, x, weight, offsets, gated)
    assert all(torch.equal(o, out) for o in again)
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,E,D,N,group", [(3000, 8, 1024, 1288, 128), (5000, 2, 392, 2056, 64), (2600, 1, 2056, 2568, 32),
                                           (9000, 60, 264, 1416, 32), (4100, 3, 640, 1800, 64), (6000, 4, 72, 2568, 32)])
def test_many_rows(R, E, D, N, group, gated):
    # enough tiles for the wide ones, experts with one row tile and with many
    g = gen(R)
    weight = Weight(g, E, 2 * N if gated else N, D, group)
    ids = (torch.rand((R, E), generator=g, device="cuda") * torch.linspace(1.0, 4.0, E, device="cuda")).argmax(1)
    offsets = offsets_of(torch.bincount(ids, minlength=E).cpu()) if E > 1 else None
    x = normal(g, R, D)
    out = call(x, weight, offsets, gated)
    again = [call(x, weight, offsets, gated) for _ in range(4)]
    check(out, x, weight, offsets, gated)
    assert all(torch.equal(o, out) for o in again)
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("gated", [False, True])
def test_values_that_are_not_finite_stay_in_their_rows_and_channels(gated):
    g = gen(2)
    N, D = 96, 520
    for R in (5, 40, 200):
        weight = Weight(g, 1, 2 * N if gated else N, D, 32)
        weight.gs[0, 3, 2] = float("nan")
        weight.cs[0, 10] = float("nan")
        x = normal(g, R, D)
        x[1, 519], x[3, 0] = float("nan"), float("inf")
        out = call(x, weight, None, gated)
        assert out[1].isnan().all() and not out[3].isfinite().any()
        assert out[:, 3].isnan().all() and out[:, 10].isnan().all()
        rows = torch.ones(R, dtype=torch.bool, device="cuda")
        rows[1], rows[3] = False, False
        columns = torch.ones(N, dtype=torch.bool, device="cuda")
        columns[3], columns[10] = False, False
        assert out[rows][:, columns].isfinite().all()


def test_gates_at_both_ends_of_the_exponential():
    # one column: g and u are x times chosen weights, up to where exp(-g) leaves FP32's range
    N, D = 8, 128
    gates = torch.tensor([0.0, 1.0, -1.0, 80.0, -80.0, 87.0, -87.5, -100.0], device="cuda")
    q = torch.zeros((1, 2 * N, D), dtype=I8, device="cuda")
    q[0, :, 0] = 1
    cs = torch.cat([gates, torch.full((N,), 2.0 ** 60, device="cuda")])[None]
    gs = torch.ones((1, 2 * N, 4), device="cuda").to(E4)
    for R in (1, 80):
        x = torch.zeros((R, D), dtype=BF, device="cuda")
        x[:, 0] = 1
        out = torch.empty((R, N), dtype=BF, device="cuda")
        mt.moe_tail_gated_product_i4(x, pack_int4(q), gs, cs, out, group=128)
        want = gates.to(F64) * torch.sigmoid(gates.to(F64)) * 2.0 ** 60
        assert ((out.to(F64) - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs()).all(), out[0]


def test_offsets_that_are_no_partition():
    # whatever the offsets hold, no row outside [0, R) is touched
    g = gen(4)
    E, N, D = 3, 136, 128
    weight = Weight(g, E, N, D, 64)
    for R in (20, 300):
        x = normal(g, R, D)
        for bad in ([0, 5, 5, 10 ** 6], [-7, 3, 2, 9], [12, 4, 30, 1], [2 ** 31 - 1, -2 ** 31, 0, 20]):
            big = torch.full((R + 64, N), 77.0, dtype=BF, device="cuda")
            call(x, weight, torch.tensor(bad, dtype=I32, device="cuda"), False, big[32:32 + R])
            torch.cuda.synchronize()
            assert (big[:32] == 77).all() and (big[32 + R:] == 77).all()
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,E", [(3, 1), (60, 4), (2000, 4)])
def test_waits_that_run_out(R, E, gated):
    # a limit of one nanosecond on the operands: the call gives up, says so and leaves the device usable
    g = gen(8)
    N, D = 264, 1032
    weight = Weight(g, E, 2 * N if gated else N, D, 128)
    x, offsets = normal(g, R, D), offsets_of([R // E] * E) if E > 1 else None
    assert mt.moe_tail_take_device_error() == 0
    mt.moe_tail_set_stage_wait_limit(1)
    try:
        call(x, weight, offsets, gated)
        torch.cuda.synchronize()
    finally:
        mt.moe_tail_set_stage_wait_limit(0)
    assert mt.moe_tail_take_device_error() & 1
    check(call(x, weight, offsets, gated), x, weight, offsets, gated)
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("gated", [False, True])
def test_on_a_side_stream_and_in_a_graph(gated):
    g = gen(9)
    E, N, D, R = 6, 200, 648, 50
    weight = Weight(g, E, 2 * N if gated else N, D, 32)
    x, offsets = normal(g, R, D), offsets_of([9, 0, 20, 1, 3, 17])
    want, out = call(x, weight, offsets, gated), torch.empty((R, N), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x, weight, offsets, gated, out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, weight, offsets, gated, out)
    first = x.clone()
    x.copy_(normal(g, R, D))
    offsets.copy_(offsets_of([0, 30, 1, 1, 10, 8]))
    graph.replay()
    other = out.clone()
    assert torch.equal(call(x, weight, offsets, gated), other) and not torch.equal(other, want)
    x.copy_(first)
    offsets.copy_(offsets_of([9, 0, 20, 1, 3, 17]))
    graph.replay()
    assert torch.equal(out, want)
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantised_weights(group):
    # what quantise_groups makes stands for the weights to half a step of each group, and the product takes it
    g = gen(group)
    E, N, D, R = 2, 72, 328, 7
    w = normal(g, E, N, D, dtype=F32) * torch.exp(normal(g, E, N, 1, dtype=F32))
    w[0, 5] = 0
    packed, gs, cs = quantise_groups(w, group)
    groups = -(-D // group)
    step = (gs[:, :, :groups].float() * cs[:, :, None]).repeat_interleave(group, 2)[:, :, :D]
    values = torch.zeros_like(w)
    for k in range(D):  # the columns that the product reads, one at a time
        x = torch.zeros((1, D), dtype=BF, device="cuda")
        x[0, k] = 1
        for e in range(E):
            out = torch.empty((1, N), dtype=BF, device="cuda")
            mt.moe_tail_expert_product_i4(x, packed[e:e + 1], gs[e:e + 1], cs[e:e + 1], out, group=group)
            values[e, :, k] = out[0].float()
    # half a step; a group scale rounded down by at most 2^-4 leaves 7 short of the largest value by 7 / 16 of a step; the
    # result's own rounding, half a unit: 2^-8 of the value it rounds, which is itself up to half a step larger than the weight
    assert ((values - w).abs() <= 0.5 * step + 2.0 ** -8 * (w.abs() + 0.5 * step) + 1e-6 * step).all()
    assert (values[0, 5] == 0).all()


def test_large_rows():
    # results past 2^31 elements
    g = gen(12)
    N, D, R = 16384, 16, 140000
    weight = Weight(g, 1, N, D, 32)
    x = torch.zeros((R, D), dtype=BF, device="cuda")
    x[-3:], x[0] = normal(g, 3, D), normal(g, D)
    out = torch.empty((R, N), dtype=BF, device="cuda")
    call(x, weight, None, False, out)
    for rows in (slice(0, 2), slice(R - 3, R)):
        check(out[rows], x[rows], weight, None, False)
    assert not out[1:R - 3].any()


def test_calls_at_once_on_several_streams():
    # every kind of tile on streams of their own, whose kernels share the SMs and their tensor memory
    g = gen(13)
    calls = []
    for R, E, D, N, gated in ((1, 1, 2048, 264, True), (512, 64, 1024, 520, False), (300, 4, 1032, 776, True), (6000, 8, 392, 2056, False)):
        weight = Weight(g, E, 2 * N if gated else N, D, 64)
        counts = [R // E] * E
        calls.append((normal(g, R, D), weight, offsets_of(counts) if E > 1 else None, gated))
    wants = [call(*c) for c in calls]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in wants]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for i in range(20):
        for c, out, stream in zip(calls, outs, streams):
            with torch.cuda.stream(stream):
                call(*c, out[i])
    torch.cuda.synchronize()
    for c, out, want in zip(calls, outs, wants):
        assert all(torch.equal(o, want) for o in out)
        check(want, *c)
    assert mt.moe_tail_take_device_error() == 0
