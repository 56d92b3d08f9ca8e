"""The 4-bit products' wide tiles (128 rows by 256 stored channels, converters and an epilogue of their own) where the other
tests take smaller ones: waits that run out, values that are not finite, offsets that are no partition, streams and graphs.
Every test asks first that its sizes take wide tiles; the first ones ask that the sizes of the others' tests take theirs."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300 import build as cuda_build
from test_product_i4 import BF, I32, Weight, call, check, gen, normal, offsets_of


@pytest.fixture(scope="module", autouse=True)
def built():
    cuda_build.build()


def tile_rows(R, E, N, D, gated):
    return mt.moe_tail_product_i4_tile_rows(R, E, N, D, gated=gated)


@pytest.mark.parametrize("sizes,rows", [
    ((1, 1, 1024, 4096, False), 8), ((8, 1, 1024, 3584, True), 8), ((9, 1, 128, 128, False), 16), ((17, 1, 128, 128, False), 32),
    ((64, 1, 128, 128, True), 64), ((512, 128, 1024, 4096, True), 16), ((1, 1, 40000, 64, False), 16), ((3, 1, 264, 1032, True), 8),
    ((60, 4, 264, 1032, False), 32), ((2000, 4, 264, 1032, False), 64), ((2000, 4, 264, 1032, True), 64),
    ((3000, 8, 1288, 1024, False), 128), ((5000, 2, 2056, 392, True), 128), ((6000, 8, 2056, 392, False), 128),
    ((32768, 128, 4096, 2048, False), 128), ((0, 4, 8, 8, False), 8)])
def test_what_sizes_take(sizes, rows):
    assert tile_rows(*sizes) == rows  # on 152 SMs


@pytest.mark.parametrize("sizes", [(-1, 1, 8, 8), (8, 0, 8, 8), (8, 1025, 8, 8), (8, 1, 12, 8), (8, 1, 8, 12), (8, 1, 8, 1 << 17),
                                   ((1 << 22) + 1, 1, 8, 8), (8, 1, (1 << 20) + 8, 8)])
def test_sizes_that_the_products_refuse_take_nothing(sizes):
    assert tile_rows(*sizes, False) == tile_rows(*sizes, True) == 0


def wide(R, E, N, D, gated):
    assert tile_rows(R, E, N, D, gated) == 128


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,E,D,N", [(2600, 1, 1032, 2568), (3200, 4, 648, 1800), (3000, 8, 72, 1288), (2560, 1, 8192, 2560)])
def test_waits_that_run_out(R, E, D, N, gated):
    g = gen(8)
    wide(R, E, N, D, gated)
    weight = Weight(g, E, 2 * N if gated else N, D, 64)
    x, offsets = normal(g, R, D), offsets_of([R // E] * E) if E > 1 else None
    assert mt.moe_tail_take_device_error() == 0
    for limit in (1, 200, 1000):  # nanoseconds: 1 gives up in any case
        mt.moe_tail_set_stage_wait_limit(limit)
        try:
            call(x, weight, offsets, gated)
            torch.cuda.synchronize()
        finally:
            mt.moe_tail_set_stage_wait_limit(0)
        bits = mt.moe_tail_take_device_error()
        assert bits & 1 or limit > 1
        check(call(x, weight, offsets, gated), x, weight, offsets, gated)
        assert mt.moe_tail_take_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("D", [520, 392, 640])  # an odd last block, a part of one, whole ones
def test_values_that_are_not_finite_stay_in_their_rows_and_channels(D, gated):
    g = gen(2)
    R, N = 2700, 2568
    wide(R, 1, N, D, gated)
    weight = Weight(g, 1, 2 * N if gated else N, D, 32)
    bad = [0, 3, 127, 128, 255, 256, 2567]
    for n in bad[::2]:
        weight.gs[0, n, (D - 1) // 32] = float("nan")
    for n in bad[1::2]:
        weight.cs[0, n] = float("nan")
    x = normal(g, R, D)
    not_finite = [1, 63, 64, 129, 2688, 2699]
    x[not_finite[::2], D - 1], x[not_finite[1::2], 0] = float("nan"), float("inf")
    out = call(x, weight, None, gated)
    assert not out[not_finite].isfinite().any() and out[not_finite[::2]].isnan().all() and out[:, bad].isnan().all()
    rows, columns = torch.ones(R, dtype=torch.bool, device="cuda"), torch.ones(N, dtype=torch.bool, device="cuda")
    rows[not_finite], columns[bad] = False, False
    assert out[rows][:, columns].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
def test_offsets_that_are_no_partition(gated):
    # whatever the offsets hold, no row outside [0, R) is touched
    g = gen(4)
    E, N, D, R = 3, 2568, 136, 2000
    wide(R, E, N, D, gated)
    weight = Weight(g, E, 2 * N if gated else N, D, 64)
    x = normal(g, R, D)
    for offsets in ([0, 5, 5, 10 ** 6], [-7, 300, 200, 900], [1200, 4, 1990, 1], [2 ** 31 - 1, -2 ** 31, 0, 2000], [5, 5, 5, 5]):
        big = torch.full((R + 256, N), 77.0, dtype=BF, device="cuda")
        call(x, weight, torch.tensor(offsets, dtype=I32, device="cuda"), gated, big[128:128 + R])
        torch.cuda.synchronize()
        assert (big[:128] == 77).all() and (big[128 + R:] == 77).all()
    assert (big == 77).all()  # no expert has a row
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
def test_few_and_no_rows_of_a_large_buffer(gated):
    # sizes that take wide tiles, of which the routes fill little
    g = gen(5)
    E, N, D, R = 8, 1288, 520, 3000
    wide(R, E, N, D, gated)
    weight = Weight(g, E, 2 * N if gated else N, D, 128)
    x = normal(g, R, D)
    for counts in ([0] * 8, [1, 0, 0, 0, 0, 0, 0, 0], [0, 3, 0, 15, 16, 17, 0, 1], [0, 0, 0, 0, 0, 0, 0, 129], [128, 127, 129, 1, 1, 1, 1, 1]):
        offsets = offsets_of(counts)
        used = int(offsets[-1])
        out = call(x, weight, offsets, gated)
        check(out, x, weight, offsets, gated)
        assert (out[used:] == 77).all()
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [False, True])
def test_on_a_side_stream_and_in_a_graph(gated):
    g = gen(9)
    E, N, D, R = 6, 1800, 648, 2400
    wide(R, E, N, D, gated)
    weight = Weight(g, E, 2 * N if gated else N, D, 32)
    first_counts, other_counts = [900, 0, 20, 1000, 3, 477], [0, 1300, 1, 1, 1000, 8]
    x, offsets = normal(g, R, D), offsets_of(first_counts)
    want, out = call(x, weight, offsets, gated), torch.full((R, N), 77.0, dtype=BF, device="cuda")
    check(want, x, weight, offsets, gated)
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
    offsets.copy_(offsets_of(other_counts))
    out.fill_(77.0)
    graph.replay()
    check(out, x, weight, offsets, gated)
    x.copy_(first)
    offsets.copy_(offsets_of(first_counts))
    for _ in range(3):
        out.fill_(77.0)
        graph.replay()
        assert torch.equal(out, want)
    assert mt.moe_tail_take_device_error() == 0
