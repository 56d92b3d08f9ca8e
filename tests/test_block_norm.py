"""The norms around a block and their gradients on a GPU, against plain implementations in 64 bits.

Tolerances, from the formulas: half a unit in the last place of a BF16 result (2^-8 of its binade's lower end), and before it
the FP32 arithmetic: a sum of H squares by threads and warps (under 100 additions in a row), root, division and products are
off by under 100 * 2^-24 = 6e-6 of the value, and the terms of a sum by that much of their own size.  So a result is
allowed 4e-5 (the gradients: rstd enters up to three times, and two reductions) or 2e-5 (forward) of its formula taken over
magnitudes; sums over b rows 2^-24 more for each row in a thread block's turn, under b * 2^-24.
"""
import pytest
import torch

import moe_decode_tail_gb300 as mt

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
WIDTHS = [8, 24, 120, 248, 256, 264, 512, 1000, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 16384, 18432, 32760, 32768]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def inputs(g, b, H, post, token, channel):
    return dict(x=normal(g, b, H, std=0.7), residual=normal(g, b, H, std=2.0),
                post_gamma=normal(g, H, std=0.2) if post else None, pre_gamma=normal(g, H, std=0.2),
                token_gate=torch.rand(b, generator=g, device="cuda") * 2 - 0.5 if token else None,
                channel_gate=normal(g, H, std=0.3, mean=0.5) if channel else None)


def to64(d):
    return {k: None if v is None else v.to(F64) for k, v in d.items()}


def plain(d, scale=1.0, center=1.0, eps=1e-6):
    """FP64 (h, y, rstd0, rstd1, magnitudes of h's terms)."""
    d = to64(d)
    n = d["x"]
    rstd0 = torch.ones(n.shape[0], dtype=F64, device="cuda")
    if d["post_gamma"] is not None:
        rstd0 = ((n * n).mean(1) + eps) ** -0.5
        n = n * rstd0[:, None] * (d["post_gamma"] + center)
    for gate, shape in (("token_gate", (-1, 1)), ("channel_gate", (1, -1))):
        if d[gate] is not None:
            n = n * d[gate].view(shape)
    h = scale * d["residual"] + n
    rstd1 = ((h * h).mean(1) + eps) ** -0.5
    return h, h * rstd1[:, None] * (d["pre_gamma"] + center), rstd0, rstd1, (scale * d["residual"]).abs() + n.abs()


def close(got, want, size, rel):
    assert got.shape == want.shape
    off = (got.to(F64) - want).abs()
    bound = rel * size + 1e-40
    if got.dtype == BF:
        bound = bound + want.abs() * 2.0 ** -8 * (1 + 2.0 ** -10)
        assert not (got.view(torch.int16) == -32768).any()  # -0 is written as +0
    bad = ~(off <= bound)
    assert not bad.any(), (int(bad.sum()), off[bad].max().item(), want[bad][:4])


def forward(d, **more):
    b, H = d["x"].shape
    out, y = (torch.full((b, H), 77.0, dtype=BF, device="cuda") for _ in range(2))
    rstd = torch.full((b, 2), 77.0, device="cuda")
    gates = {k: d[k] for k in ("token_gate", "channel_gate")}
    mt.moe_tail_block_norm(d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], out, y, rstd=rstd, **gates, **more)
    return out, y, rstd


def check_forward(d, got, **more):
    out, y, rstd = got
    h, want, rstd0, rstd1, size = plain(d, **{{"residual_scale": "scale", "gain_center": "center"}.get(k, k): v for k, v in more.items()})
    close(out, h, size, 2e-5)
    gain = (d["pre_gamma"].to(F64) + more.get("gain_center", 1.0)).abs()
    close(y, want, size * rstd1[:, None] * gain, 4e-5)
    close(rstd, torch.stack([rstd0, rstd1], 1), torch.stack([rstd0, rstd1 * (1 + size.square().mean(1).sqrt() * rstd1)], 1), 2e-5)


FORMS = [(True, True, True), (True, False, False), (False, True, False), (False, False, True), (True, True, False)]


@pytest.mark.parametrize("post,token,channel", FORMS)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward(H, post, token, channel):
    g = gen(H)
    for b in (1, 5, 333):
        d = inputs(g, b, H, post, token, channel)
        if b == 5:
            d["x"][1], d["residual"][1] = 0, 0          # a row of zeros
            d["residual"][2] = 0                        # only the block's
            d["x"][3] = 0                               # only the residual
            d["x"][4] *= 1e15
        for more in (dict(), dict(residual_scale=0.25, gain_center=0.0, eps=1e-5)):
            got = forward(d, **more)
            check_forward(d, got, **more)
        x2, r2, y = d["x"].clone(), d["residual"].clone(), torch.empty_like(d["x"])
        gates = {k: d[k] for k in ("token_gate", "channel_gate")}
        for place in (x2, r2):  # in place, without rstd
            mt.moe_tail_block_norm(x2 if place is x2 else d["x"], r2 if place is r2 else d["residual"], d["post_gamma"],
                                   d["pre_gamma"], place, y, **gates, **more)
            assert torch.equal(place, got[0]) and torch.equal(y, got[1])


@pytest.mark.parametrize("size", [1e-30, 1e-19, 1e19, 1e30, 2.0 ** 125])
@pytest.mark.parametrize("post", [True, False])
def test_rows_whose_squares_leave_the_range(size, post):
    # brought near one by a power of two: the norm is that of the row, whatever its size
    H = 520
    g = gen(3)
    d = inputs(g, 4, H, post, False, False)
    d["x"], d["residual"] = (d["x"].float() * size).to(BF), torch.zeros_like(d["residual"])
    out, y, rstd = forward(d, eps=0.0)
    h, want, rstd0, rstd1, scale = plain(d, eps=0.0)
    close(out, h, scale, 2e-5)
    close(y, want, want.abs(), 6e-5)
    d["residual"], d["x"] = (normal(g, 4, H).float() * size).to(BF), torch.zeros_like(d["x"])
    d["post_gamma"] = None
    out, y, _ = forward(d, eps=0.0)
    h, want, _, _, scale = plain(d, eps=0.0)
    close(y, want, want.abs(), 6e-5)


def test_rows_that_are_not_finite_stay_alone():
    H = 1000
    g = gen(4)
    d = inputs(g, 6, H, True, True, True)
    d["x"][1, 500], d["residual"][2, 3], d["x"][3, 0] = float("nan"), float("inf"), float("inf")
    out, y, rstd = forward(d)
    assert y[1].isnan().all() and not y[2, 3].isfinite() and not y[3, 0].isfinite()
    good = torch.tensor([0, 4, 5], device="cuda")
    check_forward({k: v if v is None or v.shape[0] != 6 else v[good] for k, v in d.items()}, (out[good], y[good], rstd[good]))


# ---- gradients ---------------------------------------------------------------------------------------------------------


def plain_grad(d, d_y, d_out, scale=1.0, center=1.0, eps=1e-6, magnitudes=False):
    """FP64 gradients by the formulas; with `magnitudes` the same over absolute values, every difference a sum."""
    h, _, rstd0, rstd1, size = plain(d, scale, center, eps)
    d = to64(d)
    a = (lambda t: t.abs()) if magnitudes else (lambda t: t)
    sign = 1.0 if magnitudes else -1.0
    if magnitudes:
        h, scale = size, abs(scale)
    H = h.shape[1]
    gain = a(d["pre_gamma"] + center)
    token = a(d["token_gate"])[:, None] if d["token_gate"] is not None else 1.0
    channel = a(d["channel_gate"])[None] if d["channel_gate"] is not None else 1.0
    u = a(d["x"]) * rstd0[:, None]
    post = a(d["post_gamma"] + center) if d["post_gamma"] is not None else 1.0
    n = u * post
    v = h * rstd1[:, None]
    d_y, d_out = a(d_y.to(F64)), 0.0 if d_out is None else a(d_out.to(F64))
    d_v = d_y * gain
    d_h = d_out + rstd1[:, None] * (d_v + sign * v * (d_v * v).sum(1, keepdim=True) / H)
    d_n = d_h * token * channel
    out = {"d_residual": scale * d_h, "d_pre_gamma": (d_y * v).sum(0)}
    if d["post_gamma"] is not None:
        d_u = d_n * post
        out["d_x"] = rstd0[:, None] * (d_u + sign * u * (d_u * u).sum(1, keepdim=True) / H)
        out["d_post_gamma"] = (d_n * u).sum(0)
    else:
        out["d_x"] = d_n
    if d["token_gate"] is not None:
        out["d_token_gate"] = (d_h * n * channel).sum(1)
    if d["channel_gate"] is not None:
        out["d_channel_gate"] = (d_h * n * token).sum(0)
    return out


def backward(d, d_y, d_out, rstd, wanted=("d_post_gamma", "d_pre_gamma", "d_token_gate", "d_channel_gate"), spare=0, **more):
    b, H = d["x"].shape
    got = {k: torch.full((b, H), 77.0, dtype=BF, device="cuda") for k in ("d_x", "d_residual")}
    for k in wanted:
        if d[k[2:]] is not None:
            got[k] = torch.full(d[k[2:]].shape, 77.0, device="cuda")
    work = torch.full((mt.moe_tail_block_norm_grad_workspace_bytes(b, H) + spare,), 0xFF, dtype=torch.uint8, device="cuda")
    more.pop("eps", None)
    mt.moe_tail_block_norm_grad(d_y, d_out, d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], rstd, got["d_x"],
                                got["d_residual"], work, token_gate=d["token_gate"], channel_gate=d["channel_gate"],
                                **{k: got[k] for k in wanted if k in got}, **more)
    return got


def check_grad(d, d_y, d_out, got, **more):
    more = {{"residual_scale": "scale", "gain_center": "center"}.get(k, k): v for k, v in more.items()}
    want, size = plain_grad(d, d_y, d_out, **more), plain_grad(d, d_y, d_out, magnitudes=True, **more)
    b = d["x"].shape[0]
    for k, t in got.items():
        close(t, want[k], size[k], 4e-5 + (b * 2.0 ** -24 if t.dtype == F32 else 0.0))


@pytest.mark.parametrize("post,token,channel", FORMS)
@pytest.mark.parametrize("H", WIDTHS)
def test_gradients(H, post, token, channel):
    g = gen(H + 1)
    for b in (1, 3, 17, 700 if H <= 8192 else 90):
        d = inputs(g, b, H, post, token, channel)
        d_y, d_out = normal(g, b, H), normal(g, b, H, std=0.5)
        if b == 17:
            d["x"][1], d["residual"][1] = 0, 0
            d_y[2], d_out[3] = 0, 0
        more = dict(residual_scale=0.25, gain_center=0.0, eps=1e-5) if b == 3 else {}
        rstd = forward(d, **more)[2]
        got = backward(d, d_y, d_out, rstd, **more)
        check_grad(d, d_y, d_out, got, **more)
        again = backward(d, d_y, d_out, rstd, spare=4096, **more)
        assert all(torch.equal(got[k], again[k]) for k in got)  # the same bits every time
        check_grad(d, d_y, None, backward(d, d_y, None, rstd, **more), **more)
        few = backward(d, d_y, d_out, rstd, wanted=("d_pre_gamma",) if b == 1 else (), **more)  # the others not wanted
        assert all(torch.equal(few[k], got[k]) for k in few)


def test_gradients_in_place():
    g = gen(5)
    for H in (520, 4096, 8200):
        d = inputs(g, 41, H, True, True, True)
        d_y, d_out = normal(g, 41, H), normal(g, 41, H)
        rstd = forward(d)[2]
        want = backward(d, d_y, d_out, rstd)
        work = torch.empty(mt.moe_tail_block_norm_grad_workspace_bytes(41, H), dtype=torch.uint8, device="cuda")
        mt.moe_tail_block_norm_grad(d_y, d_out, d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], rstd, d_y, d_out, work,
                                    token_gate=d["token_gate"], channel_gate=d["channel_gate"])
        assert torch.equal(d_y, want["d_x"]) and torch.equal(d_out, want["d_residual"])


@pytest.mark.parametrize("post,token,channel", FORMS)
def test_gradients_against_differences(post, token, channel):
    # L = sum(d_y * y + d_out * h): its change along a direction in each input, in FP64, by central differences.  The BF16
    # gradients are off by up to 2^-9 of each element, the FP32 ones by 4e-5 of their terms; a difference with a step of 1e-5
    # by 1e-9 of L's third derivative, far less.
    g = gen(6)
    b, H = 13, 264
    d = inputs(g, b, H, post, token, channel)
    d_y, d_out = normal(g, b, H), normal(g, b, H)
    got = backward(d, d_y, d_out, forward(d, residual_scale=0.5)[2], residual_scale=0.5)
    size = plain_grad(d, d_y, d_out, scale=0.5, magnitudes=True)
    for k, grad in got.items():
        name = k[2:]
        way = torch.randn(d[name].shape, generator=g, device="cuda", dtype=F64)

        def loss(step):
            moved = to64(d)
            moved[name] = moved[name] + step * way
            h, y = plain(moved, scale=0.5)[:2]
            return (d_y.to(F64) * y).sum() + (d_out.to(F64) * h).sum()

        change = (loss(1e-5) - loss(-1e-5)) / 2e-5
        off = (way.abs() * (2.0 ** -8 * grad.to(F64).abs() * (grad.dtype == BF) + 6e-5 * size[k])).sum()
        assert abs(float(change - (way * grad.to(F64)).sum())) <= float(off) + 1e-5 * abs(float(change))


def test_no_rows():
    H = 264
    g = gen(7)
    d = inputs(g, 0, H, True, True, True)
    out, y, rstd = forward(d)
    got = backward(d, out, y, rstd)
    for k in ("d_post_gamma", "d_pre_gamma", "d_channel_gate"):
        assert (got[k] == 0).all()
    assert got["d_token_gate"].numel() == 0


def test_past_the_range_of_32_bit_offsets():
    g = gen(8)
    H, b = 32768, 70000
    x, residual, d_y = (torch.zeros((b, H), dtype=BF, device="cuda") for _ in range(3))
    d = inputs(g, 3, H, True, False, False)
    last = normal(g, 3, H)
    x[-3:], residual[-3:], d_y[-3:] = d["x"], d["residual"], last
    big = dict(d, x=x, residual=residual)
    out, y, rstd = forward(big)
    tail = tuple(t[-3:] for t in (out, y, rstd))
    check_forward(d, tail)
    assert not out[:-3].any() and not y[:-3].any()
    got = backward(big, d_y, None, rstd, wanted=("d_pre_gamma",))
    want, size = plain_grad(d, last, None), plain_grad(d, last, None, magnitudes=True)
    for k in ("d_x", "d_residual"):
        close(got[k][-3:], want[k], size[k], 4e-5)
        assert not got[k][:-3].any()
    close(got["d_pre_gamma"], want["d_pre_gamma"], size["d_pre_gamma"], 5e-5)


def test_nothing_outside_the_outputs_is_written():
    for b, H in ((1, 8), (7, 264), (33, 2056), (5, 4104), (3, 20000)):
        g, buffers = gen(H), []

        def new(dtype, *shape):
            n = int(torch.tensor([], dtype=dtype).element_size() * torch.Size(shape).numel())
            whole = torch.full((n + (1 << 16),), 0xA5, dtype=torch.uint8, device="cuda")
            buffers.append((whole, n))
            return whole[1 << 15:(1 << 15) + n].view(dtype).view(shape)

        d = inputs(g, b, H, True, True, True)
        gates = {k: d[k] for k in ("token_gate", "channel_gate")}
        rstd = new(F32, b, 2)
        mt.moe_tail_block_norm(d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], new(BF, b, H), new(BF, b, H), rstd=rstd,
                               **gates)
        mt.moe_tail_block_norm_grad(d["x"], d["residual"], d["x"], d["residual"], d["post_gamma"], d["pre_gamma"], rstd,
                                    new(BF, b, H), new(BF, b, H),
                                    new(torch.uint8, mt.moe_tail_block_norm_grad_workspace_bytes(b, H)),
                                    d_post_gamma=new(F32, H), d_pre_gamma=new(F32, H), d_token_gate=new(F32, b),
                                    d_channel_gate=new(F32, H), **gates)
        torch.cuda.synchronize()
        for whole, n in buffers:
            assert (whole[:1 << 15] == 0xA5).all() and (whole[(1 << 15) + n:] == 0xA5).all()


@pytest.mark.parametrize("H", [1032, 3000, 9000, 20000])
def test_in_graphs_that_share_a_workspace_and_on_a_side_stream(H):
    g = gen(10)
    b = 50
    d, e = inputs(g, b, H, True, True, True), inputs(g, b, H, True, True, True)
    d_y, d_out = normal(g, b, H), normal(g, b, H)
    work = torch.empty(mt.moe_tail_block_norm_grad_workspace_bytes(b, H), dtype=torch.uint8, device="cuda")
    results, graphs = [], []
    names = ("d_post_gamma", "d_pre_gamma", "d_token_gate", "d_channel_gate")
    for one in (d, e):
        results.append({k: torch.empty((b, H), dtype=BF, device="cuda") for k in ("d_x", "d_residual")}
                       | {k: torch.empty(one[k[2:]].shape, device="cuda") for k in names})

    def step(one, got):
        h, y, rstd = (torch.empty_like(t) for t in (d_y, d_y, torch.empty((b, 2), device="cuda")))
        gates = {k: one[k] for k in ("token_gate", "channel_gate")}
        mt.moe_tail_block_norm(one["x"], one["residual"], one["post_gamma"], one["pre_gamma"], h, y, rstd=rstd, **gates)
        sums = {k: v for k, v in got.items() if k not in ("d_x", "d_residual")}
        mt.moe_tail_block_norm_grad(d_y, d_out, one["x"], one["residual"], one["post_gamma"], one["pre_gamma"], rstd, got["d_x"],
                                    got["d_residual"], work, **gates, **sums)

    for one, got in zip((d, e), results):  # captured before any other call of this shape
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(one, got)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    wants = [backward(one, d_y, d_out, forward(one)[2]) for one in (d, e)]
    for got, want in zip(results, wants):
        assert all(torch.equal(got[k], want[k]) for k in want)
        for v in got.values():
            v.fill_(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(d, results[0])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(results[0][k], wants[0][k]) for k in wants[0])


@pytest.mark.parametrize("size", [1e-19, 1e19, 1e30])
@pytest.mark.parametrize("H", [520, 4104, 9000])
def test_gradients_of_rows_whose_squares_leave_the_range(size, H):
    # rstd is that of the row as it was; with d_y near one every gradient is a number of FP32's range
    g = gen(11)
    d = inputs(g, 7, H, True, True, True)
    d["x"] = (d["x"].float() * size).to(BF)
    d_y, d_out = normal(g, 7, H), normal(g, 7, H)
    if size < 1:
        d["residual"].zero_()
        d["token_gate"] += 1.0
    got = backward(d, d_y, d_out, forward(d, eps=0.0)[2])
    check_grad(d, d_y, d_out, got, eps=0.0)


def test_gradients_at_once_on_several_streams():
    g = gen(12)
    calls = []
    for b, H in ((400, 1032), (300, 4104), (200, 9000), (90, 20000)):
        d = inputs(g, b, H, True, True, True)
        calls.append((d, normal(g, b, H), normal(g, b, H), forward(d)[2]))
    wants = [backward(*c) for c in calls]
    streams, got = [torch.cuda.Stream() for _ in calls], [[] for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, stream, results in zip(calls, streams, got):
            with torch.cuda.stream(stream):
                results.append(backward(*c))
    torch.cuda.synchronize()
    for want, results in zip(wants, got):
        assert all(torch.equal(r[k], want[k]) for r in results for k in want)
    assert mt.moe_tail_take_device_error() == 0
