"""The calls around the tail on a GPU, against plain implementations in 64 bits.

Tolerances, from the formulas:
  BF16 results   half a unit in the last place, 2^-9 of the value (2^-8 of its binade's lower end), and the FP32 sum's
                 error before the rounding: at most (number of terms) * 2^-24 * (sum of the terms' magnitudes).
  8-bit scales   an FP32 sum of H squares by threads and warps (under 100 additions in a row), root, division and
                 products: under 100 * 2^-24 = 6e-6 of the value; 1e-5 is asked.
  8-bit values   half a step of the rounding, and twice the scale's relative error times the largest value.
  the product    whole numbers: exact in FP32 below 2^24, else 2^-24 an addition of the sum of magnitudes.
"""
import pytest
import torch

import moe_decode_tail_gb300 as mt

pytestmark = pytest.mark.gpu

BF, I8, I32, F32, F64, E4 = torch.bfloat16, torch.int8, torch.int32, torch.float32, torch.float64, torch.float8_e4m3fn
MOST = {I8: 127.0, E4: 448.0}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def filled(dtype, *shape, value=77):
    return torch.full(shape, value, dtype=F32, device="cuda").to(dtype)


def close_bf16(got, want, slack=0.0):
    """got BF16, want FP64: half a unit in the last place, and slack (FP64, the error before the rounding)."""
    assert got.dtype == BF and got.shape == want.shape
    off = (got.to(F64) - want).abs()
    bound = want.abs() * 2.0 ** -8 * (1 + 2.0 ** -10) + slack + 1e-40
    bad = ~(off <= bound)
    assert not bad.any(), (int(bad.sum()), off[bad].max().item(), want[bad][:4])
    assert not (got.view(torch.int16) == -32768).any()  # -0 is written as +0


def check_rows(q, scale, v, group):
    """q and scale against v (FP64): every value within half a step."""
    rows, width = v.shape
    size = group or width
    for g in range(-(-width // size)):
        part, got = v[:, g * size:(g + 1) * size], q[:, g * size:(g + 1) * size].to(F32).to(F64)
        sc = (scale[:, g] if group else scale).to(F64)
        top = part.abs().max(1).values
        want = top / MOST[q.dtype]
        sane = want > 1e-36  # below, the FP32 scale itself is coarse
        assert ((sc - want).abs() <= 1e-5 * want + 1e-44).all()
        assert ((top == 0) == (sc == 0))[sane | (top == 0)].all()
        assert (got[top == 0] == 0).all()
        ratio = (part / want.clamp_min(1e-300)[:, None])[sane]
        got = got[sane]
        if q.dtype == I8:
            half = torch.full_like(ratio, 0.5)
        else:
            unit = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp_min(1e-30))).clamp_min(-6.0) - 3)
            half = unit / 2
        off = (got - ratio).abs()
        assert (off <= half * (1 + 1e-5) + 2e-5 * ratio.abs() + 1e-9).all(), (off - half).max()
        assert (got.abs() <= MOST[q.dtype]).all()


WIDTHS = [8, 24, 120, 128, 136, 264, 1000, 4096, 7168, 8192, 8200, 16376, 32768]


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_quant(H, group, dtype):
    g = gen(H + group)
    for b in (1, 5, 700):
        x, res, gamma = normal(g, b, H), normal(g, b, H, std=3.0), normal(g, H, std=0.1)
        if b == 5:
            x[1], res[1] = 0, 0                       # a row of zeros
            x[2], res[2] = x[2] * 1e-18, res[2] * 1e-18  # far below eps
            x[3], res[3] = x[3] * 1e15, res[3] * 1e15
            x[4, : H // 2], res[4, : H // 2] = 0, 0   # groups of zeros
        q, scale = filled(dtype, b, H), filled(F32, b, -(-H // 128)) if group else filled(F32, b)
        out, y = filled(BF, b, H), filled(BF, b, H)
        mt.moe_tail_norm_quant(x, res, gamma, q, scale, residual_out=out, y=y, gain_center=1.0, eps=1e-6, group=group)
        h = x.to(F64) + res.to(F64)
        v = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * (gamma.to(F64) + 1.0)
        close_bf16(out, h, h.abs() * 2.0 ** -24)
        close_bf16(y, v, v.abs() * 1e-5)
        check_rows(q, scale, v, group)
        # the optional outputs change nothing, the residual may be updated in place, and it may be absent
        q2, scale2, res2 = torch.empty_like(q), torch.empty_like(scale), res.clone()
        mt.moe_tail_norm_quant(x, res2, gamma, q2, scale2, residual_out=res2, group=group)
        assert torch.equal(q2.view(I8), q.view(I8)) and torch.equal(scale2, scale) and torch.equal(res2, out)
        mt.moe_tail_norm_quant(x, None, gamma, q2, scale2, group=group, gain_center=0.0, eps=1e-5)
        h = x.to(F64)
        check_rows(q2, scale2, h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * gamma.to(F64), group)
        x2 = x.clone()  # in place of x
        mt.moe_tail_norm_quant(x2, res, gamma, q2, scale2, residual_out=x2, group=group)
        assert torch.equal(q2.view(I8), q.view(I8)) and torch.equal(x2, out)


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
def test_quantised_rows_that_are_not_finite(group, dtype):
    H = 520
    g = gen(1)
    x, gamma = normal(g, 4, H), normal(g, H)
    x[1, 300], x[2, 7] = float("nan"), float("inf")
    q, scale = filled(dtype, 4, H), filled(F32, 4, 5) if group else filled(F32, 4)
    mt.moe_tail_norm_quant(x, None, gamma, q, scale, group=group)
    s = scale.view(4, -1)
    assert s[0].isfinite().all() and s[3].isfinite().all()
    assert s[1].isnan().all() and s[2, 0].isnan()  # a NaN's norm is the row's; an infinity leaves NaN in its place
    assert (q[1].float() == 0).all() and (q[2, :128].float() == 0).all()
    # silu: only the group with the value
    gate_up = normal(g, 4, 2 * H)
    gate_up[1, 300], gate_up[2, H + 7], gate_up[3, 5] = float("nan"), float("inf"), float("-inf")
    mt.moe_tail_silu_quant(gate_up, q, scale, group=group)
    s = scale.view(4, -1)
    assert s[0].isfinite().all()
    for row, column in ((1, 300), (2, 7), (3, 5)):
        hit = column // 128 if group else 0
        assert s[row, hit].isnan() and int(s[row].isnan().sum()) == 1
        assert (q[row, hit * 128:(hit + 1) * 128].float() == 0).all()


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("width", WIDTHS)
def test_silu_quant(width, group, dtype):
    g = gen(width + group)
    for rows in (1, 3, 600):
        gate_up = normal(g, rows, 2 * width, std=3.0)
        if rows == 3:
            gate_up[0] = 0
            gate_up[1, :width] = -100.0               # silu is a tiny negative number
            gate_up[2] = gate_up[2] * 1e-17           # products of 1e-34
        q, scale = filled(dtype, rows, width), filled(F32, rows, -(-width // 128)) if group else filled(F32, rows)
        mt.moe_tail_silu_quant(gate_up, q, scale, group=group)
        gate, up = gate_up[:, :width].to(F64), gate_up[:, width:].to(F64)
        live = torch.ones(rows, dtype=torch.bool, device="cuda")
        live[1:2] = rows != 3  # exp(100) * 100 is at the edge of FP32's normal numbers
        check_rows(q[live], scale[live], (gate * torch.sigmoid(gate) * up)[live], group)
        for used in (0, 1, rows, rows + 5, -1):
            q2, scale2 = filled(dtype, rows, width), filled(F32, *scale.shape)
            mt.moe_tail_silu_quant(gate_up, q2, scale2, group=group,
                                   used_rows=torch.tensor([used], dtype=I32, device="cuda"))
            n = max(0, min(used, rows))
            assert torch.equal(q2[:n].view(I8), q[:n].view(I8)) and torch.equal(scale2[:n], scale[:n])
            assert (q2[n:].float() == filled(dtype, 1).float()).all() and (scale2[n:] == 77).all()


# ---- routes --------------------------------------------------------------------------------------------------------


def plain_sort(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    offsets = torch.stack([(key < e).sum() for e in range(E + 1)]) if flat.numel() else flat.new_zeros(E + 1)
    n = int(offsets[E])
    idx = torch.full_like(flat, -1)
    idx[order[:n]] = torch.arange(n, device=ids.device)
    source = torch.full_like(flat, -1)
    source[:n] = order[:n]
    return offsets.to(I32), idx.reshape(ids.shape).to(I32), source.to(I32)


def sort(ids, E):
    b, K = ids.shape
    offsets, idx, source = filled(I32, E + 1), filled(I32, b, K), filled(I32, b * K)
    ws = filled(torch.uint8, mt.moe_tail_sort_workspace_bytes(b, K, E))
    mt.moe_tail_sort_routes(ids, offsets, idx, source, ws)
    return offsets, idx, source


@pytest.mark.parametrize("b,K,E", [(0, 4, 8), (1, 1, 1), (1, 8, 128), (3, 5, 1024), (64, 8, 128), (512, 8, 33), (513, 8, 7),
                                   (1024, 4, 1), (1365, 3, 1024), (4099, 16, 60), (20000, 8, 256), (65535, 32, 128)])
def test_sort_routes(b, K, E):
    g = gen(b + K)
    ids = torch.randint(0, E, (b, K), generator=g, device="cuda", dtype=I32)
    for skew in (False, True):
        if skew and b:  # one expert has most, some routes have none
            ids[torch.rand((b, K), generator=g, device="cuda") < 0.6] = E - 1
            drop = torch.rand((b, K), generator=g, device="cuda") < 0.3
            ids[drop] = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=I32, device="cuda")[
                torch.randint(0, 4, (int(drop.sum()),), generator=g, device="cuda")]
        for got, want in zip(sort(ids, E), plain_sort(ids, E)):
            assert torch.equal(got, want)
    nobody = torch.full((b, K), -1, dtype=I32, device="cuda")
    offsets, idx, source = sort(nobody, E)
    assert (offsets == 0).all() and (idx == -1).all() and (source == -1).all()


def routes(g, b, K, E, local=0.7):
    ids = torch.rand((b, E), generator=g, device="cuda").topk(K, dim=1).indices.to(I32)
    ids[torch.rand((b, K), generator=g, device="cuda") >= local] = -1
    if b > 2:
        ids[1] = -1  # a token without a row
    return ids, plain_sort(ids, E)


@pytest.mark.parametrize("dtype", [BF, I8, E4])
@pytest.mark.parametrize("b,K,E,H", [(1, 1, 1, 8), (1, 8, 16, 4096), (5, 3, 8, 24), (64, 8, 128, 7168), (300, 2, 60, 1000),
                                     (3, 32, 64, 32768), (40, 6, 9, 136)])
def test_dispatch_rows(b, K, E, H, dtype):
    g = gen(b + H)
    _, (_, idx, _) = routes(g, b, K, E)
    if b == 5:
        idx[4, 0] = b * K + 3  # past the rows
    x = normal(g, b, H, std=30.0).clamp(-120, 120).to(dtype)
    scale = torch.rand(b, generator=g, device="cuda")
    R = b * K
    rows, row_scale = filled(dtype, R, H), filled(F32, R)
    mt.moe_tail_dispatch_rows(x, idx, rows, scale=scale, row_scale=row_scale)
    want, want_scale = filled(dtype, R, H), filled(F32, R)
    for t in range(b):
        for j in idx[t].tolist():
            if 0 <= j < R:
                want[j], want_scale[j] = x[t], scale[t]
    assert torch.equal(rows.view(I8), want.view(I8)) and torch.equal(row_scale, want_scale)
    rows2 = filled(dtype, R, H)
    mt.moe_tail_dispatch_rows(x, idx, rows2)
    assert torch.equal(rows2.view(I8), want.view(I8))


def plain_combine(rows, idx, w):
    """FP64 sum over the routes with a row, and the sum of magnitudes."""
    R = rows.shape[0]
    live = (idx >= 0) & (idx < R)
    picked = rows.to(F64)[torch.where(live, idx, 0).long()]
    weight = torch.ones(idx.shape, dtype=F64, device="cuda") if w is None else w.to(F64)
    terms = torch.where(live[:, :, None], picked * weight[:, :, None], 0.0)
    return terms.sum(1), terms.abs().sum(1)


COMBINE = [(1, 1, 1, 8), (1, 8, 16, 4096), (5, 3, 8, 24), (64, 8, 128, 7168), (700, 2, 60, 1000), (3, 32, 64, 32768),
           (33, 16, 20, 8200), (2, 7, 9, 16384)]


@pytest.mark.parametrize("weights", [F32, BF, None])
@pytest.mark.parametrize("b,K,E,H", COMBINE)
def test_combine_rows(b, K, E, H, weights):
    g = gen(b * H)
    _, (_, idx, source) = routes(g, b, K, E)
    rows = normal(g, b * K, H)
    w = None if weights is None else torch.softmax(normal(g, b, K, dtype=F32), 1).to(weights)
    if b == 5:
        idx[4, 0] = b * K + 3
    live = (idx >= 0) & (idx < b * K)
    rows[source < 0] = float("nan")  # rows of no route, weights of routes without a row: never looked at
    if w is not None:
        w[~live] = float("nan")
    out = filled(BF, b, H)
    mt.moe_tail_combine_rows(rows, idx, w, out)
    clean = torch.nan_to_num(rows, nan=0.0)
    want, size = plain_combine(clean, idx, None if w is None else torch.where(live, w, 0))
    close_bf16(out, want, 2 * K * 2.0 ** -24 * size)
    if b > 2:
        assert (out[1] == 0).all()


def test_combine_keeps_what_is_not_finite():
    rows = torch.ones((4, 64), dtype=BF, device="cuda")
    rows[0, 3], rows[1, 5] = float("inf"), float("nan")
    idx = torch.tensor([[0, 1], [2, 3]], dtype=I32, device="cuda")
    out = filled(BF, 2, 64)
    mt.moe_tail_combine_rows(rows, idx, torch.ones((2, 2), device="cuda"), out)
    assert out[0, 3] == float("inf") and out[0, 5].isnan() and (out[0, 6:] == 2).all() and (out[1] == 2).all()


@pytest.mark.parametrize("weights", [F32, BF])
@pytest.mark.parametrize("b,K,E,H", COMBINE)
def test_combine_grad(b, K, E, H, weights):
    g = gen(b * H + 1)
    _, (_, idx, source) = routes(g, b, K, E)
    R = b * K
    rows, d_out = normal(g, R, H), normal(g, b, H)
    w = torch.softmax(normal(g, b, K, dtype=F32), 1).to(weights)
    if b == 5:
        idx[4, 0] = R + 3
    live = (idx >= 0) & (idx < R)
    named = torch.zeros(R, dtype=torch.bool, device="cuda")
    named[idx[live].long()] = True
    rows[~named] = float("nan")
    w[~live] = float("nan")
    d_rows, d_w = filled(BF, R, H), filled(F32, b, K)
    mt.moe_tail_combine_grad(d_out, rows, idx, w, d_rows, d_w)
    assert (d_rows[~named] == 77).all() and (d_w[~live] == 0).all()

    # the formula, by 64-bit automatic differentiation of the plain sum
    r64 = torch.nan_to_num(rows, nan=0.0).to(F64).requires_grad_()
    w64 = torch.where(live, w.to(F64), 0.0).requires_grad_()
    place = torch.where(live, idx, 0).long()
    out = (torch.where(live[:, :, None], r64[place], 0.0) * w64[:, :, None]).sum(1)
    out.backward(d_out.to(F64))
    close_bf16(d_rows[named], r64.grad[named], r64.grad[named].abs() * 2.0 ** -24)
    size = (torch.where(live[:, :, None], r64[place], 0.0) * d_out.to(F64)[:, None, :]).abs().sum(2)
    assert ((d_w.to(F64) - w64.grad).abs() <= 200 * 2.0 ** -24 * size + 1e-30).all()  # under 200 additions in a row

    # and by differences: the loss is linear in each weight and each row
    with torch.no_grad():
        loss = lambda rr, ww: float((plain_combine(rr, idx, ww)[0] * d_out.to(F64)).sum())  # noqa: E731
        base_r, base_w = r64.detach(), w64.detach()
        for t, k in ((0, 0), (b - 1, K - 1), (b // 2, K // 2)):
            up, down = base_w.clone(), base_w.clone()
            up[t, k] += 0.5
            down[t, k] -= 0.5
            diff = loss(base_r, up) - loss(base_r, down)
            assert abs(diff - float(d_w[t, k])) <= 200 * 2.0 ** -24 * float(size[t, k]) + 1e-9 * abs(loss(base_r, base_w)) + 1e-9
            if live[t, k]:
                j = int(idx[t, k])
                up = base_r.clone()
                up[j, H // 2] += 1.0
                diff = loss(up, base_w) - loss(base_r, base_w)
                assert abs(diff - float(d_rows[j, H // 2])) <= 2.0 ** -8 * abs(diff) + 1e-9 * abs(loss(base_r, base_w)) + 1e-9


def test_dispatch_gradient_is_the_unweighted_combine():
    g = gen(9)
    b, K, E, H = 37, 4, 10, 264
    _, (_, idx, _) = routes(g, b, K, E)
    R = b * K
    d_rows = normal(g, R, H)
    x = normal(g, b, H).to(F64).requires_grad_()
    live = idx >= 0
    rows = torch.zeros((R, H), dtype=F64, device="cuda")
    token = torch.arange(b, device="cuda")[:, None].expand(b, K)
    rows = rows.index_put((idx[live].long(),), x[token[live]])
    rows.backward(d_rows.to(F64))
    d_x = filled(BF, b, H)
    mt.moe_tail_combine_rows(d_rows, idx, None, d_x)
    close_bf16(d_x, x.grad, 2 * K * 2.0 ** -24 * plain_combine(d_rows, idx, None)[1])


# ---- the 8-bit product ---------------------------------------------------------------------------------------------


def product(x, xs, w, ws, offsets, slack=0):
    R, (E, N, D) = x.shape[0], w.shape
    out = filled(BF, R, N)
    work = torch.empty(mt.moe_tail_expert_product_workspace_bytes(R, E, N, D) + slack, dtype=torch.uint8, device="cuda")
    work.fill_(255)  # NaNs, whatever its parts are read as
    mt.moe_tail_expert_product(x, xs, w, ws, out, work, expert_offsets=offsets)
    return out


def check_product(out, x, xs, w, ws, offsets):
    ends = [0, x.shape[0]] if offsets is None else offsets.tolist()
    for e in range(w.shape[0]):
        i, j = ends[e], ends[e + 1]
        if i == j:
            continue
        x64, w64 = x[i:j].to(F64), w[e].to(F64)
        scale = xs[i:j].to(F64)[:, None] * ws[e].to(F64)[None, :]
        size = (x64.abs() @ w64.abs().T) * scale.abs()
        want = (x64 @ w64.T) * scale
        exact = size < 2.0 ** 24 * scale.abs()
        slack = want.abs() * 2.0 ** -22 + torch.where(exact, 0.0, x.shape[1] * 2.0 ** -24 * size)
        close_bf16(out[i:j], want, slack)
    assert (out[ends[-1]:] == 77).all()  # rows of no expert


def int8(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=I32).to(I8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.02 + 0.001


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 144, 272, 1040])
@pytest.mark.parametrize("N", [8, 24, 128, 136, 384])
def test_dense_product(N, D):
    g = gen(N * D)
    w, ws = int8(g, 1, N, D), scales(g, 1, N)
    for R in (1, 7, 16, 17, 33, 64, 130, 257, 600):
        x, xs = int8(g, R, D), scales(g, R)
        out = product(x, xs, w, ws, None)
        check_product(out, x, xs, w, ws, None)
        offsets = torch.tensor([0, R], dtype=I32, device="cuda")
        assert torch.equal(product(x, xs, w, ws, offsets, slack=512), out)


@pytest.mark.parametrize("E,N,D", [(2, 8, 16), (5, 136, 144), (16, 256, 512), (60, 128, 256), (128, 512, 1024), (1024, 128, 64)])
def test_expert_product(E, N, D):
    g = gen(E + D)
    w, ws = int8(g, E, N, D), scales(g, E, N)
    for kind in ("few", "even", "odd", "one", "none", "many"):
        if kind == "few":
            counts = torch.zeros(E, dtype=torch.long)
            counts[torch.randperm(E)[: max(1, E // 3)]] = 1
        elif kind == "even":
            counts = torch.full((E,), 3)
        elif kind == "odd":
            counts = torch.arange(E) * 7 % 41
        elif kind == "one":  # one expert has every row
            counts = torch.zeros(E, dtype=torch.long)
            counts[E // 2] = 333
        elif kind == "none":
            counts = torch.zeros(E, dtype=torch.long)
        else:
            counts = torch.randint(0, 2 + 3000 // E, (E,)) + (torch.arange(E) == 1) * 300
        offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(I32).cuda()
        R = int(offsets[-1]) + 5  # rows of no expert at the end
        x, xs = int8(g, R, D), scales(g, R)
        xs[-5:] = float("nan")
        check_product(product(x, xs, w, ws, offsets), x, xs, w, ws, offsets)


@pytest.mark.parametrize("b", [4, 100, 200, 500, 1000, 3000])
def test_expert_product_over_many_tiles(b):
    # several tiles for every thread block at each tile height (16 to 256 rows), uneven experts with several row tiles,
    # the reduction longer than the rings; several calls in flight at once, each reading what the last one left
    g = gen(b)
    E, K, N, D = 64, 4, 1032, 2064
    w, ws = int8(g, E, N, D), scales(g, E, N)
    ids = (torch.rand((b, E), generator=g, device="cuda") * torch.linspace(1.0, 3.0, E, device="cuda")).topk(K, 1).indices
    offsets, _, _ = plain_sort(ids.to(I32), E)
    R = b * K
    x, xs = int8(g, R, D), scales(g, R)
    out = product(x, xs, w, ws, offsets)
    work = torch.empty(mt.moe_tail_expert_product_workspace_bytes(R, E, N, D), dtype=torch.uint8, device="cuda")
    again = [filled(BF, R, N) for _ in range(6)]
    for o in again:
        mt.moe_tail_expert_product(x, xs, w, ws, o, work, expert_offsets=offsets)
    check_product(out, x, xs, w, ws, offsets)
    assert all(torch.equal(o, out) for o in again)
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("b", [512, 1024])
def test_expert_product_of_a_weight_that_streams(b):
    # 1 GB of weights, so that copies land late and in any order, at 64 and 128 rows a tile
    g = gen(b)
    E, K, N, D = 128, 8, 2048, 4096
    w, ws = int8(g, E, N, D // 4).repeat(1, 1, 4), scales(g, E, N)
    ids = (torch.rand((b, E), generator=g, device="cuda") * torch.linspace(1.0, 2.0, E, device="cuda")).topk(K, 1).indices
    offsets, _, _ = plain_sort(ids.to(I32), E)
    x, xs = int8(g, b * K, D), scales(g, b * K)
    out = product(x, xs, w, ws, offsets)
    check_product(out, x, xs, w, ws, offsets)
    work = torch.empty(mt.moe_tail_expert_product_workspace_bytes(b * K, E, N, D), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        again = filled(BF, b * K, N)
        mt.moe_tail_expert_product(x, xs, w, ws, again, work, expert_offsets=offsets)
        assert torch.equal(again, out)
    assert mt.moe_tail_take_device_error() == 0


@pytest.mark.parametrize("R", [80, 128])
def test_dense_product_of_tall_tiles(R):
    g = gen(R)
    N, D = 19456 // 2, 2000
    w, ws, x, xs = int8(g, 1, N, D), scales(g, 1, N), int8(g, R, D), scales(g, R)
    check_product(product(x, xs, w, ws, None), x, xs, w, ws, None)


def test_product_at_the_largest_sums_and_with_scales_that_are_not_finite():
    g = gen(3)
    R, N, D = 40, 256, 4096
    w, x = torch.full((1, N, D), 127, dtype=I8, device="cuda"), torch.full((R, D), -127, dtype=I8, device="cuda")
    w[0, 1::2], x[1::3], w[0, 5], x[4] = -128, -128, 0, 0
    xs, ws = scales(g, R), scales(g, 1, N)
    check_product(product(x, xs, w, ws, None), x, xs, w, ws, None)
    xs[7], ws[0, 9] = float("nan"), float("inf")
    out = product(x, xs, w, ws, None)
    assert out[7].isnan().all() and out[4, 9].isnan() and out[0, 9].isinf()
    keep = torch.ones((R, N), dtype=torch.bool, device="cuda")
    keep[7], keep[:, 9] = False, False
    assert out[keep].isfinite().all()


def test_product_with_offsets_that_are_no_partition():
    # whatever the offsets hold, no row outside [0, R) is touched
    g = gen(4)
    E, N, D, R = 3, 128, 128, 20
    w, ws, x, xs = int8(g, E, N, D), scales(g, E, N), int8(g, R, D), scales(g, R)
    for bad in ([0, 5, 5, 10 ** 6], [-7, 3, 2, 9], [12, 4, 30, 1], [2 ** 31 - 1, -2 ** 31, 0, 20]):
        big = filled(BF, R + 64, N)
        work = torch.empty(mt.moe_tail_expert_product_workspace_bytes(R, E, N, D), dtype=torch.uint8, device="cuda")
        mt.moe_tail_expert_product(x, xs, w, ws, big[32:32 + R], work,
                                   expert_offsets=torch.tensor(bad, dtype=I32, device="cuda"))
        torch.cuda.synchronize()
        assert (big[:32] == 77).all() and (big[32 + R:] == 77).all()
    assert mt.moe_tail_take_device_error() == 0


def test_product_whose_waits_run_out():
    # a limit of one nanosecond on the tensor cores' operands: the call gives up, says so and leaves the device usable
    g = gen(8)
    E, N, D, R = 4, 256, 512, 60
    w, ws, x, xs = int8(g, E, N, D), scales(g, E, N), int8(g, R, D), scales(g, R)
    offsets = torch.tensor([0, 20, 20, 45, 60], dtype=I32, device="cuda")
    assert mt.moe_tail_take_device_error() == 0
    mt.moe_tail_set_stage_wait_limit(1)
    try:
        product(x, xs, w, ws, offsets)
        torch.cuda.synchronize()
    finally:
        mt.moe_tail_set_stage_wait_limit(0)
    assert mt.moe_tail_take_device_error() & 1
    check_product(product(x, xs, w, ws, offsets), x, xs, w, ws, offsets)
    assert mt.moe_tail_take_device_error() == 0


# ---- together, on other streams and in graphs -------------------------------------------------------------------------


def layer(g, b, E, K, H, I, finalize):
    from moe_decode_tail_gb300.expert_layer import ExpertLayerI8, quantise_channels

    wg, sg = quantise_channels(normal(g, E, 2 * I, H, std=0.05))
    wd, sd = quantise_channels(normal(g, E, H, I, std=0.05))
    return ExpertLayerI8(normal(g, H, std=0.1), wg, sg, wd, sd, max_tokens=b, top_k=K,
                         finalize_gamma=normal(g, H, std=0.1) if finalize else None)


def plain_layer(m, x, residual, ids, w):
    """The layer in FP64 but for the roundings to 8 bits and BF16 that it defines."""
    def eight(v):
        scale = v.abs().amax(1, keepdim=True) / 127.0
        return torch.where(scale > 0, torch.round(v / scale), 0.0) * scale

    h = x.to(F64) + residual.to(F64)
    v = eight(h / torch.sqrt((h * h).mean(1, keepdim=True) + m.eps) * (m.gamma.to(F64) + m.gain_center))
    out = torch.zeros_like(v)
    I = m.I2 // 2
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if not 0 <= e < m.E:
                continue
            gu = ((m.w_gate_up[e].to(F64) * m.s_gate_up[e].to(F64)[:, None]) @ v[t]).to(BF).to(F64)
            z = eight((gu[:I] * torch.sigmoid(gu[:I]) * gu[I:])[None])[0]
            row = ((m.w_down[e].to(F64) * m.s_down[e].to(F64)[:, None]) @ z).to(BF).to(F64)
            if m.finalize_gamma is not None:
                row = row * (m.finalize_gamma.to(F64) + m.gain_center)
                row = row / torch.sqrt((row * row).mean() + m.eps)
            out[t] += float(w[t, k]) * row
    return h, out


@pytest.mark.parametrize("finalize", [True, False])
def test_expert_layer(finalize):
    g = gen(5)
    b, E, K, H, I = 19, 12, 3, 512, 256
    m = layer(g, b + 4, E, K, H, I, finalize)
    for tokens in (b, 1, 7):
        x, residual = normal(g, tokens, H), normal(g, tokens, H)
        ids, _ = routes(g, tokens, K, E, local=0.8)
        w = torch.softmax(normal(g, tokens, K, dtype=F32), 1)
        h, want = plain_layer(m, x, residual, ids, w)
        y, out = filled(BF, tokens, H), filled(BF, tokens, H)
        res = residual.clone()
        assert m.norm(x, res, y=y) is res
        m.experts(ids, w, out)
        close_bf16(res, h, h.abs() * 2.0 ** -24)
        # a rounding to 8 bits may fall to the other side where FP32 and FP64 differ: one step of one of 256 or 512
        # values, 1/127 of the largest, moves a row by under 1/127 / sqrt(256) = 5e-4 of its size; BF16 by 2^-9
        off = (out.to(F64) - want).norm(dim=1)
        assert (off <= 5e-3 * want.norm(dim=1) + 1e-6).all(), (off / want.norm(dim=1)).max()
    with pytest.raises(ValueError, match="tokens"):
        m.norm(normal(g, b + 5, H), None)


def test_expert_layer_without_tokens_and_without_local_experts():
    g = gen(11)
    E, K, H, I = 8, 2, 256, 128
    for finalize in (True, False):
        m = layer(g, 6, E, K, H, I, finalize)
        none, out = filled(BF, 0, H), filled(BF, 0, H)
        m.norm(none, none.clone())
        m.experts(torch.empty((0, K), dtype=I32, device="cuda"), torch.empty((0, K), device="cuda"), out)
        assert (m._offsets == 0).all()
        x, out = normal(g, 6, H), filled(BF, 6, H)
        m.norm(x, None)
        m.experts(torch.full((6, K), -1, dtype=I32, device="cuda"), torch.ones((6, K), device="cuda"), out)
        assert (out == 0).all()
    assert mt.moe_tail_take_device_error() == 0


def test_expert_layer_in_a_graph_and_on_a_side_stream():
    g = gen(6)
    b, E, K, H, I = 24, 16, 4, 256, 128
    m = layer(g, b, E, K, H, I, True)
    x, residual, res = normal(g, b, H), normal(g, b, H), filled(BF, b, H)
    ids, _ = routes(g, b, K, E)
    w = torch.softmax(normal(g, b, K, dtype=F32), 1)
    out = filled(BF, b, H)

    def step():
        m.norm(x, residual, residual_out=res)
        m.experts(ids, w, out)

    step()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.fill_(0)
        step()
        again = out.clone()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # another input in the same buffers: other routes, then the first again
    x0, ids0 = x.clone(), ids.clone()
    x.copy_(normal(g, b, H))
    ids.copy_(routes(g, b, K, E)[0])
    out.fill_(0)
    graph.replay()
    other = out.clone()
    step()
    assert torch.equal(out, other) and not torch.equal(other, want)
    x.copy_(x0)
    ids.copy_(ids0)
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, want)
    assert mt.moe_tail_take_device_error() == 0


def test_large_offsets():
    # rows past 2^31 elements: the last ones are read and written where they belong
    g = gen(7)
    H, R = 32768, 70000
    rows = torch.zeros((R, H), dtype=BF, device="cuda")
    rows[-3:] = normal(g, 3, H)
    idx = torch.tensor([[R - 1, 0], [R - 3, R - 2]], dtype=I32, device="cuda")
    w = torch.tensor([[1.0, 1.0], [0.5, 2.0]], device="cuda")
    out = filled(BF, 2, H)
    mt.moe_tail_combine_rows(rows, idx, w, out)
    want, size = plain_combine(rows[-3:], idx - (R - 3), w)
    close_bf16(out, want, 4 * 2.0 ** -24 * size)
    d_rows, d_w = torch.zeros_like(rows), filled(F32, 2, 2)
    mt.moe_tail_combine_grad(out, rows, idx, w, d_rows, d_w)
    assert torch.equal(d_rows[R - 2], out[1] * 2) and torch.equal(d_rows[R - 1], out[0]) and torch.equal(d_rows[0], out[0])
    assert not d_rows[1:R - 3].any()
    mt.moe_tail_dispatch_rows(out, idx, rows)
    assert torch.equal(rows[R - 1], out[0]) and torch.equal(rows[R - 2], out[1]) and torch.equal(rows[0], out[0])


class Guarded:
    """Output tensors inside larger buffers, whose other bytes must stay as they are."""

    def __init__(self):
        self.buffers = []

    def __call__(self, dtype, *shape, align=256):
        n = int(torch.tensor([], dtype=dtype).element_size() * torch.Size(shape).numel())
        pad = 1 << 16
        whole = torch.full((pad + n + pad,), 0xA5, dtype=torch.uint8, device="cuda")
        start = pad + (-(whole.data_ptr() + pad)) % align
        self.buffers.append((whole, start, n))
        return whole[start:start + n].view(dtype).view(shape)

    def intact(self):
        return all((w[:s] == 0xA5).all() and (w[s + n:] == 0xA5).all() for w, s, n in self.buffers)


@pytest.mark.parametrize("b,K,E,H,N", [(1, 1, 1, 16, 8), (3, 2, 5, 48, 24), (37, 3, 9, 272, 136), (130, 4, 16, 1040, 392),
                                       (513, 6, 60, 528, 200), (700, 2, 3, 4112, 1032)])
def test_nothing_outside_the_outputs_is_written(b, K, E, H, N):
    g, new = gen(b + H), Guarded()
    R = b * K
    x, res, gamma = normal(g, b, H), normal(g, b, H), normal(g, H)
    for dtype, group in ((I8, 0), (E4, 128)):
        scale = [b] if not group else [b, -(-H // 128)]
        mt.moe_tail_norm_quant(x, res, gamma, new(dtype, b, H), new(F32, *scale), residual_out=new(BF, b, H),
                               y=new(BF, b, H), group=group)
        mt.moe_tail_silu_quant(normal(g, b, 2 * H), new(dtype, b, H), new(F32, *scale), group=group)
    ids, _ = routes(g, b, K, E, local=0.8)
    offsets, idx, source = new(I32, E + 1), new(I32, b, K), new(I32, R)
    mt.moe_tail_sort_routes(ids, offsets, idx, source, new(torch.uint8, mt.moe_tail_sort_workspace_bytes(b, K, E)))
    for got, want in zip((offsets, idx, source), plain_sort(ids, E)):
        assert torch.equal(got, want)
    x8, xs = int8(g, b, H), scales(g, b)
    rows8, row_scale = new(I8, R, H), new(F32, R)
    mt.moe_tail_dispatch_rows(x8, idx, rows8, scale=xs, row_scale=row_scale)
    mt.moe_tail_dispatch_rows(x, idx, new(BF, R, H))
    w = torch.softmax(normal(g, b, K, dtype=F32), 1)
    rows = normal(g, R, H)
    mt.moe_tail_combine_rows(rows, idx, w, new(BF, b, H))
    mt.moe_tail_combine_grad(x, rows, idx, w, new(BF, R, H), new(F32, b, K))
    wide, ws = int8(g, E, N, H), scales(g, E, N)
    mt.moe_tail_expert_product(rows8, row_scale, wide, ws, new(BF, R, N),
                               new(torch.uint8, mt.moe_tail_expert_product_workspace_bytes(R, E, N, H)),
                               expert_offsets=offsets)
    mt.moe_tail_expert_product(x8, xs, wide[:1], ws[:1], new(BF, b, N),
                               new(torch.uint8, mt.moe_tail_expert_product_workspace_bytes(b, 1, N, H)))
    torch.cuda.synchronize()
    assert new.intact()
    assert mt.moe_tail_take_device_error() == 0
