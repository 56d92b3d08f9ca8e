"""The 4-bit layer's calls together on a GPU (norms, sort, dispatch, gated product, product, finalize), against the same
steps in 64 bits with the BF16 roundings between them.

Tolerance: between two calls the values are BF16; where FP32 and FP64 differ, a rounding may fall to the other side, one unit
(2^-8 of a value) in a few elements of a row: under 2^-9 of the row's size after each of the three roundings on the way (rows,
activations, route rows), and 2^-9 for the result's own: 5e-3 of a row's size is asked in all."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300.expert_layer import ExpertLayerI4, quantise_groups

pytestmark = pytest.mark.gpu

BF, I32, F32, F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def stands_for(packed, gs, cs, group, D):
    """FP64 weights of quantise_groups' result."""
    nibbles = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).to(torch.int64) - 8  # in a word's order
    words = nibbles.view(*packed.shape[:-1], -1, 4, 4, 8)                                  # block, t, i, nibble
    columns = torch.empty_like(words)
    columns[..., 0::2], columns[..., 1::2] = words[..., :4], words[..., 4:]
    q = columns.transpose(-2, -3).reshape(*packed.shape[:-1], -1)[..., :D].to(F64)
    return q * gs.float().to(F64).repeat_interleave(group, -1)[..., :D] * cs.to(F64)[..., None]


def make(g, b, E, K, H, I, group, post, finalize):
    m = ExpertLayerI4(normal(g, H, std=0.1), quantise_groups(normal(g, E, 2 * I, H, std=0.05), group),
                      quantise_groups(normal(g, E, H, I, std=0.05), group), max_tokens=b, top_k=K, group=group,
                      post_gamma=normal(g, H, std=0.1) if post else None, residual_scale=0.75,
                      finalize_gamma=normal(g, H, std=0.1) if finalize else None)
    m.weights = stands_for(*m.gate_up, group, H), stands_for(*m.down, group, I)
    return m


def plain(m, x, residual, token, ids, w):
    n = x.to(F64)
    if m.post_gamma is not None:
        n = n / torch.sqrt((n * n).mean(1, keepdim=True) + m.eps) * (m.post_gamma.to(F64) + m.gain_center)
    h = m.residual_scale * residual.to(F64) + (n if token is None else n * token.to(F64)[:, None])
    v = (h / torch.sqrt((h * h).mean(1, keepdim=True) + m.eps) * (m.gamma.to(F64) + m.gain_center)).to(BF).to(F64)
    out = torch.zeros_like(v)
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if not 0 <= e < m.E:
                continue
            p = m.weights[0][e] @ v[t]
            z = (p[:m.I] * torch.sigmoid(p[:m.I]) * p[m.I:]).to(BF).to(F64)
            row = (m.weights[1][e] @ z).to(BF).to(F64)
            if m.finalize_gamma is not None:
                row = row * (m.finalize_gamma.to(F64) + m.gain_center)
                row = row / torch.sqrt((row * row).mean() + m.eps)
            out[t] += float(w[t, k]) * row
    return h, v, out


def routes(g, b, K, E, local=0.8):
    ids = torch.rand((b, E), generator=g, device="cuda").topk(K, 1).indices.to(I32)
    ids[torch.rand((b, K), generator=g, device="cuda") >= local] = -1
    return ids, torch.softmax(normal(g, b, K, dtype=F32), 1)


@pytest.mark.parametrize("post,finalize", [(True, True), (False, False)])
@pytest.mark.parametrize("E,K,H,I,group", [(12, 3, 512, 256, 128), (5, 2, 328, 136, 32)])
def test_layer(E, K, H, I, group, post, finalize):
    g = gen(E)
    m = make(g, 40, E, K, H, I, group, post, finalize)
    for b in (40, 1, 7):
        x, residual = normal(g, b, H), normal(g, b, H)
        token = torch.rand(b, generator=g, device="cuda") if post else None
        ids, w = routes(g, b, K, E)
        h, v, want = plain(m, x, residual, token, ids, w)
        out, res = torch.full((b, H), 77.0, dtype=BF, device="cuda"), residual.clone()
        got, rows = m.norm(x, res, token_gate=token)
        assert got is res
        assert ((res.to(F64) - h).abs() <= 2.0 ** -8 * h.abs() + 1e-4).all()
        assert ((rows.to(F64) - v).norm(dim=1) <= 2.0 ** -9 * v.norm(dim=1)).all()
        assert m.experts(ids, w, out) is out
        off = (out.to(F64) - want).norm(dim=1)
        assert (off <= 5e-3 * want.norm(dim=1) + 1e-6).all(), (off / want.norm(dim=1)).max()
    assert mt.moe_tail_take_device_error() == 0


def test_layer_without_tokens_and_without_local_experts():
    g = gen(3)
    for finalize in (True, False):
        m = make(g, 6, 8, 2, 256, 128, 64, True, finalize)
        none = torch.empty((0, 256), dtype=BF, device="cuda")
        m.norm(none, none.clone())
        m.experts(torch.empty((0, 2), dtype=I32, device="cuda"), torch.empty((0, 2), device="cuda"), none.clone())
        x, out = normal(g, 6, 256), torch.full((6, 256), 77.0, dtype=BF, device="cuda")
        m.norm(x, x.clone())
        m.experts(torch.full((6, 2), -1, dtype=I32, device="cuda"), torch.ones((6, 2), device="cuda"), out)
        assert (out == 0).all()
        with pytest.raises(ValueError, match="norm"):
            m.experts(torch.zeros((5, 2), dtype=I32, device="cuda"), torch.ones((5, 2), device="cuda"), out[:5])
    assert mt.moe_tail_take_device_error() == 0


def test_layer_in_a_graph():
    g = gen(4)
    b, E, K, H, I = 24, 16, 4, 256, 128
    m = make(g, b, E, K, H, I, 32, True, True)
    x, residual, res, out = (normal(g, b, H) for _ in range(4))
    ids, w = routes(g, b, K, E)

    def step():
        m.norm(x, residual, residual_out=res)
        m.experts(ids, w, out)

    step()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x0, ids0 = x.clone(), ids.clone()
    x.copy_(normal(g, b, H))
    ids.copy_(routes(g, b, K, E)[0])
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


@pytest.mark.parametrize("finalize", [True, False])
def test_a_token_with_one_expert_several_times(finalize):
    g = gen(5)
    b, E, K, H, I = 9, 4, 3, 264, 136
    m = make(g, b, E, K, H, I, 64, True, finalize)
    x, residual, out = normal(g, b, H), normal(g, b, H), torch.empty((b, H), dtype=BF, device="cuda")
    ids, w = routes(g, b, K, E, local=1.0)
    ids[0], ids[1, 1], ids[2], ids[3, 0] = 2, ids[1, 0], E, 10 ** 9  # all one, two alike, none here
    _, _, want = plain(m, x, residual, None, ids, w)
    m.norm(x, residual)
    m.experts(ids, w, out)
    off = (out.to(F64) - want).norm(dim=1)
    assert (off <= 5e-3 * want.norm(dim=1) + 1e-6).all()
    assert mt.moe_tail_take_device_error() == 0
