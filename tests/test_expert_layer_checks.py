"""ExpertLayerI8 refuses what it would get wrong: routes of other tokens than the last norm's, sizes that its calls take no
part of."""
import pytest
import torch

from moe_decode_tail_gb300 import build as cuda_build
from moe_decode_tail_gb300.expert_layer import ExpertLayerI8

BF, I8, I32, F32 = torch.bfloat16, torch.int8, torch.int32, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()


def layer(E=4, H=64, I=32, tokens=8, K=2, device="cpu", **more):
    w_gate_up = torch.ones((E, 2 * I, H), dtype=I8, device=device)
    w_down = torch.ones((E, H, I), dtype=I8, device=device)
    return ExpertLayerI8(torch.zeros(H, dtype=BF, device=device), w_gate_up, torch.full((E, 2 * I), 0.01, device=device),
                         w_down, torch.full((E, H), 0.01, device=device), max_tokens=tokens, top_k=K, **more)


def routes(b, K=2, device="cpu"):
    return (torch.zeros((b, K), dtype=I32, device=device), torch.full((b, K), 0.5, device=device),
            torch.zeros((b, 64), dtype=BF, device=device))


def test_experts_before_any_norm():
    with pytest.raises(ValueError, match="norm"):
        layer().experts(*routes(3))


@pytest.mark.gpu
@pytest.mark.parametrize("b", [0, 1, 4, 6, 8])
def test_experts_of_other_tokens_than_the_norm(b):
    m = layer(device="cuda")
    x = torch.ones((5, 64), dtype=BF, device="cuda")
    m.norm(x, None)
    with pytest.raises(ValueError, match="norm"):
        m.experts(*routes(b, device="cuda"))
    m.experts(*routes(5, device="cuda"))  # and those it has, any number of times
    m.experts(*routes(5, device="cuda"))
    m.norm(torch.ones((b, 64), dtype=BF, device="cuda"), None)
    m.experts(*routes(b, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_refused_norm_leaves_no_rows_to_use():
    m = layer(device="cuda")
    m.norm(torch.ones((5, 64), dtype=BF, device="cuda"), None)
    with pytest.raises(ValueError):
        m.norm(torch.ones((3, 64), dtype=F32, device="cuda"), None)
    for b in (3, 5):
        with pytest.raises(ValueError, match="norm"):
            m.experts(*routes(b, device="cuda"))


# ---- sizes ---------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("sizes", [dict(I=24), dict(I=8), dict(H=72), dict(H=520), dict(H=8), dict(K=0), dict(K=33),
                                   dict(tokens=-1), dict(E=1025, H=16, I=16), dict(H=32784, I=16, E=1), dict(I=32784, H=16, E=1),
                                   dict(tokens=(1 << 20) + 1)])
def test_sizes_that_a_call_would_refuse(sizes):
    with pytest.raises(ValueError):
        layer(**sizes)


def test_tokens_beyond_the_finalize_call():
    gamma = torch.zeros(16, dtype=BF)
    sizes = dict(E=1, H=16, I=16, K=1)
    assert layer(tokens=65535, finalize_gamma=gamma, **sizes).max_tokens == 65535
    assert layer(tokens=65536, **sizes).max_tokens == 65536  # the plain weighted sum takes them
    with pytest.raises(ValueError, match="65535"):
        layer(tokens=65536, finalize_gamma=gamma, **sizes)


def test_operands_of_another_type_or_shape():
    E, H, I = 4, 64, 32
    good = dict(gamma=torch.zeros(H, dtype=BF), w_gate_up=torch.ones((E, 2 * I, H), dtype=I8), s_gate_up=torch.ones((E, 2 * I)),
                w_down=torch.ones((E, H, I), dtype=I8), s_down=torch.ones((E, H)), finalize_gamma=torch.zeros(H, dtype=BF))
    ExpertLayerI8(**good, max_tokens=2, top_k=2)
    for name, old in good.items():
        for new in (old.to(torch.float64), torch.zeros([s + 16 for s in old.shape], dtype=old.dtype)):
            with pytest.raises(ValueError):
                ExpertLayerI8(**{**good, name: new}, max_tokens=2, top_k=2)


@pytest.mark.gpu
@pytest.mark.parametrize("E,H,I,K", [(1, 16, 16, 1), (1024, 32, 16, 2), (2, 32768, 16, 1), (2, 16, 32768, 2), (3, 48, 80, 32)])
def test_sizes_at_the_limits_run(E, H, I, K):
    for finalize in (None, torch.zeros(H, dtype=BF, device="cuda")):
        m = layer(E=E, H=H, I=I, tokens=3, K=K, device="cuda", finalize_gamma=finalize)
        x, out = torch.ones((3, H), dtype=BF, device="cuda"), torch.empty((3, H), dtype=BF, device="cuda")
        m.norm(x, None)
        ids = (torch.arange(3 * K, device="cuda") % E).to(I32).view(3, K)
        m.experts(ids, torch.full((3, K), 1.0 / K, device="cuda"), out)
        torch.cuda.synchronize()
        assert out.isfinite().all()
