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
