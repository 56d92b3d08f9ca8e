"""The 4-bit products and the norms around a block refuse bad arguments on the host, before any CUDA call: through the C ABI
with fake device addresses (nothing is launched), and through the binding with CPU tensors."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300 import build as cuda_build
from moe_decode_tail_gb300.expert_layer import ExpertLayerI4, pack_int4, quantise_groups

EINVAL, OK = 1, 0
FAKE = 0x7F0000000000
GB = 1 << 30
BF, U8, I32, F32, E4 = torch.bfloat16, torch.uint8, torch.int32, torch.float32, torch.float8_e4m3fn

# fake device addresses: only where no GPU is visible, so that a missing check can never launch on them
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return mt.lib()


def p(i, off=0):
    """The i-th of a row of fake buffers, 64 GB apart."""
    return FAKE + 64 * GB * i + off


PRODUCT = dict(x=p(0), w=p(1), gs=p(2), cs=p(3), offsets=p(4), rows=8, E=4, N=64, D=256, group=64, out=p(5), stream=None)
CALLS = {
    "moe_tail_block_norm": dict(x=p(0), residual=p(1), post=p(2), pre=p(3), token=p(4), channel=p(5), scale=1.0, center=1.0,
                                eps=1e-6, b=4, H=256, out=p(6), y=p(7), rstd=p(8), stream=None),
    "moe_tail_block_norm_grad": dict(d_y=p(0), d_out=p(1), x=p(2), residual=p(3), post=p(4), pre=p(5), token=p(6),
                                     channel=p(7), rstd=p(8), scale=1.0, center=1.0, b=4, H=256, d_x=p(9), d_res=p(10),
                                     d_post=p(11), d_pre=p(12), d_token=p(13), d_channel=p(14), ws=p(15), wsb=1 << 30,
                                     stream=None),
    "moe_tail_expert_product_i4": PRODUCT,
    "moe_tail_gated_product_i4": PRODUCT,
}
MAX_ROWS = 1 << 22
BAD_PRODUCT = [
    dict(x=None), dict(w=None), dict(gs=None), dict(cs=None), dict(offsets=None), dict(out=None), dict(rows=-1),
    dict(rows=MAX_ROWS + 1), dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(N=(1 << 20) + 8), dict(D=0), dict(D=12),
    dict(D=65544), dict(group=0), dict(group=16), dict(group=256), dict(group=-32), dict(x=p(0, 8)), dict(w=p(1, 8)),
    dict(gs=p(2, 2)), dict(cs=p(3, 2)), dict(offsets=p(4, 2)), dict(out=p(5, 8)), dict(out=p(0)), dict(out=p(1)),
    dict(out=p(2)), dict(out=p(3)), dict(out=p(4)), dict(out=p(0, 16 * 255))]
BAD = {
    "moe_tail_block_norm": [
        dict(x=None), dict(residual=None), dict(pre=None), dict(out=None), dict(y=None), dict(b=-1), dict(b=MAX_ROWS + 1),
        dict(H=0), dict(H=12), dict(H=32776), dict(x=p(0, 8)), dict(residual=p(1, 8)), dict(post=p(2, 8)), dict(pre=p(3, 8)),
        dict(token=p(4, 2)), dict(channel=p(5, 8)), dict(out=p(6, 8)), dict(y=p(7, 8)), dict(rstd=p(8, 4)), dict(out=p(0, 16)),
        dict(out=p(1, 16)), dict(out=p(2)), dict(y=p(0)), dict(y=p(1)), dict(y=p(6)), dict(rstd=p(4)), dict(rstd=p(6)),
        dict(out=p(0), y=p(0))],
    "moe_tail_block_norm_grad": [
        dict(d_y=None), dict(x=None), dict(residual=None), dict(pre=None), dict(rstd=None), dict(d_x=None), dict(d_res=None),
        dict(ws=None), dict(wsb=0), dict(b=-1), dict(b=MAX_ROWS + 1), dict(H=4), dict(H=36), dict(H=32776), dict(post=None),
        dict(token=None), dict(channel=None), dict(d_y=p(0, 8)), dict(rstd=p(8, 4)), dict(d_post=p(11, 8)),
        dict(d_pre=p(12, 4)), dict(d_token=p(13, 2)), dict(d_channel=p(14, 8)), dict(ws=p(15, 8)), dict(d_x=p(1)),
        dict(d_x=p(2)), dict(d_res=p(0)), dict(d_res=p(3)), dict(d_x=p(0, 16)), dict(d_res=p(1, 16)), dict(d_res=p(9)),
        dict(d_post=p(4)), dict(d_pre=p(11)), dict(d_token=p(6)), dict(d_channel=p(8)), dict(ws=p(9)), dict(ws=p(0))],
    "moe_tail_expert_product_i4": BAD_PRODUCT,
    "moe_tail_gated_product_i4": BAD_PRODUCT,
}
REFUSALS = [(name, bad) for name, many in BAD.items() for bad in many]


@host_only
@pytest.mark.parametrize("name,bad", REFUSALS, ids=[f"{n[9:]}-{b}" for n, b in REFUSALS])
def test_refuses(lib, name, bad):
    assert getattr(lib, name)(*{**CALLS[name], **bad}.values()) == EINVAL


@host_only
@pytest.mark.parametrize("name", CALLS)
def test_defaults_pass_every_check(lib, name):
    # each refusal changes one argument of these: they get as far as the first CUDA call
    assert getattr(lib, name)(*CALLS[name].values()) in (2, 3)


@host_only
def test_optional_arguments_may_be_null_and_outputs_in_place(lib):
    grad = "moe_tail_block_norm_grad"
    for name, more in (("moe_tail_block_norm", dict(post=None)), ("moe_tail_block_norm", dict(token=None, channel=None)),
                       ("moe_tail_block_norm", dict(rstd=None)), ("moe_tail_block_norm", dict(out=p(0))),
                       ("moe_tail_block_norm", dict(out=p(1))), (grad, dict(d_out=None)), (grad, dict(post=None, d_post=None)),
                       (grad, dict(token=None, d_token=None)), (grad, dict(channel=None, d_channel=None)),
                       (grad, dict(d_post=None, d_pre=None, d_token=None, d_channel=None)), (grad, dict(d_x=p(0))),
                       (grad, dict(d_res=p(1))), (grad, dict(d_x=p(0), d_res=p(1))),
                       ("moe_tail_expert_product_i4", dict(offsets=None, E=1)),
                       ("moe_tail_gated_product_i4", dict(offsets=None, E=1, D=65536, N=1 << 20, rows=1 << 22, gs=p(2), out=p(40)))):
        assert getattr(lib, name)(*{**CALLS[name], **more}.values()) in (2, 3), (name, more)


def test_nothing_to_do_is_no_call(lib):
    for name, none in (("moe_tail_block_norm", dict(b=0)), ("moe_tail_expert_product_i4", dict(rows=0, E=1)),
                       ("moe_tail_gated_product_i4", dict(rows=0, E=1))):
        args = {k: (None if isinstance(v, int) and v >= FAKE else v) for k, v in CALLS[name].items()}
        assert getattr(lib, name)(*{**args, **none}.values()) == OK, name


def test_a_workspace_serves_fewer_rows(lib):
    for H in (8, 256, 264, 2048, 4096, 4104, 8200, 32768):
        sizes = [lib.moe_tail_block_norm_grad_workspace_bytes(b, H) for b in (0, 1, 2, 15, 16, 17, 160, 161, 2560, 2561, 10 ** 6)]
        assert sizes == sorted(sizes) and sizes[0] >= 12 * H
    for b, H in ((-1, 256), (MAX_ROWS + 1, 256), (4, 12), (4, 32776), (4, 0)):
        assert lib.moe_tail_block_norm_grad_workspace_bytes(b, H) == 0


# ---- the binding ---------------------------------------------------------------------------------------------------


def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


def good():
    b, H, E, R, N, D = 3, 256, 4, 6, 64, 200
    rows, vector = lambda: t(BF, b, H), lambda: t(BF, H)  # noqa: E731
    weight = lambda n: [t(BF, R, D), t(U8, E, n, 128), t(E4, E, n, 4), t(F32, E, n), t(BF, R, N)]  # noqa: E731
    more = dict(group=64, expert_offsets=t(I32, E + 1))
    return {
        "moe_tail_block_norm": ([rows(), rows(), vector(), vector(), rows(), rows()],
                                dict(token_gate=t(F32, b), channel_gate=vector(), rstd=t(F32, b, 2))),
        "moe_tail_block_norm_grad": ([rows(), rows(), rows(), rows(), vector(), vector(), t(F32, b, 2), rows(), rows(),
                                      t(U8, 1 << 16)],
                                     dict(token_gate=t(F32, b), channel_gate=vector(), d_post_gamma=t(F32, H),
                                          d_pre_gamma=t(F32, H), d_token_gate=t(F32, b), d_channel_gate=t(F32, H))),
        "moe_tail_expert_product_i4": (weight(N), more),
        "moe_tail_gated_product_i4": (weight(2 * N), more),
    }


@pytest.mark.parametrize("name", CALLS)
def test_binding_accepts_its_shapes_up_to_the_cuda_check(name):
    args, more = good()[name]
    with pytest.raises(ValueError, match="contiguous CUDA tensors"):
        getattr(mt, name)(*args, **more)


@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses_every_tensor_of_another_type_or_shape(name):
    args, more = good()[name]
    for where in list(range(len(args))) + list(more):
        old = args[where] if isinstance(where, int) else more[where]
        if not isinstance(old, torch.Tensor) or (name.endswith("grad") and where == 9):  # the workspace
            continue
        for new in (old.to(torch.float64), torch.zeros([*old.shape, 2], dtype=old.dtype),
                    torch.zeros([s + 1 for s in old.shape], dtype=old.dtype)):
            a, k = list(args), dict(more)
            if isinstance(where, int):
                a[where] = new
            else:
                k[where] = new
            with pytest.raises(ValueError) as e:
                getattr(mt, name)(*a, **k)
            assert "contiguous CUDA tensors" not in str(e.value), (name, where, tuple(new.shape), new.dtype)


def test_binding_refuses_unknown_groups_odd_channels_and_gradients_of_nothing():
    args, more = good()["moe_tail_expert_product_i4"]
    with pytest.raises(ValueError, match="group"):
        mt.moe_tail_expert_product_i4(*args, **{**more, "group": 48})
    args, more = good()["moe_tail_gated_product_i4"]
    args[1], args[2], args[3] = t(U8, 4, 129, 128), t(E4, 4, 129, 4), t(F32, 4, 129)
    with pytest.raises(ValueError, match="even"):
        mt.moe_tail_gated_product_i4(*args, **more)
    args, more = good()["moe_tail_block_norm_grad"]
    for name in ("token_gate", "channel_gate"):
        with pytest.raises(ValueError, match="d_" + name):
            mt.moe_tail_block_norm_grad(*args, **{**more, name: None})
    args[4] = None
    with pytest.raises(ValueError, match="d_post_gamma"):
        mt.moe_tail_block_norm_grad(*args, **more)


# ---- the layout and the layer ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("D", [8, 32, 120, 128, 136, 520])
def test_layout(D):
    # the header's definition, a column at a time
    q = torch.randint(-8, 8, (2, 3, D), generator=torch.Generator().manual_seed(D)).to(torch.int8)
    w = pack_int4(q)
    assert w.shape == (2, 3, 64 * -(-D // 128)) and w.dtype == U8 and w.is_contiguous()
    for k in range(D):
        block, column = divmod(k, 128)
        i, rest = divmod(column, 32)
        tt, c = divmod(rest, 8)
        nibble = c // 2 if c % 2 == 0 else 4 + c // 2
        byte = w[..., 64 * block + 4 * (4 * tt + i) + nibble // 2].to(I32)
        assert torch.equal((byte >> (4 * (nibble % 2))) & 15, q[..., k].to(I32) + 8)


def make(E=4, H=264, I=40, tokens=8, K=2, group=32, **more):
    g = torch.Generator().manual_seed(0)
    return ExpertLayerI4(torch.zeros(H, dtype=BF), quantise_groups(torch.randn((E, 2 * I, H), generator=g), group),
                         quantise_groups(torch.randn((E, H, I), generator=g), group), max_tokens=tokens, top_k=K, group=group,
                         **more)


def test_layer_refuses_sizes_and_operands(lib):
    make()
    for sizes in (dict(I=12), dict(H=60), dict(K=0), dict(K=33), dict(tokens=-1), dict(E=1025, H=8, I=8),
                  dict(H=32776, I=8, E=1), dict(I=32776, H=8, E=1), dict(tokens=(1 << 20) + 1)):
        with pytest.raises(ValueError):
            make(**sizes)
    with pytest.raises(ValueError, match="65535"):
        make(tokens=65536, E=1, H=8, I=8, K=1, finalize_gamma=torch.zeros(8, dtype=BF))
    m = make(post_gamma=torch.zeros(264, dtype=BF))
    good = dict(gamma=m.gamma, gate_up=m.gate_up, down=m.down, group=32, max_tokens=2, top_k=2, post_gamma=m.post_gamma)
    for bad in (dict(group=64, down=m.gate_up), dict(group=48), dict(gamma=m.gamma.float()), dict(post_gamma=torch.zeros(72, dtype=BF)),
                dict(gate_up=m.down), dict(down=(m.down[0], m.down[1], m.down[2].double())),
                dict(gate_up=(m.gate_up[0].to(I32), *m.gate_up[1:]))):
        with pytest.raises(ValueError):
            ExpertLayerI4(**{**good, **bad})
    with pytest.raises(ValueError, match="norm"):
        m.experts(torch.zeros((3, 2), dtype=I32), torch.ones((3, 2)), torch.zeros((3, 264), dtype=BF))
    with pytest.raises(ValueError, match="tokens"):
        m.norm(torch.zeros((9, 264), dtype=BF), torch.zeros((9, 264), dtype=BF))
    with pytest.raises(ValueError, match="group"):
        quantise_groups(torch.zeros((8, 64)), 100)
