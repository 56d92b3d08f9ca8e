"""The calls around the tail (8-bit rows, routes, the 8-bit product) refuse bad arguments on the host, before any CUDA
call: through the C ABI with fake device addresses (nothing is launched), and through the binding with CPU tensors."""
import pytest
import torch

import moe_decode_tail_gb300 as mt
from moe_decode_tail_gb300 import build as cuda_build

EINVAL, OK = 1, 0
FAKE = 0x7F0000000000
GB = 1 << 30
BF, I8, I32, F32, E4 = torch.bfloat16, torch.int8, torch.int32, torch.float32, torch.float8_e4m3fn

# fake device addresses: only where no GPU is visible, so that a missing check can never launch on them
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return mt.lib()


def p(i, off=0):
    """The i-th of a row of fake buffers, 64 GB apart."""
    return FAKE + 64 * GB * i + off


CALLS = {
    "moe_tail_norm_quant": dict(x=p(0), residual=p(1), gamma=p(2), gain_center=1.0, eps=1e-6, b=4, H=256, q_dtype=0,
                                group=0, residual_out=p(3), y=p(4), q=p(5), scale=p(6), stream=None),
    "moe_tail_silu_quant": dict(gate_up=p(0), used=p(1), rows=4, I=256, q_dtype=0, group=0, q=p(2), scale=p(3),
                                stream=None),
    "moe_tail_sort_routes": dict(ids=p(0), b=4, K=2, E=8, offsets=p(1), idx=p(2), source=p(3), ws=p(4), wsb=4096,
                                 stream=None),
    "moe_tail_dispatch_rows": dict(x=p(0), scale=p(1), idx=p(2), b=4, K=2, H=256, elem=1, num_rows=8, rows=p(3),
                                   row_scale=p(4), stream=None),
    "moe_tail_combine_rows": dict(rows=p(0), num_rows=8, idx=p(1), w=p(2), w_dtype=0, b=4, K=2, H=256, out=p(3),
                                  stream=None),
    "moe_tail_combine_grad": dict(d_out=p(0), rows=p(1), num_rows=8, idx=p(2), w=p(3), w_dtype=0, b=4, K=2, H=256,
                                  d_rows=p(4), d_w=p(5), stream=None),
    "moe_tail_expert_product": dict(x=p(0), x_scale=p(1), w=p(2), w_scale=p(3), offsets=p(4), rows=8, E=4, N=64, D=128,
                                    out=p(5), ws=p(6), wsb=1 << 32, stream=None),
}
MAX_ROWS = 1 << 22
BAD = {
    "moe_tail_norm_quant": [
        dict(x=None), dict(gamma=None), dict(q=None), dict(scale=None), dict(b=-1), dict(b=MAX_ROWS + 1), dict(H=0),
        dict(H=12), dict(H=32776), dict(q_dtype=2), dict(q_dtype=-1), dict(group=64), dict(group=-128), dict(x=p(0, 2)),
        dict(residual=p(1, 8)), dict(gamma=p(2, 8)), dict(q=p(5, 8)), dict(scale=p(6, 2)), dict(residual_out=p(0, 16)),
        dict(residual_out=p(1, 16)), dict(y=p(0)), dict(y=p(1)), dict(q=p(0)), dict(scale=p(2)), dict(y=p(3)),
        dict(scale=p(5)), dict(residual_out=p(2))],
    "moe_tail_silu_quant": [
        dict(gate_up=None), dict(q=None), dict(scale=None), dict(rows=-1), dict(rows=MAX_ROWS + 1), dict(I=4),
        dict(I=32776), dict(q_dtype=3), dict(group=1), dict(gate_up=p(0, 8)), dict(used=p(1, 1)), dict(q=p(0)),
        dict(scale=p(2)), dict(scale=p(1)), dict(q=p(0, 4 * 4 * 256 - 16))],
    "moe_tail_sort_routes": [
        dict(ids=None), dict(offsets=None), dict(idx=None), dict(source=None), dict(ws=None), dict(wsb=0), dict(b=-1),
        dict(K=0), dict(K=33), dict(E=0), dict(E=1025), dict(b=(1 << 20) + 1), dict(ids=p(0, 2)), dict(offsets=p(1, 1)),
        dict(idx=p(0)), dict(source=p(2)), dict(offsets=p(3)), dict(ws=p(0)), dict(ws=p(4, 8)), dict(wsb=31)],
    "moe_tail_dispatch_rows": [
        dict(x=None), dict(idx=None), dict(rows=None), dict(scale=None), dict(row_scale=None), dict(b=-1), dict(K=0),
        dict(K=33), dict(H=4), dict(H=32776), dict(elem=4), dict(elem=0), dict(num_rows=-1), dict(num_rows=MAX_ROWS + 1),
        dict(x=p(0, 8)), dict(rows=p(3, 8)), dict(rows=p(0)), dict(row_scale=p(1)), dict(row_scale=p(3)),
        dict(b=MAX_ROWS)],
    "moe_tail_combine_rows": [
        dict(rows=None), dict(idx=None), dict(out=None), dict(b=-1), dict(K=0), dict(K=33), dict(H=20), dict(H=32776),
        dict(w_dtype=2), dict(num_rows=-1), dict(num_rows=MAX_ROWS + 1), dict(rows=p(0, 8)), dict(w=p(2, 2)),
        dict(out=p(0)), dict(out=p(2)), dict(out=p(1)), dict(out=p(3, 4))],
    "moe_tail_combine_grad": [
        dict(d_out=None), dict(rows=None), dict(idx=None), dict(w=None), dict(d_rows=None), dict(d_w=None), dict(b=-1),
        dict(K=0), dict(H=20), dict(w_dtype=-1), dict(num_rows=MAX_ROWS + 1), dict(d_rows=p(1)), dict(d_rows=p(0)),
        dict(d_w=p(3)), dict(d_w=p(4)), dict(d_rows=p(4, 8)), dict(d_w=p(5, 2))],
    "moe_tail_expert_product": [
        dict(x=None), dict(x_scale=None), dict(w=None), dict(w_scale=None), dict(offsets=None), dict(out=None),
        dict(ws=None), dict(wsb=0), dict(rows=-1), dict(rows=MAX_ROWS + 1), dict(E=0), dict(E=1025), dict(N=12), dict(N=0),
        dict(N=(1 << 20) + 8), dict(D=8), dict(D=24), dict(D=65552), dict(x=p(0, 8)), dict(w=p(2, 8)),
        dict(w_scale=p(3, 2)), dict(offsets=p(4, 2)), dict(out=p(5, 8)), dict(ws=p(6, 16)), dict(out=p(0)), dict(out=p(2)),
        dict(out=p(4)), dict(ws=p(1)), dict(ws=p(5))],
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
def test_optional_arguments_may_be_null(lib):
    for name, more in (("moe_tail_norm_quant", dict(residual=None)), ("moe_tail_norm_quant", dict(residual_out=None, y=None)),
                       ("moe_tail_norm_quant", dict(residual_out=p(0))), ("moe_tail_norm_quant", dict(residual_out=p(1))),
                       ("moe_tail_norm_quant", dict(group=128, q_dtype=1)), ("moe_tail_silu_quant", dict(used=None)),
                       ("moe_tail_dispatch_rows", dict(scale=None, row_scale=None)),
                       ("moe_tail_combine_rows", dict(w=None)), ("moe_tail_combine_rows", dict(w=p(2, 2), w_dtype=1)),
                       ("moe_tail_expert_product", dict(offsets=None, E=1))):
        assert getattr(lib, name)(*{**CALLS[name], **more}.values()) in (2, 3), (name, more)


def test_nothing_to_do_is_no_call(lib):
    nulls = {"moe_tail_norm_quant": dict(b=0), "moe_tail_silu_quant": dict(rows=0), "moe_tail_dispatch_rows": dict(b=0),
             "moe_tail_combine_rows": dict(b=0), "moe_tail_combine_grad": dict(b=0), "moe_tail_expert_product": dict(rows=0)}
    for name, none in nulls.items():
        args = {k: (None if isinstance(v, int) and v >= FAKE else v) for k, v in CALLS[name].items()}
        if name == "moe_tail_expert_product":
            none = dict(none, E=1)
        assert getattr(lib, name)(*{**args, **none}.values()) == OK, name
    assert lib.moe_tail_dispatch_rows(*{**CALLS["moe_tail_dispatch_rows"], "num_rows": 0}.values()) == OK


def test_workspace_sizes(lib):
    assert lib.moe_tail_sort_workspace_bytes(64, 8, 128) >= 4 * 128
    assert lib.moe_tail_sort_workspace_bytes(8192, 8, 128) >= 4 * 128 * 16
    assert lib.moe_tail_sort_workspace_bytes(-1, 8, 128) == lib.moe_tail_sort_workspace_bytes(1, 8, 1025) == 0
    assert lib.moe_tail_expert_product_workspace_bytes(512, 128, 2048, 4096) > 0
    assert lib.moe_tail_expert_product_workspace_bytes(512, 128, 2048, 4100) == 0


# ---- the binding ---------------------------------------------------------------------------------------------------


def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


def good():
    b, K, H, E, R, N, D = 3, 2, 256, 4, 6, 64, 128
    return {
        "moe_tail_norm_quant": ([t(BF, b, H), t(BF, b, H), t(BF, H), t(I8, b, H), t(F32, b)],
                                dict(residual_out=t(BF, b, H), y=t(BF, b, H))),
        "moe_tail_silu_quant": ([t(BF, R, 2 * H), t(E4, R, H), t(F32, R, 2)], dict(group=128, used_rows=t(I32, 1))),
        "moe_tail_sort_routes": ([t(I32, b, K), t(I32, E + 1), t(I32, b, K), t(I32, b * K), t(torch.uint8, 4096)], {}),
        "moe_tail_dispatch_rows": ([t(I8, b, H), t(I32, b, K), t(I8, R, H)], dict(scale=t(F32, b), row_scale=t(F32, R))),
        "moe_tail_combine_rows": ([t(BF, R, H), t(I32, b, K), t(F32, b, K), t(BF, b, H)], {}),
        "moe_tail_combine_grad": ([t(BF, b, H), t(BF, R, H), t(I32, b, K), t(BF, b, K), t(BF, R, H), t(F32, b, K)], {}),
        "moe_tail_expert_product": ([t(I8, R, D), t(F32, R), t(I8, E, N, D), t(F32, E, N), t(BF, R, N),
                                     t(torch.uint8, 4096)], dict(expert_offsets=t(I32, E + 1))),
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
        if not isinstance(old, torch.Tensor) or old.dtype == torch.uint8:
            continue
        for new in (old.to(torch.float64), torch.zeros([*old.shape, 2], dtype=old.dtype),
                    torch.zeros([s + 1 for s in old.shape], dtype=old.dtype)):
            if name == "moe_tail_sort_routes" and where == 1 and new.dim() == 1 and new.dtype == I32:
                continue  # another number of experts
            a, k = list(args), dict(more)
            if isinstance(where, int):
                a[where] = new
            else:
                k[where] = new
            with pytest.raises(ValueError) as e:
                getattr(mt, name)(*a, **k)
            assert "contiguous CUDA tensors" not in str(e.value), (name, where, tuple(new.shape), new.dtype)


def test_binding_refuses_half_of_a_pair_and_unknown_groups():
    args, more = good()["moe_tail_dispatch_rows"]
    with pytest.raises(ValueError, match="together"):
        mt.moe_tail_dispatch_rows(*args, scale=more["scale"])
    args, more = good()["moe_tail_norm_quant"]
    with pytest.raises(ValueError, match="group"):
        mt.moe_tail_norm_quant(*args, group=64)
