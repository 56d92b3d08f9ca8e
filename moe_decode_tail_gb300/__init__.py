"""GB300-native MoE decode tail: thin Python binding of libmoetail.so.

Every function here only marshals torch CUDA tensors into the C ABI of
``include/moe_tail.h`` (same names, sizes read from tensor shapes); all of the
tail's arithmetic runs in the library's CUDA kernels.  There is no CPU path:
if the library is missing or a call is refused, these functions raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB

__all__ = [
    "MoeTailError", "lib", "moe_tail_ep_finalize", "moe_tail_tp_finalize", "moe_tail_latent_up",
    "moe_shared_expert", "moe_tail_workspace_bytes", "moe_tail_status_str", "moe_tail_take_device_error",
    "moe_tail_latent_up_noalloc", "NOALLOC_SCRATCH_BYTES", "moe_tail_selftest_wait_timeout",
    "moe_tail_latent_norm", "moe_tail_up_project", "WEIGHTS_STATIC", "INPUTS_READY",
    "moe_shared_gate_up", "moe_shared_down", "moe_tail_latent_up_flags", "moe_tail_ep_finalize_flags",
    "moe_tail_tp_finalize_flags", "moe_tail_set_kernel_form", "kernel_form", "FORM_EP", "FORM_TP", "FORM_LATENT",
    "FORM_LATENT_ONE_KERNEL", "moe_tail_set_stage_wait_limit", "moe_tail_up_project_shared_down",
    "moe_shared_down_persistent", "moe_tail_norm_quant", "moe_tail_silu_quant", "moe_tail_sort_routes",
    "moe_tail_sort_workspace_bytes", "moe_tail_dispatch_rows", "moe_tail_combine_rows", "moe_tail_combine_grad",
    "moe_tail_expert_product", "moe_tail_expert_product_workspace_bytes", "moe_tail_block_norm",
    "moe_tail_block_norm_grad", "moe_tail_block_norm_grad_workspace_bytes", "moe_tail_expert_product_i4",
    "moe_tail_gated_product_i4", "moe_tail_product_i4_tile_rows",
]

OK, EINVAL, ECUDA, ENOTSUP = 0, 1, 2, 3
NOALLOC_SCRATCH_BYTES = 1 << 20  # MOE_TAIL_NOALLOC_SCRATCH_BYTES
W_FP32, W_BF16 = 0, 1
Q_DTYPES = {torch.int8: 0, torch.float8_e4m3fn: 1}  # MOE_TAIL_Q_*: the types of 8-bit rows
I4_GROUPS = (32, 64, 128)  # columns of a group of 4-bit weights
QUANT_GROUP = 128  # columns of a group where a row has several scales
WEIGHTS_STATIC = 1  # MOE_TAIL_WEIGHTS_STATIC
INPUTS_READY = 2  # MOE_TAIL_INPUTS_READY
FORM_EP, FORM_TP, FORM_LATENT = 0, 1, 2  # MOE_TAIL_FORM_*: the calls whose kernel form can be pinned
FORM_LATENT_ONE_KERNEL = 1  # MOE_TAIL_FORM_LATENT_ONE_KERNEL


class MoeTailError(RuntimeError):
    def __init__(self, name: str, status: int):
        super().__init__(f"{name}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built).  The
    MOE_TAIL_LIBRARY environment variable selects another build of it (the
    trace build, whose records moe_decode_tail_gb300.trace reads) before the first call."""
    global _lib
    if _lib is None:
        path = os.environ.get("MOE_TAIL_LIBRARY", LIB)
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with moe_decode_tail_gb300.build.build()")
        L = ctypes.CDLL(path)
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        fin = [P, i64, P, P, i32, P, f32, f32, i32, i32, i32, i32, i32, P, P]
        L.moe_tail_ep_finalize.argtypes = fin
        L.moe_tail_tp_finalize.argtypes = fin
        fin_flags = fin[:-1] + [i32, P]
        L.moe_tail_ep_finalize_flags.argtypes = fin_flags
        L.moe_tail_tp_finalize_flags.argtypes = fin_flags
        L.moe_tail_latent_up.argtypes = [P, P, f32, P, P, i32, i32, i32, i32, i32, P, P, sz, P]
        L.moe_shared_expert.argtypes = [P, P, P, P, i32, i32, i32, P, i32, P, sz, P]
        L.moe_tail_latent_up_noalloc.argtypes = [P, P, f32, P, P, i32, i32, i32, i32, i32, P, P]
        L.moe_tail_selftest_wait_timeout.argtypes = [ctypes.c_uint, P]
        L.moe_tail_latent_norm.argtypes = [P, P, f32, i32, i32, i32, P, i32, P]
        L.moe_tail_up_project.argtypes = [P, P, P, i32, i32, i32, i32, P, i32, P]
        L.moe_tail_latent_up_flags.argtypes = [P, P, f32, P, P, i32, i32, i32, i32, i32, P, P, i32, P]
        L.moe_shared_gate_up.argtypes = [P, P, P, i32, i32, i32, P, i32, P]
        L.moe_shared_down.argtypes = [P, P, i32, i32, i32, P, i32, i32, P]
        L.moe_shared_down_persistent.argtypes = [P, P, i32, i32, i32, P, i32, i32, i32, P]
        L.moe_tail_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_tail_workspace_bytes.restype = sz
        L.moe_tail_status_str.argtypes = [i32]
        L.moe_tail_status_str.restype = ctypes.c_char_p
        L.moe_tail_take_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.moe_tail_set_kernel_form.argtypes = [i32, i32]
        L.moe_tail_set_stage_wait_limit.argtypes = [ctypes.c_ulonglong]
        L.moe_tail_up_project_shared_down.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32, P, P, i32, P]
        L.moe_tail_norm_quant.argtypes = [P, P, P, f32, f32, i32, i32, i32, i32, P, P, P, P, P]
        L.moe_tail_silu_quant.argtypes = [P, P, i32, i32, i32, i32, P, P, P]
        L.moe_tail_sort_routes.argtypes = [P, i32, i32, i32, P, P, P, P, sz, P]
        L.moe_tail_sort_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_tail_sort_workspace_bytes.restype = sz
        L.moe_tail_dispatch_rows.argtypes = [P, P, P, i32, i32, i32, i32, i64, P, P, P]
        L.moe_tail_combine_rows.argtypes = [P, i64, P, P, i32, i32, i32, i32, P, P]
        L.moe_tail_combine_grad.argtypes = [P, P, i64, P, P, i32, i32, i32, i32, P, P, P]
        L.moe_tail_expert_product.argtypes = [P, P, P, P, P, i64, i32, i32, i32, P, P, sz, P]
        L.moe_tail_expert_product_workspace_bytes.argtypes = [i64, i32, i32, i32]
        L.moe_tail_expert_product_workspace_bytes.restype = sz
        L.moe_tail_block_norm.argtypes = [P, P, P, P, P, P, f32, f32, f32, i32, i32, P, P, P, P]
        L.moe_tail_block_norm_grad.argtypes = [P] * 9 + [f32, f32, i32, i32] + [P] * 7 + [sz, P]
        L.moe_tail_block_norm_grad_workspace_bytes.argtypes = [i32, i32]
        L.moe_tail_block_norm_grad_workspace_bytes.restype = sz
        L.moe_tail_expert_product_i4.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i32, P, P]
        L.moe_tail_gated_product_i4.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i32, P, P]
        L.moe_tail_product_i4_tile_rows.argtypes = [i64, i32, i32, i32, i32]
        for name in ("moe_tail_ep_finalize", "moe_tail_tp_finalize", "moe_tail_latent_up", "moe_shared_expert",
                     "moe_tail_norm_quant", "moe_tail_silu_quant", "moe_tail_sort_routes", "moe_tail_dispatch_rows",
                     "moe_tail_combine_rows", "moe_tail_combine_grad", "moe_tail_expert_product",
                     "moe_tail_take_device_error", "moe_tail_latent_up_noalloc", "moe_tail_selftest_wait_timeout",
                     "moe_tail_latent_norm", "moe_tail_up_project", "moe_shared_gate_up", "moe_shared_down",
                     "moe_tail_latent_up_flags", "moe_tail_ep_finalize_flags", "moe_tail_tp_finalize_flags",
                     "moe_tail_set_kernel_form", "moe_tail_set_stage_wait_limit",
                     "moe_tail_up_project_shared_down", "moe_shared_down_persistent", "moe_tail_block_norm",
                     "moe_tail_block_norm_grad", "moe_tail_expert_product_i4", "moe_tail_gated_product_i4",
                     "moe_tail_product_i4_tile_rows"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_tail_status_str(status).decode()


def _check(name: str, status: int) -> None:
    if status != OK:
        raise MoeTailError(name, status)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        try:  # the current stream's handle, without making a Stream object for it
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:  # a torch without these functions, which are not public
            stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _cuda(*ts):
    for t in ts:
        if t is not None and not (t.is_cuda and t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _operands(*operands) -> None:
    """Operands (name, tensor or None, dtype, shape): each of that type and shape, contiguous and on the current device, which
    is where a call launches its kernels.  One look at each where all is well, since the host's time counts in decode."""
    try:
        here = torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):  # a torch without this function, which is not public, or without a GPU
        here = torch.cuda.current_device() if torch.cuda.is_available() else None
    for _, t, dtype, shape in operands:
        if t is not None and not (t.get_device() == here and t.dtype == dtype and t.shape == shape and t.is_contiguous()):
            break
    else:
        return
    for name, t, dtype, shape in operands:
        if t is not None:
            _like(name, t, dtype, shape)
    for name, t, _, _ in operands:
        _cuda(t)
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name} must be on the current device, cuda:{here}, got {t.device}")


def _dims(name: str, t, n: int) -> tuple:
    """The shape of t, which must have n dimensions."""
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(shape)}")
    return shape


def _like(name: str, t, dtype, shape) -> None:
    """t must be dtype with exactly this shape: the C entry points receive only
    a pointer and take the layout from the sizes, so a tensor of another type
    or shape would be read (or written) as if it had this one."""
    if t.dtype == dtype and t.shape == shape:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _finalize_args(kind: str, src, permuted_idx, route_weights, gamma, out) -> tuple:
    """Shapes of a finalize call: src [tp, rows, P] BF16, route weights [b, K]
    FP32 or BF16, permuted_idx int32 [tp, b, K] (EP) or [b, K] (expert-TP),
    gamma BF16 [P], out BF16 [b, P].  Returns (tp, rows, P, b, K)."""
    tp, rows, P = _dims(kind, src, 3)
    b, K = _dims("route_weights", route_weights, 2)
    _like(kind, src, torch.bfloat16, (tp, rows, P))
    _weights(route_weights)
    _like("permuted_idx", permuted_idx, torch.int32, (tp, b, K) if kind == "rows" else (b, K))
    _like("gamma", gamma, torch.bfloat16, (P,))
    _like("out", out, torch.bfloat16, (b, P))
    _cuda(src, permuted_idx, route_weights, gamma, out)
    return tp, rows, P, b, K


def _latent_args(latent, gamma, w_up, shared, out, y) -> tuple:
    """Shapes of a latent-tail call: latent BF16 [tp, b, L], gamma BF16 [L],
    w_up BF16 [H, L], shared BF16 [tp_s, b, H] or None, out BF16 [b, H], y
    BF16 [b, L] or None.  Returns (tp, b, L, H, tp_s)."""
    tp, b, L = _dims("latent", latent, 3)
    H, _ = _dims("w_up", w_up, 2)
    tp_s = 0 if shared is None else _dims("shared", shared, 3)[0]
    _like("latent", latent, torch.bfloat16, (tp, b, L))
    _like("gamma", gamma, torch.bfloat16, (L,))
    _like("w_up", w_up, torch.bfloat16, (H, L))
    if shared is not None:
        _like("shared", shared, torch.bfloat16, (tp_s, b, H))
    _like("out", out, torch.bfloat16, (b, H))
    if y is not None:
        _like("y", y, torch.bfloat16, (b, L))
    _cuda(latent, gamma, w_up, shared, out, y)
    return tp, b, L, H, tp_s


def _weights(w: torch.Tensor) -> int:
    if w.dtype == torch.float32:
        return W_FP32
    if w.dtype == torch.bfloat16:
        return W_BF16
    raise ValueError("route weights must be FP32 or BF16")


def moe_tail_ep_finalize(rows, permuted_idx, route_weights, gamma, out, *, gain_center=1.0, eps=1e-6,
                         weight_before_norm=True, stream=None) -> torch.Tensor:
    """EP finalize into out (BF16 [b, P]); rows BF16 [tp, rows_per_slot, P],
    permuted_idx int32 [tp, b, K], route_weights [b, K], gamma BF16 [P]."""
    tp, rows_per_slot, P, b, K = _finalize_args("rows", rows, permuted_idx, route_weights, gamma, out)
    _check("moe_tail_ep_finalize", lib().moe_tail_ep_finalize(
        _p(rows), rows_per_slot, _p(permuted_idx), _p(route_weights), _weights(route_weights), _p(gamma),
        gain_center, eps, int(bool(weight_before_norm)), b, tp, K, P, _p(out), _stream(stream)))
    return out


def moe_tail_tp_finalize(partials, permuted_idx, route_weights, gamma, out, *, gain_center=1.0, eps=1e-6,
                         weight_before_norm=True, stream=None) -> torch.Tensor:
    """Expert-TP finalize into out (BF16 [b, P]); partials BF16 [tp, num_rows, P],
    permuted_idx int32 [b, K], route_weights [b, K], gamma BF16 [P]."""
    tp, num_rows, P, b, K = _finalize_args("partials", partials, permuted_idx, route_weights, gamma, out)
    _check("moe_tail_tp_finalize", lib().moe_tail_tp_finalize(
        _p(partials), num_rows, _p(permuted_idx), _p(route_weights), _weights(route_weights), _p(gamma),
        gain_center, eps, int(bool(weight_before_norm)), b, tp, K, P, _p(out), _stream(stream)))
    return out


def moe_tail_ep_finalize_flags(rows, permuted_idx, route_weights, gamma, out, *, gain_center=1.0, eps=1e-6,
                               weight_before_norm=True, inputs_ready=False, stream=None) -> torch.Tensor:
    """moe_tail_ep_finalize with the promise inputs_ready: rows, indices, route
    weights and gamma are not written by work still in flight on the stream."""
    tp, rows_per_slot, P, b, K = _finalize_args("rows", rows, permuted_idx, route_weights, gamma, out)
    _check("moe_tail_ep_finalize_flags", lib().moe_tail_ep_finalize_flags(
        _p(rows), rows_per_slot, _p(permuted_idx), _p(route_weights), _weights(route_weights), _p(gamma),
        gain_center, eps, int(bool(weight_before_norm)), b, tp, K, P, _p(out), INPUTS_READY if inputs_ready else 0,
        _stream(stream)))
    return out


def moe_tail_tp_finalize_flags(partials, permuted_idx, route_weights, gamma, out, *, gain_center=1.0, eps=1e-6,
                               weight_before_norm=True, inputs_ready=False, stream=None) -> torch.Tensor:
    """moe_tail_tp_finalize with the promise inputs_ready: partials, indices,
    route weights and gamma are not written by work still in flight on the stream."""
    tp, num_rows, P, b, K = _finalize_args("partials", partials, permuted_idx, route_weights, gamma, out)
    _check("moe_tail_tp_finalize_flags", lib().moe_tail_tp_finalize_flags(
        _p(partials), num_rows, _p(permuted_idx), _p(route_weights), _weights(route_weights), _p(gamma),
        gain_center, eps, int(bool(weight_before_norm)), b, tp, K, P, _p(out), INPUTS_READY if inputs_ready else 0,
        _stream(stream)))
    return out


def moe_tail_workspace_bytes(which: int, b: int, dim: int) -> int:
    return int(lib().moe_tail_workspace_bytes(which, b, dim))


def moe_tail_latent_up(latent, gamma, w_up, shared, out, workspace, *, eps=1e-6, stream=None) -> torch.Tensor:
    """Latent tail into out (BF16 [b, H]): latent BF16 [tp, b, L], gamma BF16 [L],
    w_up BF16 [H, L], shared BF16 [tp_s, b, H] or None, workspace uint8 CUDA
    tensor of at least moe_tail_workspace_bytes(0, b, L) bytes (y after the call)."""
    tp, b, L, H, tp_s = _latent_args(latent, gamma, w_up, shared, out, None)
    _cuda(workspace)
    _check("moe_tail_latent_up", lib().moe_tail_latent_up(
        _p(latent), _p(gamma), eps, _p(w_up), _p(shared), tp_s, b, tp, L, H, _p(out), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def moe_tail_latent_up_flags(latent, gamma, w_up, shared, out, y, *, eps=1e-6, inputs_ready=False,
                             weights_static=False, stream=None) -> torch.Tensor:
    """The latent tail into out (BF16 [b, H]) and y (BF16 [b, L]), with the
    split calls' promises: inputs_ready (latent and gamma, as for
    moe_tail_latent_norm) and weights_static (w_up, as for moe_tail_up_project).
    The norm and the up-projection, or with the latent tail's kernel form
    pinned to one kernel (moe_tail_set_kernel_form(FORM_LATENT, FORM_LATENT_ONE_KERNEL)) one kernel
    that forms y on chip (slower on GB300); the result is bit for bit that of
    the two split calls either way."""
    tp, b, L, H, tp_s = _latent_args(latent, gamma, w_up, shared, out, y)
    flags = (INPUTS_READY if inputs_ready else 0) | (WEIGHTS_STATIC if weights_static else 0)
    _check("moe_tail_latent_up_flags", lib().moe_tail_latent_up_flags(
        _p(latent), _p(gamma), eps, _p(w_up), _p(shared), tp_s, b, tp, L, H, _p(out), _p(y), flags,
        _stream(stream)))
    return out


def moe_tail_latent_norm(latent, gamma, y, *, eps=1e-6, inputs_ready=False, stream=None) -> torch.Tensor:
    """The latent tail's first step into y (BF16 [b, L]): the slot-summed latent
    BF16 [tp, b, L], RMS-normalised and scaled by gamma BF16 [L].
    inputs_ready: latent and gamma are not written by work still in flight on
    the stream, so the kernel may read them before the preceding kernel ends."""
    tp, b, L = _dims("latent", latent, 3)
    _like("latent", latent, torch.bfloat16, (tp, b, L))
    _like("gamma", gamma, torch.bfloat16, (L,))
    _like("y", y, torch.bfloat16, (b, L))
    _cuda(latent, gamma, y)
    _check("moe_tail_latent_norm", lib().moe_tail_latent_norm(
        _p(latent), _p(gamma), eps, b, tp, L, _p(y), INPUTS_READY if inputs_ready else 0, _stream(stream)))
    return y


def moe_tail_up_project(y, w_up, shared, out, *, weights_static=False, stream=None) -> torch.Tensor:
    """The latent tail's second step into out (BF16 [b, H]): y BF16 [b, L] times
    w_up BF16 [H, L] transposed, plus shared BF16 [tp_s, b, H] (or None).
    weights_static: w_up is not written by work still in flight on the stream,
    so the kernel may request weight tiles before the preceding kernel ends."""
    b, L = _dims("y", y, 2)
    H, _ = _dims("w_up", w_up, 2)
    tp_s = 0 if shared is None else _dims("shared", shared, 3)[0]
    _like("y", y, torch.bfloat16, (b, L))
    _like("w_up", w_up, torch.bfloat16, (H, L))
    if shared is not None:
        _like("shared", shared, torch.bfloat16, (tp_s, b, H))
    _like("out", out, torch.bfloat16, (b, H))
    _cuda(y, w_up, shared, out)
    _check("moe_tail_up_project", lib().moe_tail_up_project(
        _p(y), _p(w_up), _p(shared), tp_s, b, L, H, _p(out), WEIGHTS_STATIC if weights_static else 0,
        _stream(stream)))
    return out


def moe_tail_up_project_shared_down(y, w_up, shared, h, w_down, out, d_out=None, *, weights_static=False,
                                    stream=None) -> torch.Tensor:
    """The up-projection of y (BF16 [b, L]) with w_up (BF16 [H, L]) plus the
    shared partials (BF16 [tp_s, b, H] or None) plus bf16(d), d the down
    projection of h (BF16 [b, I]) with w_down (BF16 [H, I]), in one kernel,
    into out (BF16 [b, H]); d_out (BF16 [b, H], optional) receives bf16(d)."""
    b, L = _dims("y", y, 2)
    H, _ = _dims("w_up", w_up, 2)
    _, I = _dims("h", h, 2)
    tp_s = 0 if shared is None else _dims("shared", shared, 3)[0]
    _like("y", y, torch.bfloat16, (b, L))
    _like("w_up", w_up, torch.bfloat16, (H, L))
    if shared is not None:
        _like("shared", shared, torch.bfloat16, (tp_s, b, H))
    _like("h", h, torch.bfloat16, (b, I))
    _like("w_down", w_down, torch.bfloat16, (H, I))
    _like("out", out, torch.bfloat16, (b, H))
    if d_out is not None:
        _like("d_out", d_out, torch.bfloat16, (b, H))
    _cuda(y, w_up, shared, h, w_down, out, d_out)
    _check("moe_tail_up_project_shared_down", lib().moe_tail_up_project_shared_down(
        _p(y), _p(w_up), _p(shared), tp_s, _p(h), _p(w_down), b, L, I, H, _p(out), _p(d_out),
        WEIGHTS_STATIC if weights_static else 0, _stream(stream)))
    return out


def moe_shared_gate_up(x, w_gate, w_up, h, *, weights_static=False, inputs_ready=False, stream=None) -> torch.Tensor:
    """The shared expert's gate/up projection and SiLU into h (BF16 [b, I]):
    x BF16 [b, H], w_gate and w_up BF16 [I, H].  inputs_ready promises that x
    is not being written by work in flight on the stream (h is written only
    after that work ends)."""
    b, H = _dims("x", x, 2)
    I, _ = _dims("w_gate", w_gate, 2)
    _like("x", x, torch.bfloat16, (b, H))
    _like("w_gate", w_gate, torch.bfloat16, (I, H))
    _like("w_up", w_up, torch.bfloat16, (I, H))
    _like("h", h, torch.bfloat16, (b, I))
    _cuda(x, w_gate, w_up, h)
    _check("moe_shared_gate_up", lib().moe_shared_gate_up(
        _p(x), _p(w_gate), _p(w_up), b, H, I, _p(h),
        (WEIGHTS_STATIC if weights_static else 0) | (INPUTS_READY if inputs_ready else 0), _stream(stream)))
    return h


def moe_shared_down(h, w_down, out, *, accumulate=True, weights_static=False, stream=None) -> torch.Tensor:
    """The shared expert's down projection of h (BF16 [b, I]) with w_down BF16
    [H, I], written into out (BF16 [b, H]) or added into it (accumulate)."""
    b, I = _dims("h", h, 2)
    H, _ = _dims("w_down", w_down, 2)
    _like("h", h, torch.bfloat16, (b, I))
    _like("w_down", w_down, torch.bfloat16, (H, I))
    _like("out", out, torch.bfloat16, (b, H))
    _cuda(h, w_down, out)
    _check("moe_shared_down", lib().moe_shared_down(
        _p(h), _p(w_down), b, H, I, _p(out), int(bool(accumulate)), WEIGHTS_STATIC if weights_static else 0,
        _stream(stream)))
    return out


def moe_shared_down_persistent(h, w_down, out, *, accumulate=True, ctas=0, weights_static=False,
                               stream=None) -> torch.Tensor:
    """The down projection as a persistent kernel: ctas CTAs (0: one per output
    tile, at most one per SM) walk the output tiles over the whole K range with
    two alternating tensor-memory accumulators.  Same arguments and result as
    moe_shared_down, up to the order of d's FP32 sum."""
    b, I = _dims("h", h, 2)
    H, _ = _dims("w_down", w_down, 2)
    _like("h", h, torch.bfloat16, (b, I))
    _like("w_down", w_down, torch.bfloat16, (H, I))
    _like("out", out, torch.bfloat16, (b, H))
    _cuda(h, w_down, out)
    _check("moe_shared_down_persistent", lib().moe_shared_down_persistent(
        _p(h), _p(w_down), b, H, I, _p(out), int(bool(accumulate)), int(ctas),
        WEIGHTS_STATIC if weights_static else 0, _stream(stream)))
    return out


def moe_tail_latent_up_noalloc(latent, gamma, w_up, shared, out, *, eps=1e-6, stream=None) -> torch.Tensor:
    """The latent tail without a workspace, for callers that cannot allocate
    device memory (a plugin given only its input and output buffers, a host
    whose device memory is all held by its own pool, a path that must not
    call cudaMalloc): y lives in a fixed array of NOALLOC_SCRATCH_BYTES inside
    the library, shared by every call.  Same arguments as moe_tail_latent_up
    minus the workspace; b * L * 2 must not exceed NOALLOC_SCRATCH_BYTES.
    Calls that may overlap on the GPU race on the shared array."""
    tp, b, L, H, tp_s = _latent_args(latent, gamma, w_up, shared, out, None)
    if b * L * 2 > NOALLOC_SCRATCH_BYTES:
        raise ValueError(f"moe_tail_latent_up_noalloc: y needs {b * L * 2} bytes, more than the library's "
                         f"built-in {NOALLOC_SCRATCH_BYTES}-byte scratch; use moe_tail_latent_up with a workspace")
    _check("moe_tail_latent_up_noalloc", lib().moe_tail_latent_up_noalloc(
        _p(latent), _p(gamma), eps, _p(w_up), _p(shared), tp_s, b, tp, L, H, _p(out), _stream(stream)))
    return out


def moe_shared_expert(x, w_gate, w_up, w_down, out, workspace, *, accumulate=True, stream=None) -> torch.Tensor:
    """Fused shared expert into out (BF16 [b, H]): x BF16 [b, H], w_gate/w_up BF16
    [I, H], w_down BF16 [H, I], workspace of at least moe_tail_workspace_bytes(1, b, I)
    bytes (h after the call); out += down(...) when accumulate."""
    b, H = _dims("x", x, 2)
    I, _ = _dims("w_gate", w_gate, 2)
    _like("x", x, torch.bfloat16, (b, H))
    _like("w_gate", w_gate, torch.bfloat16, (I, H))
    _like("w_up", w_up, torch.bfloat16, (I, H))
    _like("w_down", w_down, torch.bfloat16, (H, I))
    _like("out", out, torch.bfloat16, (b, H))
    _cuda(x, w_gate, w_up, w_down, out, workspace)
    _check("moe_shared_expert", lib().moe_shared_expert(
        _p(x), _p(w_gate), _p(w_up), _p(w_down), b, H, I, _p(out), int(bool(accumulate)), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def _eight_bits(q, scale, rows: int, width: int, group: int) -> int:
    """The type code of 8-bit rows q [rows, width] and their FP32 scales: [rows]
    (group 0) or [rows, ceil(width / 128)] (group 128)."""
    kind = Q_DTYPES.get(q.dtype)
    if kind is None:
        raise ValueError(f"q must be torch.int8 or torch.float8_e4m3fn, got {q.dtype}")
    if group != 0 and group != QUANT_GROUP:
        raise ValueError(f"group must be 0 (one scale a row) or {QUANT_GROUP}, got {group}")
    _like("q", q, q.dtype, (rows, width))
    _like("scale", scale, torch.float32, (rows, -(-width // group)) if group else (rows,))
    return kind


def moe_tail_norm_quant(x, residual, gamma, q, scale, *, residual_out=None, y=None, gain_center=1.0, eps=1e-6, group=0,
                        stream=None):
    """h = x + residual, its RMS norm with gains gamma + gain_center, in 8 bits
    into q (int8 or float8_e4m3fn [b, H]) and scale (FP32 [b], or with
    group=128 [b, ceil(H / 128)]); x, residual BF16 [b, H] (residual may be
    None), gamma BF16 [H].  residual_out (BF16 [b, H], may be x or residual)
    receives bf16(h), y the normed row in BF16.  Returns (q, scale)."""
    shape = b, H = _dims("x", x, 2)
    _like("x", x, torch.bfloat16, shape)
    _like("gamma", gamma, torch.bfloat16, (H,))
    if residual is not None:
        _like("residual", residual, torch.bfloat16, shape)
    if residual_out is not None:
        _like("residual_out", residual_out, torch.bfloat16, shape)
    if y is not None:
        _like("y", y, torch.bfloat16, shape)
    kind = _eight_bits(q, scale, b, H, group)
    _cuda(x, residual, gamma, q, scale, residual_out, y)
    _check("moe_tail_norm_quant", lib().moe_tail_norm_quant(
        _p(x), _p(residual), _p(gamma), gain_center, eps, b, H, kind, group, _p(residual_out), _p(y), _p(q), _p(scale),
        _stream(stream)))
    return q, scale


def moe_tail_silu_quant(gate_up, q, scale, *, used_rows=None, group=0, stream=None):
    """silu(gate) * up in 8 bits into q (int8 or float8_e4m3fn [rows, I]) and
    scale (as for moe_tail_norm_quant); gate_up BF16 [rows, 2 I], a row's gate
    columns before its up columns.  used_rows (int32 CUDA tensor of one
    element): rows from it on are neither read nor written.  Returns (q, scale)."""
    rows, I2 = _dims("gate_up", gate_up, 2)
    _like("gate_up", gate_up, torch.bfloat16, (rows, I2 // 2 * 2))
    if used_rows is not None:
        if used_rows.numel() != 1:
            raise ValueError(f"used_rows must have one element, got shape {tuple(used_rows.shape)}")
        _like("used_rows", used_rows, torch.int32, used_rows.shape)
    kind = _eight_bits(q, scale, rows, I2 // 2, group)
    _cuda(gate_up, q, scale, used_rows)
    _check("moe_tail_silu_quant", lib().moe_tail_silu_quant(
        _p(gate_up), _p(used_rows), rows, I2 // 2, kind, group, _p(q), _p(scale), _stream(stream)))
    return q, scale


def moe_tail_block_norm(x, residual, post_gamma, pre_gamma, residual_out, y, *, token_gate=None, channel_gate=None, rstd=None,
                        residual_scale=1.0, gain_center=1.0, eps=1e-6, stream=None):
    """h = residual_scale * residual + token_gate * channel_gate * n into residual_out, n the RMS norm of x with gains
    post_gamma + gain_center (post_gamma None: x itself), and the RMS norm of h with gains pre_gamma + gain_center into y:
    x, residual, residual_out, y BF16 [b, H] (residual_out may be x or residual), gammas BF16 [H].  token_gate (FP32 [b])
    and channel_gate (BF16 [H]) may each be None: ones.  rstd (FP32 [b, 2] or None) receives 1 / rms of x and of h, for
    moe_tail_block_norm_grad.  Returns (residual_out, y)."""
    shape = b, H = _dims("x", x, 2)
    bf, f32 = torch.bfloat16, torch.float32
    _operands(("x", x, bf, shape), ("residual", residual, bf, shape), ("post_gamma", post_gamma, bf, (H,)),
              ("pre_gamma", pre_gamma, bf, (H,)), ("residual_out", residual_out, bf, shape), ("y", y, bf, shape),
              ("token_gate", token_gate, f32, (b,)), ("channel_gate", channel_gate, bf, (H,)), ("rstd", rstd, f32, (b, 2)))
    _check("moe_tail_block_norm", lib().moe_tail_block_norm(
        _p(x), _p(residual), _p(post_gamma), _p(pre_gamma), _p(token_gate), _p(channel_gate), residual_scale, gain_center, eps,
        b, H, _p(residual_out), _p(y), _p(rstd), _stream(stream)))
    return residual_out, y


def moe_tail_block_norm_grad_workspace_bytes(b: int, H: int) -> int:
    return int(lib().moe_tail_block_norm_grad_workspace_bytes(b, H))


def moe_tail_block_norm_grad(d_y, d_residual_out, x, residual, post_gamma, pre_gamma, rstd, d_x, d_residual, workspace, *,
                             token_gate=None, channel_gate=None, d_post_gamma=None, d_pre_gamma=None, d_token_gate=None,
                             d_channel_gate=None, residual_scale=1.0, gain_center=1.0, stream=None):
    """The gradients of moe_tail_block_norm given d_y and d_residual_out (BF16 [b, H]; d_residual_out may be None: zeros), its
    inputs and the rstd it left: d_x and d_residual (BF16 [b, H]; they may be d_y and d_residual_out), and where they are
    wanted d_post_gamma, d_pre_gamma and d_channel_gate (FP32 [H]) and d_token_gate (FP32 [b]).  workspace: a CUDA tensor of
    at least moe_tail_block_norm_grad_workspace_bytes(b, H) bytes.  Returns (d_x, d_residual)."""
    shape = b, H = _dims("d_y", d_y, 2)
    bf, f32 = torch.bfloat16, torch.float32
    for name, grad, of in (("d_post_gamma", d_post_gamma, post_gamma), ("d_token_gate", d_token_gate, token_gate),
                           ("d_channel_gate", d_channel_gate, channel_gate)):
        if grad is not None and of is None:
            raise ValueError(f"{name} must be None where {name[2:]} is")
    _operands(("d_y", d_y, bf, shape), ("d_residual_out", d_residual_out, bf, shape), ("x", x, bf, shape),
              ("residual", residual, bf, shape), ("post_gamma", post_gamma, bf, (H,)), ("pre_gamma", pre_gamma, bf, (H,)),
              ("rstd", rstd, f32, (b, 2)), ("d_x", d_x, bf, shape), ("d_residual", d_residual, bf, shape),
              ("workspace", workspace, workspace.dtype, workspace.shape), ("token_gate", token_gate, f32, (b,)),
              ("channel_gate", channel_gate, bf, (H,)), ("d_post_gamma", d_post_gamma, f32, (H,)),
              ("d_pre_gamma", d_pre_gamma, f32, (H,)), ("d_token_gate", d_token_gate, f32, (b,)),
              ("d_channel_gate", d_channel_gate, f32, (H,)))
    _check("moe_tail_block_norm_grad", lib().moe_tail_block_norm_grad(
        _p(d_y), _p(d_residual_out), _p(x), _p(residual), _p(post_gamma), _p(pre_gamma), _p(token_gate), _p(channel_gate),
        _p(rstd), residual_scale, gain_center, b, H, _p(d_x), _p(d_residual), _p(d_post_gamma), _p(d_pre_gamma),
        _p(d_token_gate), _p(d_channel_gate), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return d_x, d_residual


def moe_tail_sort_workspace_bytes(b: int, K: int, num_experts: int) -> int:
    return int(lib().moe_tail_sort_workspace_bytes(b, K, num_experts))


def moe_tail_sort_routes(expert_ids, expert_offsets, permuted_idx, source, workspace, *, stream=None):
    """The routes of expert_ids (int32 [b, K]) sorted by expert, stably:
    expert_offsets (int32 [num_experts + 1]), permuted_idx (int32 [b, K], a
    route's row or -1 where its id is outside [0, num_experts)) and source
    (int32 [b * K], a row's route or -1).  workspace: a CUDA tensor of at least
    moe_tail_sort_workspace_bytes(b, K, num_experts) bytes."""
    b, K = _dims("expert_ids", expert_ids, 2)
    E = _dims("expert_offsets", expert_offsets, 1)[0] - 1
    _like("expert_ids", expert_ids, torch.int32, (b, K))
    _like("expert_offsets", expert_offsets, torch.int32, (E + 1,))
    _like("permuted_idx", permuted_idx, torch.int32, (b, K))
    _like("source", source, torch.int32, (b * K,))
    _cuda(expert_ids, expert_offsets, permuted_idx, source, workspace)
    _check("moe_tail_sort_routes", lib().moe_tail_sort_routes(
        _p(expert_ids), b, K, E, _p(expert_offsets), _p(permuted_idx), _p(source), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return expert_offsets, permuted_idx, source


def moe_tail_dispatch_rows(x, permuted_idx, rows, *, scale=None, row_scale=None, stream=None) -> torch.Tensor:
    """rows[permuted_idx[t, k]] = x[t]: x [b, H] and rows [num_rows, H] of one
    type (BF16, int8 or float8_e4m3fn), permuted_idx int32 [b, K]; 8-bit rows'
    scales likewise from scale (FP32 [b]) into row_scale (FP32 [num_rows])."""
    b, H = _dims("x", x, 2)
    num_rows, _ = _dims("rows", rows, 2)
    _, K = _dims("permuted_idx", permuted_idx, 2)
    if x.dtype != torch.bfloat16 and x.dtype not in Q_DTYPES:
        raise ValueError(f"x must be torch.bfloat16, torch.int8 or torch.float8_e4m3fn, got {x.dtype}")
    _like("rows", rows, x.dtype, (num_rows, H))
    _like("permuted_idx", permuted_idx, torch.int32, (b, K))
    if (scale is None) != (row_scale is None):
        raise ValueError("scale and row_scale must be given together")
    if scale is not None:
        _like("scale", scale, torch.float32, (b,))
        _like("row_scale", row_scale, torch.float32, (num_rows,))
    _cuda(x, permuted_idx, rows, scale, row_scale)
    _check("moe_tail_dispatch_rows", lib().moe_tail_dispatch_rows(
        _p(x), _p(scale), _p(permuted_idx), b, K, H, x.element_size(), num_rows, _p(rows), _p(row_scale),
        _stream(stream)))
    return rows


def moe_tail_combine_rows(rows, permuted_idx, route_weights, out, *, stream=None) -> torch.Tensor:
    """out[t] (BF16 [b, H]) = the sum over t's routes, in order, of their weight
    times their row of rows (BF16 [num_rows, H]); permuted_idx int32 [b, K],
    route_weights FP32 or BF16 [b, K], or None for ones (the gradient of
    moe_tail_dispatch_rows, given the rows' gradients)."""
    num_rows, H = _dims("rows", rows, 2)
    b, K = _dims("permuted_idx", permuted_idx, 2)
    _like("rows", rows, torch.bfloat16, (num_rows, H))
    _like("permuted_idx", permuted_idx, torch.int32, (b, K))
    if route_weights is not None:
        _weights(route_weights)
        _like("route_weights", route_weights, route_weights.dtype, (b, K))
    _like("out", out, torch.bfloat16, (b, H))
    _cuda(rows, permuted_idx, route_weights, out)
    _check("moe_tail_combine_rows", lib().moe_tail_combine_rows(
        _p(rows), num_rows, _p(permuted_idx), _p(route_weights),
        W_FP32 if route_weights is None else _weights(route_weights), b, K, H, _p(out), _stream(stream)))
    return out


def moe_tail_combine_grad(d_out, rows, permuted_idx, route_weights, d_rows, d_weights, *, stream=None):
    """The gradients of moe_tail_combine_rows given d_out (BF16 [b, H]): d_rows
    (BF16 [num_rows, H]) and d_weights (FP32 [b, K], whatever the weights'
    type).  Returns (d_rows, d_weights)."""
    b, H = _dims("d_out", d_out, 2)
    num_rows, _ = _dims("rows", rows, 2)
    _, K = _dims("permuted_idx", permuted_idx, 2)
    _like("d_out", d_out, torch.bfloat16, (b, H))
    _like("rows", rows, torch.bfloat16, (num_rows, H))
    _like("permuted_idx", permuted_idx, torch.int32, (b, K))
    wdtype = _weights(route_weights)
    _like("route_weights", route_weights, route_weights.dtype, (b, K))
    _like("d_rows", d_rows, torch.bfloat16, (num_rows, H))
    _like("d_weights", d_weights, torch.float32, (b, K))
    _cuda(d_out, rows, permuted_idx, route_weights, d_rows, d_weights)
    _check("moe_tail_combine_grad", lib().moe_tail_combine_grad(
        _p(d_out), _p(rows), num_rows, _p(permuted_idx), _p(route_weights), wdtype, b, K, H, _p(d_rows), _p(d_weights),
        _stream(stream)))
    return d_rows, d_weights


def moe_tail_expert_product_workspace_bytes(rows: int, num_experts: int, N: int, D: int) -> int:
    return int(lib().moe_tail_expert_product_workspace_bytes(rows, num_experts, N, D))


def moe_tail_expert_product(x, x_scale, w, w_scale, out, workspace, *, expert_offsets=None, stream=None) -> torch.Tensor:
    """out (BF16 [rows, N]) = x (int8 [rows, D], x_scale FP32 [rows]) times the
    transpose of each row's expert's weight w[e] (int8 [num_experts, N, D],
    w_scale FP32 [num_experts, N]); expert_offsets int32 [num_experts + 1]
    (moe_tail_sort_routes), or None with one expert.  workspace: a CUDA tensor
    of at least moe_tail_expert_product_workspace_bytes(rows, num_experts, N, D) bytes."""
    rows, D = _dims("x", x, 2)
    E, N, _ = _dims("w", w, 3)
    _like("x", x, torch.int8, (rows, D))
    _like("x_scale", x_scale, torch.float32, (rows,))
    _like("w", w, torch.int8, (E, N, D))
    _like("w_scale", w_scale, torch.float32, (E, N))
    if expert_offsets is not None:
        _like("expert_offsets", expert_offsets, torch.int32, (E + 1,))
    _like("out", out, torch.bfloat16, (rows, N))
    _cuda(x, x_scale, w, w_scale, expert_offsets, out, workspace)
    _check("moe_tail_expert_product", lib().moe_tail_expert_product(
        _p(x), _p(x_scale), _p(w), _p(w_scale), _p(expert_offsets), rows, E, N, D, _p(out), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def _product_i4(name, x, w, group_scale, channel_scale, out, group, expert_offsets, halves, stream):
    rows, D = _dims("x", x, 2)
    E, channels, _ = _dims("w", w, 3)
    if group not in I4_GROUPS:
        raise ValueError(f"group must be one of {I4_GROUPS}, got {group}")
    if channels % halves:
        raise ValueError(f"w must have an even number of channels (gate and up), got shape {tuple(w.shape)}")
    _operands(("x", x, torch.bfloat16, (rows, D)), ("w", w, torch.uint8, (E, channels, -(-D // 128) * 64)),
              ("group_scale", group_scale, torch.float8_e4m3fn, (E, channels, -(-(-(-D // group)) // 4) * 4)),
              ("channel_scale", channel_scale, torch.float32, (E, channels)),
              ("expert_offsets", expert_offsets, torch.int32, (E + 1,)), ("out", out, torch.bfloat16, (rows, channels // halves)))
    _check(name, getattr(lib(), name)(
        _p(x), _p(w), _p(group_scale), _p(channel_scale), _p(expert_offsets), rows, E, channels // halves, D, group, _p(out),
        _stream(stream)))
    return out


def moe_tail_expert_product_i4(x, w, group_scale, channel_scale, out, *, group, expert_offsets=None, stream=None) -> torch.Tensor:
    """out (BF16 [rows, N]) = x (BF16 [rows, D]) times the transpose of each row's expert's 4-bit weight: w uint8
    [num_experts, N, 64 * ceil(D / 128)] in the layout of include/moe_tail.h (expert_layer.quantise_groups makes it),
    group_scale float8_e4m3fn [num_experts, N, ceil(D / group) up to a multiple of 4], channel_scale FP32 [num_experts, N];
    group 32, 64 or 128; expert_offsets int32 [num_experts + 1] (moe_tail_sort_routes), or None with one expert."""
    return _product_i4("moe_tail_expert_product_i4", x, w, group_scale, channel_scale, out, group, expert_offsets, 1, stream)


def moe_tail_gated_product_i4(x, w, group_scale, channel_scale, out, *, group, expert_offsets=None, stream=None) -> torch.Tensor:
    """out (BF16 [rows, I]) = silu(gate) * up in one kernel, gate and up the first and last I channels of that product
    with a weight of 2 I channels (arguments as for moe_tail_expert_product_i4)."""
    return _product_i4("moe_tail_gated_product_i4", x, w, group_scale, channel_scale, out, group, expert_offsets, 2, stream)


def moe_tail_product_i4_tile_rows(rows: int, num_experts: int, N: int, D: int, *, gated: bool = False) -> int:
    """Rows of a tile that the 4-bit products take for these sizes: 8 (the kernel for few rows), 16, 32, 64 or 128 (wide
    tiles); 0 where they refuse the sizes.  N: channels of the result."""
    return int(lib().moe_tail_product_i4_tile_rows(rows, num_experts, N, D, int(bool(gated))))


def moe_tail_status_str(status: int) -> str:
    return status_string(status)


def moe_tail_take_device_error() -> int:
    """Bits raised by bounded waits inside the kernels since the last read (0: none)."""
    bits = ctypes.c_uint(0)
    _check("moe_tail_take_device_error", lib().moe_tail_take_device_error(ctypes.byref(bits)))
    return int(bits.value)


def moe_tail_set_kernel_form(call: int, form: int) -> None:
    """Pin the kernel form of a call (FORM_EP, FORM_TP, FORM_LATENT; form 0 is
    the library's choice, see include/moe_tail.h).  Every form of a call gives
    the same bits; the setting is process-wide."""
    _check("moe_tail_set_kernel_form", lib().moe_tail_set_kernel_form(call, form))


def moe_tail_set_stage_wait_limit(limit_ns: int) -> None:
    """Failure-detection test hook: the operand-stage wait limit (ns) of the
    GEMM, staged finalize, product and wide norm-gradient kernels for later
    calls; 0 restores the default.
    A limit shorter than a memory trip makes calls abort (device error bit 1)."""
    _check("moe_tail_set_stage_wait_limit", lib().moe_tail_set_stage_wait_limit(limit_ns))


class kernel_form:
    """Context manager: the call's kernel form pinned inside the block, the
    library's choice again after it."""

    def __init__(self, call: int, form: int):
        self.call, self.form = call, form

    def __enter__(self):
        moe_tail_set_kernel_form(self.call, self.form)
        return self

    def __exit__(self, *exc):
        moe_tail_set_kernel_form(self.call, 0)
        return False


def moe_tail_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launch the failure-detection self-test: a bounded wait that expires after
    limit_us and reports it through moe_tail_take_device_error()."""
    _check("moe_tail_selftest_wait_timeout", lib().moe_tail_selftest_wait_timeout(limit_us, _stream(stream)))
