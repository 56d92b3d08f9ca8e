"""Mixture-of-Experts layers with 8-bit and with 4-bit experts, made of the library's calls.  ExpertLayerI8:

    norm      h = x + residual, its RMS norm in int8 rows (and in BF16, for the router)   moe_tail_norm_quant
    experts   routes sorted by expert, rows copied into that order                        moe_tail_sort_routes,
                                                                                          moe_tail_dispatch_rows
              gate and up, silu(gate) * up in int8 rows, down                             moe_tail_expert_product,
                                                                                          moe_tail_silu_quant
              back to tokens: the EP finalize (each route's row normalised) or the        moe_tail_ep_finalize,
              plain weighted sum                                                          moe_tail_combine_rows

ExpertLayerI4, for 4-bit weights and blocks whose output is normed and gated:

    norm      the norm after the last block, its gate, the scaled residual,               moe_tail_block_norm
              and the norm before this one
    experts   routes sorted, rows copied, gate and up with silu(gate) * up in one         moe_tail_gated_product_i4,
              kernel, down, back to tokens                                                moe_tail_expert_product_i4

The router stands between the two steps and belongs to the caller.  Buffers are allocated once, for max_tokens tokens;
the calls only enqueue work on the current stream, so both steps can be captured in a CUDA graph.

    python -m moe_decode_tail_gb300.expert_layer --tokens 64 --bits 4

runs a layer on random weights and prints its time.
"""
from __future__ import annotations

import torch

from . import (I4_GROUPS, _like, moe_tail_block_norm, moe_tail_combine_rows, moe_tail_dispatch_rows, moe_tail_ep_finalize,
               moe_tail_expert_product, moe_tail_expert_product_i4, moe_tail_expert_product_workspace_bytes,
               moe_tail_gated_product_i4, moe_tail_norm_quant, moe_tail_silu_quant, moe_tail_sort_routes,
               moe_tail_sort_workspace_bytes)

__all__ = ["ExpertLayerI8", "ExpertLayerI4", "quantise_channels", "quantise_groups", "pack_int4"]

MAX_WIDTH = 32768            # columns of a row
MAX_ROUTES = 1 << 21         # of one sort
MAX_FINALIZE_TOKENS = 65535


def quantise_channels(w):
    """A weight [..., N, D] in int8 with a scale for each channel [..., N]: done once, when weights are loaded."""
    scale = w.float().abs().amax(-1).clamp_min(1e-30) / 127.0
    return torch.round(w.float() / scale[..., None]).to(torch.int8), scale


def pack_int4(q):
    """q int8 [..., N, D], values in [-8, 7], in the 4-bit products' layout: uint8 [..., N, 64 * ceil(D / 128)]."""
    q = torch.nn.functional.pad(q, (0, -q.shape[-1] % 128)) + 8
    lead, blocks = q.shape[:-1], q.shape[-1] // 128
    columns = q.view(*lead, blocks, 4, 4, 8).transpose(-2, -3)  # word 4 t + i: columns 32 i + 8 t + c
    # nibbles 0 .. 3 the even columns, 4 .. 7 the odd ones; a byte has two
    nibbles = torch.cat([columns[..., 0::2], columns[..., 1::2]], -1).to(torch.uint8)
    return (nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)).reshape(*lead, blocks * 64).contiguous()


def quantise_groups(w, group=128):
    """A weight [..., N, D] in 4 bits with scales: (packed uint8 [..., N, 64 * ceil(D / 128)], group scales float8_e4m3fn
    [..., N, ceil(D / group) up to a multiple of 4], channel scales FP32 [..., N]), done once, when weights are loaded.  A
    channel's largest group has the group scale 448 or near it, and every weight is rounded by the scales as they are
    stored."""
    if group not in I4_GROUPS:
        raise ValueError(f"group must be one of {I4_GROUPS}, got {group}")
    D = w.shape[-1]
    groups = -(-D // group)
    w = torch.nn.functional.pad(w.float(), (0, groups * group - D)).unflatten(-1, (groups, group))
    top = w.abs().amax(-1)
    channel_scale = top.amax(-1).clamp_min(1e-30) / (7.0 * 448.0)
    group_scale = (top / (7.0 * channel_scale[..., None])).clamp_max(448.0).to(torch.float8_e4m3fn)
    step = group_scale.float() * channel_scale[..., None]
    q = torch.where(step[..., None] > 0, torch.round(w / step[..., None]), 0.0).clamp(-8, 7).to(torch.int8)
    padded = torch.nn.functional.pad(group_scale.float(), (0, -groups % 4)).to(torch.float8_e4m3fn)
    return pack_int4(q.flatten(-2)[..., :D]), padded, channel_scale


class _ExpertLayer:
    """What the layers share: the routes' buffers, the way back to tokens, and that experts() follows the norm() of its
    tokens."""

    def _make_routes(self, gamma, E, H, max_tokens, top_k, finalize_gamma, gain_center, eps):
        """The buffers and values that both layers have; returns the maker of more buffers."""
        dev = gamma.device
        self.gamma, self.finalize_gamma = gamma, finalize_gamma
        self.max_tokens, self.K, self.gain_center, self.eps = max_tokens, top_k, gain_center, eps
        self._normed = None  # tokens of the last norm()

        def new(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=dev)

        self._offsets = new(torch.int32, E + 1)
        self._idx, self._source = new(torch.int32, max_tokens, top_k), new(torch.int32, max_tokens * top_k)
        self._rows = new(torch.bfloat16, max_tokens * top_k, H)
        return new

    @staticmethod
    def _sort_bytes(tokens, K, E, finalize) -> int:
        """The sort's workspace for so many tokens; ValueError for sizes that a call on the routes does not take."""
        rows = tokens * K
        sort = moe_tail_sort_workspace_bytes(tokens, K, E) if 0 <= rows <= MAX_ROUTES else 0
        if sort == 0:
            raise ValueError(f"{tokens} tokens of {K} routes each over {E} experts: 1 to 32 routes a token, {MAX_ROUTES} "
                             "in all and 1 to 1024 experts")
        if finalize and tokens > MAX_FINALIZE_TOKENS:
            raise ValueError(f"{tokens} tokens: moe_tail_ep_finalize takes at most {MAX_FINALIZE_TOKENS}")
        return sort

    def _sort(self, expert_ids):
        """The routes of the last norm's tokens sorted: (tokens, routes, permuted index)."""
        b, R = self._tokens(expert_ids), expert_ids.shape[0] * self.K
        if b != self._normed:
            raise ValueError(f"routes of {b} tokens, and the rows are those of "
                             + ("no norm()" if self._normed is None else f"a norm() of {self._normed}"))
        idx = self._idx[:b]
        moe_tail_sort_routes(expert_ids, self._offsets, idx, self._source[:R], self._workspace)
        return b, R, idx

    def _back(self, rows, idx, route_weights, out) -> torch.Tensor:
        """Route rows to tokens: each normalised and weighted, or only weighted."""
        if self.finalize_gamma is None:
            return moe_tail_combine_rows(rows, idx, route_weights, out)
        return moe_tail_ep_finalize(rows[None], idx[None], route_weights, self.finalize_gamma, out,
                                    gain_center=self.gain_center, eps=self.eps)

    def _tokens(self, t) -> int:
        if t.shape[0] > self.max_tokens:
            raise ValueError(f"{t.shape[0]} tokens, and the layer was made for {self.max_tokens}")
        return t.shape[0]


class ExpertLayerI8(_ExpertLayer):
    """gamma BF16 [H]; w_gate_up int8 [E, 2 I, H] (the I gate channels before the up channels) with scales FP32
    [E, 2 I]; w_down int8 [E, H, I] with scales FP32 [E, H].  finalize_gamma (BF16 [H]): the route rows are normalised
    with it before they are weighted and summed (moe_tail_ep_finalize); None: they are not (moe_tail_combine_rows).

    A layer keeps the rows of a norm() for its experts() in buffers of its own, so one layer serves one stream and one
    thread at a time."""

    def __init__(self, gamma, w_gate_up, s_gate_up, w_down, s_down, *, max_tokens, top_k, finalize_gamma=None,
                 gain_center=1.0, eps=1e-6):
        self.E, self.I2, self.H = w_gate_up.shape
        if self.I2 % 2 or tuple(w_down.shape) != (self.E, self.H, self.I2 // 2):
            raise ValueError(f"w_gate_up {tuple(w_gate_up.shape)} and w_down {tuple(w_down.shape)} do not belong together")
        workspace = self._workspace_bytes(max_tokens, top_k, finalize_gamma is not None)
        for name, t, dtype, shape in (
                ("gamma", gamma, torch.bfloat16, (self.H,)), ("w_gate_up", w_gate_up, torch.int8, w_gate_up.shape),
                ("s_gate_up", s_gate_up, torch.float32, (self.E, self.I2)), ("w_down", w_down, torch.int8, w_down.shape),
                ("s_down", s_down, torch.float32, (self.E, self.H)),
                ("finalize_gamma", finalize_gamma, torch.bfloat16, (self.H,))):
            if t is not None:
                _like(name, t, dtype, shape)
        self.w_gate_up, self.s_gate_up, self.w_down, self.s_down = w_gate_up, s_gate_up, w_down, s_down
        new = self._make_routes(gamma, self.E, self.H, max_tokens, top_k, finalize_gamma, gain_center, eps)
        rows, I = max_tokens * top_k, self.I2 // 2
        self._q, self._scale = new(torch.int8, max_tokens, self.H), new(torch.float32, max_tokens)
        self._x, self._x_scale = new(torch.int8, rows, self.H), new(torch.float32, rows)
        self._gate_up = new(torch.bfloat16, rows, self.I2)
        self._h, self._h_scale = new(torch.int8, rows, I), new(torch.float32, rows)
        self._workspace = new(torch.uint8, workspace)

    def _workspace_bytes(self, tokens, K, finalize) -> int:
        """What the calls need of workspace for so many tokens; ValueError for sizes that one of them does not take."""
        H, I, rows = self.H, self.I2 // 2, tokens * K
        sort = self._sort_bytes(tokens, K, self.E, finalize)
        products = [moe_tail_expert_product_workspace_bytes(rows, self.E, N, D) for N, D in ((self.I2, H), (H, I))]
        if max(H, I) > MAX_WIDTH or 0 in products:
            raise ValueError(f"H = {H} and I = {I} must be multiples of 16 up to {MAX_WIDTH}")
        return max(sort, *products)

    def norm(self, x, residual, *, y=None, residual_out=None):
        """x + residual normalised into the layer's int8 rows; residual_out (by default in place, where there is a
        residual) receives the sum, y (BF16, for the router) the normed rows.  Returns residual_out."""
        b = self._tokens(x)
        if residual_out is None:
            residual_out = residual
        self._normed = None
        moe_tail_norm_quant(x, residual, self.gamma, self._q[:b], self._scale[:b], residual_out=residual_out, y=y,
                            gain_center=self.gain_center, eps=self.eps)
        self._normed = b
        return residual_out

    def experts(self, expert_ids, route_weights, out) -> torch.Tensor:
        """The experts' contribution for the rows of the last norm() into out (BF16 [b, H]); expert_ids int32 [b, K] for
        that norm's b tokens (an id outside [0, E): not one of this layer's experts), route_weights [b, K]."""
        b, R, idx = self._sort(expert_ids)
        used = self._offsets[self.E:]
        x, h, rows = (t[:R] for t in (self._x, self._h, self._rows))
        moe_tail_dispatch_rows(self._q[:b], idx, x, scale=self._scale[:b], row_scale=self._x_scale[:R])
        moe_tail_expert_product(x, self._x_scale[:R], self.w_gate_up, self.s_gate_up, self._gate_up[:R], self._workspace,
                                expert_offsets=self._offsets)
        moe_tail_silu_quant(self._gate_up[:R], h, self._h_scale[:R], used_rows=used)
        moe_tail_expert_product(h, self._h_scale[:R], self.w_down, self.s_down, rows, self._workspace,
                                expert_offsets=self._offsets)
        return self._back(rows, idx, route_weights, out)


class ExpertLayerI4(_ExpertLayer):
    """gate_up: (packed uint8 [E, 2 I, ...], group scales, channel scales [E, 2 I]) as quantise_groups makes them from
    [E, 2 I, H] (the I gate channels before the up channels); down: the same from [E, H, I]; gamma BF16 [H], the norm before
    this layer's experts; post_gamma BF16 [H] or None, the norm of the last block's output before it joins the residual,
    which is scaled by residual_scale.  finalize_gamma as for ExpertLayerI8.

    A layer keeps the rows of a norm() for its experts() in buffers of its own, so one layer serves one stream and one
    thread at a time."""

    def __init__(self, gamma, gate_up, down, *, max_tokens, top_k, group=128, post_gamma=None, finalize_gamma=None,
                 residual_scale=1.0, gain_center=1.0, eps=1e-6):
        self.H = H = gamma.shape[0]
        self.E, I2, _ = gate_up[0].shape
        self.I = I = I2 // 2
        if group not in I4_GROUPS:
            raise ValueError(f"group must be one of {I4_GROUPS}, got {group}")
        if I2 % 2 or tuple(down[0].shape[:2]) != (self.E, H):
            raise ValueError(f"gate_up {tuple(gate_up[0].shape)} and down {tuple(down[0].shape)} do not belong together")
        if any(n % 8 or not 8 <= n <= MAX_WIDTH for n in (H, I)):
            raise ValueError(f"H = {H} and I = {I} must be multiples of 8 up to {MAX_WIDTH}")
        workspace = self._sort_bytes(max_tokens, top_k, self.E, finalize_gamma is not None)
        for name, t in (("gamma", gamma), ("post_gamma", post_gamma), ("finalize_gamma", finalize_gamma)):
            if t is not None:
                _like(name, t, torch.bfloat16, (H,))
        for name, (w, gs, cs), N, D in (("gate_up", gate_up, I2, H), ("down", down, H, I)):
            _like(name + "[0]", w, torch.uint8, (self.E, N, -(-D // 128) * 64))
            _like(name + "[1]", gs, torch.float8_e4m3fn, (self.E, N, -(-(-(-D // group)) // 4) * 4))
            _like(name + "[2]", cs, torch.float32, (self.E, N))
        self.gate_up, self.down, self.group = gate_up, down, group
        self.post_gamma, self.residual_scale = post_gamma, residual_scale
        new = self._make_routes(gamma, self.E, H, max_tokens, top_k, finalize_gamma, gain_center, eps)
        rows = max_tokens * top_k
        self._y, self._x = new(torch.bfloat16, max_tokens, H), new(torch.bfloat16, rows, H)
        self._h = new(torch.bfloat16, rows, I)
        self._workspace = new(torch.uint8, workspace)

    def norm(self, x, residual, *, residual_out=None, token_gate=None, channel_gate=None, rstd=None):
        """x, the last block's output, normed with post_gamma, gated and added to the scaled residual (in place, or into
        residual_out), and the sum normed with gamma into the layer's rows.  Returns (the sum, those rows), BF16 [b, H]:
        the rows are the router's input, and stay until the next norm().  rstd (FP32 [b, 2]) receives what
        moe_tail_block_norm_grad takes; its x and residual are those of before the call, so residual_out is one's own then."""
        b = self._tokens(x)
        if residual_out is None:
            residual_out = residual
        self._normed = None
        y = self._y[:b]
        moe_tail_block_norm(x, residual, self.post_gamma, self.gamma, residual_out, y, token_gate=token_gate,
                            channel_gate=channel_gate, rstd=rstd, residual_scale=self.residual_scale,
                            gain_center=self.gain_center, eps=self.eps)
        self._normed = b
        return residual_out, y

    def experts(self, expert_ids, route_weights, out) -> torch.Tensor:
        """The experts' contribution for the rows of the last norm() into out; arguments as for ExpertLayerI8."""
        b, R, idx = self._sort(expert_ids)
        x, h, rows = (t[:R] for t in (self._x, self._h, self._rows))
        moe_tail_dispatch_rows(self._y[:b], idx, x)
        moe_tail_gated_product_i4(x, *self.gate_up, h, group=self.group, expert_offsets=self._offsets)
        moe_tail_expert_product_i4(h, *self.down, rows, group=self.group, expert_offsets=self._offsets)
        return self._back(rows, idx, route_weights, out)


def main() -> None:
    import argparse

    ap = argparse.ArgumentParser(description="Run an expert layer on random weights and print its time")
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--intermediate", type=int, default=1024)
    ap.add_argument("--bits", type=int, choices=(8, 4), default=8, help="of a weight")
    ap.add_argument("--steps", type=int, default=20)
    o = ap.parse_args()
    b, E, K, H, I = o.tokens, o.experts, o.top_k, o.hidden, o.intermediate
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)

    quantise = quantise_channels if o.bits == 8 else quantise_groups
    gate_up = list(map(torch.stack, zip(*(quantise(normal(2 * I, H, std=0.02)) for _ in range(E)))))
    down = list(map(torch.stack, zip(*(quantise(normal(H, I, std=0.02)) for _ in range(E)))))
    sizes = dict(max_tokens=b, top_k=K, finalize_gamma=normal(H, std=0.1))
    if o.bits == 8:
        layer = ExpertLayerI8(normal(H, std=0.1), *gate_up, *down, **sizes)
    else:
        layer = ExpertLayerI4(normal(H, std=0.1), gate_up, down, post_gamma=normal(H, std=0.1), **sizes)
    x, residual, w_router = normal(b, H), normal(b, H), normal(E, H, std=0.02)
    y, out = torch.empty_like(x), torch.empty_like(x)

    def step():
        rows = y
        if o.bits == 8:
            layer.norm(x, residual, y=y)
        else:
            rows = layer.norm(x, residual)[1]
        logits, ids = (rows @ w_router.T).float().topk(K, dim=1)
        return layer.experts(ids.to(torch.int32), torch.softmax(logits, dim=1), out)

    for _ in range(3):
        step()
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(o.steps):
        step()
    end.record()
    torch.cuda.synchronize()
    print(f"{b} tokens, {E} {o.bits}-bit experts of {H} x {I}, top {K}: {1e3 * start.elapsed_time(end) / o.steps:.1f} us a step")


if __name__ == "__main__":
    main()
