"""A Mixture-of-Experts layer with 8-bit experts, made of the library's calls:

    norm      h = x + residual, its RMS norm in int8 rows (and in BF16, for the router)   moe_tail_norm_quant
    experts   routes sorted by expert, rows copied into that order                        moe_tail_sort_routes,
                                                                                          moe_tail_dispatch_rows
              gate and up, silu(gate) * up in int8 rows, down                             moe_tail_expert_product,
                                                                                          moe_tail_silu_quant
              back to tokens: the EP finalize (each route's row normalised) or the        moe_tail_ep_finalize,
              plain weighted sum                                                          moe_tail_combine_rows

The router stands between the two steps and belongs to the caller.  Buffers are allocated once, for max_tokens tokens;
the calls only enqueue work on the current stream, so both steps can be captured in a CUDA graph.

    python -m moe_decode_tail_gb300.expert_layer --tokens 64

runs a layer on random weights and prints its time.
"""
from __future__ import annotations

import torch

from . import (_like, moe_tail_combine_rows, moe_tail_dispatch_rows, moe_tail_ep_finalize, moe_tail_expert_product,
               moe_tail_expert_product_workspace_bytes, moe_tail_norm_quant, moe_tail_silu_quant, moe_tail_sort_routes,
               moe_tail_sort_workspace_bytes)

__all__ = ["ExpertLayerI8", "quantise_channels"]

MAX_WIDTH = 32768            # columns of a row in 8 bits
MAX_ROUTES = 1 << 21         # of one sort
MAX_FINALIZE_TOKENS = 65535


def quantise_channels(w):
    """A weight [..., N, D] in int8 with a scale for each channel [..., N]: done once, when weights are loaded."""
    scale = w.float().abs().amax(-1).clamp_min(1e-30) / 127.0
    return torch.round(w.float() / scale[..., None]).to(torch.int8), scale


class ExpertLayerI8:
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
        self.gamma, self.finalize_gamma = gamma, finalize_gamma
        self.w_gate_up, self.s_gate_up, self.w_down, self.s_down = w_gate_up, s_gate_up, w_down, s_down
        self.max_tokens, self.K, self.gain_center, self.eps = max_tokens, top_k, gain_center, eps
        self._normed = None  # tokens of the last norm()
        dev, rows, I = gamma.device, max_tokens * top_k, self.I2 // 2

        def new(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=dev)

        self._q, self._scale = new(torch.int8, max_tokens, self.H), new(torch.float32, max_tokens)
        self._offsets = new(torch.int32, self.E + 1)
        self._idx, self._source = new(torch.int32, max_tokens, top_k), new(torch.int32, rows)
        self._x, self._x_scale = new(torch.int8, rows, self.H), new(torch.float32, rows)
        self._gate_up = new(torch.bfloat16, rows, self.I2)
        self._h, self._h_scale = new(torch.int8, rows, I), new(torch.float32, rows)
        self._rows = new(torch.bfloat16, rows, self.H)
        self._workspace = new(torch.uint8, workspace)

    def _workspace_bytes(self, tokens, K, finalize) -> int:
        """What the calls need of workspace for so many tokens; ValueError for sizes that one of them does not take."""
        H, I, rows = self.H, self.I2 // 2, tokens * K
        sort = moe_tail_sort_workspace_bytes(tokens, K, self.E) if 0 <= rows <= MAX_ROUTES else 0
        if sort == 0:
            raise ValueError(f"{tokens} tokens of {K} routes each over {self.E} experts: 1 to 32 routes a token, {MAX_ROUTES} "
                             "in all and 1 to 1024 experts")
        products = [moe_tail_expert_product_workspace_bytes(rows, self.E, N, D) for N, D in ((self.I2, H), (H, I))]
        if max(H, I) > MAX_WIDTH or 0 in products:
            raise ValueError(f"H = {H} and I = {I} must be multiples of 16 up to {MAX_WIDTH}")
        if finalize and tokens > MAX_FINALIZE_TOKENS:
            raise ValueError(f"{tokens} tokens: moe_tail_ep_finalize takes at most {MAX_FINALIZE_TOKENS}")
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
        b, R = self._tokens(expert_ids), expert_ids.shape[0] * self.K
        if b != self._normed:
            raise ValueError(f"routes of {b} tokens, and the rows are those of "
                             + ("no norm()" if self._normed is None else f"a norm() of {self._normed}"))
        idx, used = self._idx[:b], self._offsets[self.E:]
        x, h, rows = (t[:R] for t in (self._x, self._h, self._rows))
        moe_tail_sort_routes(expert_ids, self._offsets, idx, self._source[:R], self._workspace)
        moe_tail_dispatch_rows(self._q[:b], idx, x, scale=self._scale[:b], row_scale=self._x_scale[:R])
        moe_tail_expert_product(x, self._x_scale[:R], self.w_gate_up, self.s_gate_up, self._gate_up[:R], self._workspace,
                                expert_offsets=self._offsets)
        moe_tail_silu_quant(self._gate_up[:R], h, self._h_scale[:R], used_rows=used)
        moe_tail_expert_product(h, self._h_scale[:R], self.w_down, self.s_down, rows, self._workspace,
                                expert_offsets=self._offsets)
        if self.finalize_gamma is None:
            return moe_tail_combine_rows(rows, idx, route_weights, out)
        return moe_tail_ep_finalize(rows[None], idx[None], route_weights, self.finalize_gamma, out,
                                    gain_center=self.gain_center, eps=self.eps)

    def _tokens(self, t) -> int:
        if t.shape[0] > self.max_tokens:
            raise ValueError(f"{t.shape[0]} tokens, and the layer was made for {self.max_tokens}")
        return t.shape[0]


def main() -> None:
    import argparse

    ap = argparse.ArgumentParser(description="Run an 8-bit expert layer on random weights and print its time")
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--intermediate", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    o = ap.parse_args()
    b, E, K, H, I = o.tokens, o.experts, o.top_k, o.hidden, o.intermediate
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)

    gate_up = [quantise_channels(normal(2 * I, H, std=0.02)) for _ in range(E)]
    down = [quantise_channels(normal(H, I, std=0.02)) for _ in range(E)]
    layer = ExpertLayerI8(normal(H, std=0.1), *map(torch.stack, zip(*gate_up)), *map(torch.stack, zip(*down)),
                          max_tokens=b, top_k=K, finalize_gamma=normal(H, std=0.1))
    x, residual, w_router = normal(b, H), normal(b, H), normal(E, H, std=0.02)
    y, out = torch.empty_like(x), torch.empty_like(x)

    def step():
        layer.norm(x, residual, y=y)
        logits, ids = (y @ w_router.T).float().topk(K, dim=1)
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
    print(f"{b} tokens, {E} experts of {H} x {I}, top {K}: {1e3 * start.elapsed_time(end) / o.steps:.1f} us a step")


if __name__ == "__main__":
    main()
