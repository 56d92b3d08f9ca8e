"""Workloads of the operators of an expert layer with 4-bit weights: what it does in place of the 8-bit products, and the
norms of a block whose output is normed and gated before it joins the residual.

    product    4-bit weights with group scales, dense or by expert           moe_tail_expert_product_i4
    gated      gate and up channels of such a weight, silu(gate) * up        moe_tail_gated_product_i4
    norm       a block's output normed, gated, added to the scaled           moe_tail_block_norm
               residual, and the norm before the next block
    gradient   the gradients of that                                         moe_tail_block_norm_grad

Each case has a plain form (elementary torch operations in 32 bits) and, with `own` set, the library's calls.

A weight is q * group_scale * channel_scale: q in [-8, 7], group_scale e4m3 for every `group` columns of a channel,
channel_scale FP32.  A channel's columns are stored in blocks of 128, 64 bytes each (sixteen 32-bit words, little endian):
word 4 t + i of a block holds the columns 32 i + 8 t + c, c = 0 .. 7, as q + 8 in nibble c / 2 (even c) or 4 + c / 2 (odd c).
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3 = torch.float8_e4m3fn
GAIN_CENTER, EPS = 1.0, 1e-6


def listed():
    return [
        # one dense 4-bit weight and the token of a single conversation: a matrix-vector product, a latency
        {"name": "product, one token", "op": "product", "b": 1, "K": 1, "E": 1, "N": 7168, "D": 3584, "group": 128,
         "local": 1.0, "skew": 0.0},
        # the down projections of 128 experts in a decode step with 64 tokens: a few rows for nearly every expert
        {"name": "product, experts decode", "op": "product", "b": 64, "K": 8, "E": 128, "N": 4096, "D": 1024, "group": 32,
         "local": 1.0, "skew": 0.0},
        # the same over prompts, about 256 rows for each expert, unevenly: tensor-core work
        {"name": "product, experts prompts", "op": "product", "b": 4096, "K": 8, "E": 128, "N": 4096, "D": 2048, "group": 128,
         "local": 1.0, "skew": 0.5},
        # gate and up of the 8 experts that one token goes to
        {"name": "gated, one token", "op": "gated", "b": 1, "K": 8, "E": 128, "N": 1024, "D": 4096, "group": 128,
         "local": 1.0, "skew": 0.0},
        # of 128 experts in a decode step with 64 tokens
        {"name": "gated, experts decode", "op": "gated", "b": 64, "K": 8, "E": 128, "N": 1024, "D": 4096, "group": 128,
         "local": 1.0, "skew": 0.0},
        # a shared expert's gate and up for a batch of 48 tokens
        {"name": "gated, dense batch", "op": "gated", "b": 48, "K": 1, "E": 1, "N": 6144, "D": 7168, "group": 32, "local": 1.0,
         "skew": 0.0},
        # prompts of odd lengths over 60 experts of odd sizes, half of them another GPU's
        {"name": "gated, experts prompts", "op": "gated", "b": 1999, "K": 6, "E": 60, "N": 1416, "D": 2056, "group": 64,
         "local": 0.5, "skew": 0.5},
        # the norms between two blocks for the one token of a single conversation
        {"name": "norm, one token", "op": "norm", "b": 1, "H": 7168, "post": True, "token": True, "channel": False},
        # over the tokens of a batch of prompts, with a gate for each channel
        {"name": "norm, prompts", "op": "norm", "b": 16384, "H": 4096, "post": True, "token": False, "channel": True},
        # the gradients for a small batch of odd length
        {"name": "gradient, small batch", "op": "gradient", "b": 333, "H": 3584, "post": True, "token": True, "channel": False},
        # over a training batch, all of them
        {"name": "gradient, training", "op": "gradient", "b": 8192, "H": 4096, "post": True, "token": True, "channel": True},
        # rows wider than a thread block holds, without a norm after the block
        {"name": "gradient, wide rows", "op": "gradient", "b": 1500, "H": 18432, "post": False, "token": False, "channel": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step))


def draw(rng):
    op = rng.choice(["product", "product", "gated", "gated", "norm", "gradient"])
    if op in ("product", "gated"):
        D, N, group = _spread(rng, 512, 4096, 8), _spread(rng, 256, 2048, 8), rng.choice([32, 64, 128])
        if rng.random() < 0.4:  # one dense weight
            return {"op": op, "b": _spread(rng, 1, 4096), "K": 1, "E": 1, "N": 2 * N, "D": D, "group": group, "local": 1.0,
                    "skew": 0.0}
        K = rng.choice([1, 2, 4, 6, 8])
        most = (1 << 37) // (N * D * K)  # tokens, for the largest listed product's cost
        return {"op": op, "b": _spread(rng, 1, min(most, 6000)), "K": K, "E": rng.choice([8, 60, 128]), "N": N,
                "D": D, "group": group, "local": rng.choice([1.0, 1.0, 0.5]), "skew": rng.choice([0.0, 0.5, 1.5])}
    H = _spread(rng, 256, 20000, 8)
    b = _spread(rng, 1, (16384 if op == "norm" else 8192) * 4096 // H)
    return {"op": op, "b": b, "H": H, "post": rng.random() < 0.75, "token": rng.random() < 0.5, "channel": rng.random() < 0.5}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _expert_offsets(g, b, K, E, local, skew):
    """[E + 1] int32: the places of the routes sorted by expert, K distinct experts for each of b tokens, the lower ones
    more likely with `skew`; a route is another GPU's with probability 1 - local."""
    scores = torch.empty((b, E), device="cuda").exponential_(generator=g).log_().neg_()
    scores -= skew * torch.log1p(torch.arange(E, device="cuda", dtype=F32))
    ids = scores.topk(K, dim=1).indices
    if local < 1.0:
        ids = torch.where(torch.rand((b, K), device="cuda", generator=g) >= local, E, ids)
    count = torch.bincount(ids.reshape(-1), minlength=E + 1)[:E]
    return torch.cat([count.new_zeros(1), count.cumsum(0)]).to(I32)


def _stored(g, E, channels, D):
    """Packed 4-bit weights [E, channels, 64 * ceil(D / 128)]: a normal distribution rounded to [-7, 7]."""
    blocks = -(-D // 128)
    out = torch.empty((E, channels, blocks * 64), dtype=torch.uint8, device="cuda")
    # a byte holds two columns of a word, one or the other nibble of four; the order within does not matter for random values
    for part in out.view(-1).split(1 << 27):
        low, high = (torch.empty(part.shape, dtype=BF16, device="cuda").normal_(0.0, 2.6, generator=g).round_().clamp_(-7, 7)
                     .add_(8).to(torch.uint8) for _ in range(2))
        part.copy_(low | (high << 4))
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, mean=0.0, scale=1.0):
        return torch.empty(shape, dtype=BF16, device="cuda").normal_(mean, scale, generator=g)

    def uniform(*shape, lo, hi):
        return torch.rand(shape, device="cuda", generator=g).mul_(hi - lo).add_(lo)

    def new(dtype, *shape):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    s = {"case": c}
    op, b = c["op"], c["b"]
    if op in ("product", "gated"):
        R, E, D = b * c["K"], c["E"], c["D"]
        channels = 2 * c["N"] if op == "gated" else c["N"]
        s["offsets"] = _expert_offsets(g, b, c["K"], E, c["local"], c["skew"])
        s["most"] = int(s["offsets"].diff().max())  # the plain form's padded batch
        # the rows of a norm, or what silu(gate) * up leaves
        s["x"] = normal(R, D) if op == "gated" else normal(R, D) * normal(R, D)
        s["w"] = _stored(g, E, channels, D)
        groups = -(-D // c["group"])
        scales = new(F32, E, channels, -(-groups // 4) * 4)
        scales[:, :, :groups] = torch.exp2(uniform(E, channels, groups, lo=5.5, hi=8.75))
        s["group_scale"] = scales.to(E4M3)
        s["channel_scale"] = uniform(E, channels, lo=0.5, hi=1.5).mul_(1.0 / (250.0 * math.sqrt(D)))
        s["out"] = new(BF16, R, c["N"])
        return s
    H = c["H"]
    s["x"], s["residual"] = normal(b, H, scale=0.7), normal(b, H, scale=3.0)
    s["post"] = normal(H, scale=0.1) if c["post"] else None
    s["pre"] = normal(H, scale=0.1)
    s["token"] = torch.sigmoid(normal(b).float()) if c["token"] else None
    s["channel"] = normal(H, mean=0.5, scale=0.1) if c["channel"] else None
    s["scale"] = 0.875
    if op == "norm":
        s["residual_out"], s["y"], s["rstd"] = new(BF16, b, H), new(BF16, b, H), new(F32, b, 2)
        return s
    s["rstd"] = torch.stack(_forward(s, F64)[2:], dim=1).to(F32)  # what the forward call has left
    s["d_y"], s["d_residual_out"] = normal(b, H), normal(b, H, scale=0.5)
    s["d_x"], s["d_residual"] = new(BF16, b, H), new(BF16, b, H)
    s["d_post"] = new(F32, H) if c["post"] else None
    s["d_pre"] = new(F32, H)
    s["d_token"] = new(F32, b) if c["token"] else None
    s["d_channel"] = new(F32, H) if c["channel"] else None
    s["workspace"] = torch.empty(12 * H * 512, dtype=torch.uint8, device="cuda")  # at least what the library asks for
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------


def _lib():
    import moe_decode_tail_gb300

    return moe_decode_tail_gb300


def _unpacked(w, D):
    """[E, channels, D] FP32: q of the stored weights."""
    E, channels, stored = w.shape
    words = w.view(I32).view(E, channels, stored // 64, 4, 4)          # block, t, i
    shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=I32, device=w.device)  # of column c of a word
    q = (words.transpose(3, 4).unsqueeze(-1) >> shifts) & 15           # block, i, t, c
    return q.reshape(E, channels, stored * 2)[:, :, :D].float().sub_(8.0)


def _weights(s):
    """[E, channels, D] FP32: the weights without their channels' scales."""
    c = s["case"]
    q = _unpacked(s["w"], c["D"])
    groups = -(-c["D"] // c["group"])
    return q.mul_(s["group_scale"][:, :, :groups].float().repeat_interleave(c["group"], 2)[:, :, :c["D"]])


def _products(s):
    """(places [E, most], products FP32 [E, most, channels]) of the rows by expert; places past an expert's rows point
    behind the last row."""
    first, count = s["offsets"][:-1].long(), s["offsets"].diff().long()
    column = torch.arange(s["most"], device="cuda")
    at = torch.where(column[None, :] < count[:, None], first[:, None] + column[None, :], s["x"].shape[0])
    padded = torch.nn.functional.pad(s["x"].float(), (0, 0, 0, 1))[at]
    return at, torch.bmm(padded, _weights(s).transpose(1, 2)) * s["channel_scale"][:, None, :]


def _placed(s, at, values):
    out = torch.zeros((s["x"].shape[0] + 1, s["case"]["N"]), dtype=BF16, device="cuda")
    out.index_copy_(0, at.reshape(-1), values.reshape(-1, s["case"]["N"]).to(BF16))
    return out[:-1]


def _product(s):
    c = s["case"]
    if own:
        return _lib().moe_tail_expert_product_i4(s["x"], s["w"], s["group_scale"], s["channel_scale"], s["out"],
                                                  group=c["group"], expert_offsets=s["offsets"] if c["E"] > 1 else None)
    return _placed(s, *_products(s))


def _gated(s):
    c = s["case"]
    if own:
        return _lib().moe_tail_gated_product_i4(s["x"], s["w"], s["group_scale"], s["channel_scale"], s["out"],
                                                 group=c["group"], expert_offsets=s["offsets"] if c["E"] > 1 else None)
    at, both = _products(s)
    gate, up = both.chunk(2, dim=2)
    return _placed(s, at, gate / (1.0 + torch.exp(-gate)) * up)


def _forward(s, dtype):
    """(h, y, 1 / rms of the block's output, 1 / rms of h) in `dtype`."""
    x = s["x"].to(dtype)
    first = torch.rsqrt(x.square().mean(1) + EPS)
    n = x if s["post"] is None else x * first[:, None] * (s["post"].to(dtype) + GAIN_CENTER)
    if s["token"] is not None:
        n = n * s["token"].to(dtype)[:, None]
    if s["channel"] is not None:
        n = n * s["channel"].to(dtype)
    h = s["scale"] * s["residual"].to(dtype) + n
    second = torch.rsqrt(h.square().mean(1) + EPS)
    return h, h * second[:, None] * (s["pre"].to(dtype) + GAIN_CENTER), first, second


def _gates(s):
    return {"token_gate": s["token"], "channel_gate": s["channel"], "residual_scale": s["scale"], "gain_center": GAIN_CENTER}


def _norm(s):
    if own:
        _lib().moe_tail_block_norm(s["x"], s["residual"], s["post"], s["pre"], s["residual_out"], s["y"], rstd=s["rstd"],
                                    eps=EPS, **_gates(s))
        return {"residual": s["residual_out"], "y": s["y"], "rstd": s["rstd"][:, 0 if s["post"] is not None else 1:]}
    h, y, first, second = _forward(s, F32)
    rstd = torch.stack([first, second], dim=1)
    return {"residual": h.to(BF16), "y": y.to(BF16), "rstd": rstd[:, 0 if s["post"] is not None else 1:]}


def _gradient(s):
    if own:
        _lib().moe_tail_block_norm_grad(s["d_y"], s["d_residual_out"], s["x"], s["residual"], s["post"], s["pre"], s["rstd"],
                                         s["d_x"], s["d_residual"], s["workspace"], d_post_gamma=s["d_post"],
                                         d_pre_gamma=s["d_pre"], d_token_gate=s["d_token"], d_channel_gate=s["d_channel"],
                                         **_gates(s))
        return {k: s[k] for k in ("d_x", "d_residual", "d_post", "d_pre", "d_token", "d_channel") if s[k] is not None}
    x, first, second = s["x"].float(), s["rstd"][:, :1], s["rstd"][:, 1:]
    token = None if s["token"] is None else s["token"][:, None]
    channel = None if s["channel"] is None else s["channel"].float()
    unit = x * first if s["post"] is not None else x
    n = unit * (s["post"].float() + GAIN_CENTER) if s["post"] is not None else x
    gate = (1.0 if token is None else token) * (1.0 if channel is None else channel)
    h = s["scale"] * s["residual"].float() + gate * n
    out = {}
    hat = h * second
    d_y = s["d_y"].float()
    d_hat = d_y * (s["pre"].float() + GAIN_CENTER)
    d_h = s["d_residual_out"].float() + second * (d_hat - hat * (d_hat * hat).mean(1, keepdim=True))
    d_n = gate * d_h
    if s["post"] is not None:
        d_unit = d_n * (s["post"].float() + GAIN_CENTER)
        out["d_x"] = (first * (d_unit - unit * (d_unit * unit).mean(1, keepdim=True))).to(BF16)
        out["d_post"] = (d_n * unit).sum(0)
    else:
        out["d_x"] = d_n.to(BF16)
    out["d_residual"] = (s["scale"] * d_h).to(BF16)
    out["d_pre"] = (d_y * hat).sum(0)
    if token is not None:
        out["d_token"] = (d_h * n * (1.0 if channel is None else channel)).sum(1)
    if channel is not None:
        out["d_channel"] = (d_h * n * (1.0 if token is None else token)).sum(0)
    return {k: out[k] for k in ("d_x", "d_residual", "d_post", "d_pre", "d_token", "d_channel") if k in out}


def run(state):
    return {"product": _product, "gated": _gated, "norm": _norm, "gradient": _gradient}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------


def work(case):
    c = case
    op, b = c["op"], c["b"]
    if op in ("product", "gated"):
        channels = 2 * c["N"] if op == "gated" else c["N"]
        live = b * c["K"] * c["local"]  # expected
        hit = c["E"] * (1.0 - (1.0 - c["K"] * c["local"] / c["E"]) ** b) if c["E"] > 1 else 1  # experts with a row
        weight = channels * (c["D"] / 2 + -(-c["D"] // c["group"]) + 4)
        return {"bytes": hit * weight + 2 * live * (c["D"] + c["N"]), "flops": 2.0 * live * channels * c["D"]}
    n = b * c["H"]
    sums = 2 if c["post"] else 1
    token = 4 * b if c["token"] else 0
    vectors = 2 * c["H"] * (1 + c["post"] + c["channel"])
    if op == "norm":
        return {"bytes": 8 * n + 4 * b * sums + token + vectors, "flops": (7 + 4 * c["post"]) * n}
    return {"bytes": 12 * n + 8 * b + 2 * token + 3 * vectors, "flops": (16 + 8 * c["post"] + 2 * (c["token"] + c["channel"])) * n}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------


def _exact_weight(s, e):
    """[channels, D] FP64 of expert e, from the layout's definition, one column of a word at a time."""
    c = s["case"]
    stored = s["w"][e].to(torch.int64).view(s["w"].shape[1], -1, 16, 4)  # block, word, byte
    word = stored[..., 0] + stored[..., 1] * 256 + stored[..., 2] * 65536 + stored[..., 3] * 16777216
    full = torch.empty((word.shape[0], word.shape[1] * 128), dtype=F64, device="cuda")
    blocks = full.view(word.shape[0], word.shape[1], 128)
    for t in range(4):
        for i in range(4):
            for col in range(8):
                nibble = col // 2 if col % 2 == 0 else 4 + col // 2
                blocks[:, :, 32 * i + 8 * t + col] = (torch.div(word[:, :, 4 * t + i], 16 ** nibble, rounding_mode="floor") % 16 - 8).to(F64)
    w = full[:, :c["D"]].clone()
    for first in range(0, c["D"], c["group"]):
        w[:, first:first + c["group"]] *= s["group_scale"][e, :, first // c["group"], None].to(F64)
    return w * s["channel_scale"][e, :, None].to(F64)


def exact(case, seed):
    c = case
    op = c["op"]
    s = prepare(case, seed)
    if op in ("product", "gated"):
        out = torch.zeros(s["out"].shape, dtype=F64, device="cuda")
        ends = s["offsets"].tolist()
        for e in range(c["E"]):
            i, j = ends[e], ends[e + 1]
            if j > i:
                d = s["x"][i:j].to(F64) @ _exact_weight(s, e).T
                if op == "gated":
                    d = d[:, :c["N"]] * torch.sigmoid(d[:, :c["N"]]) * d[:, c["N"]:]
                out[i:j] = d
        return out
    # the norms and, by the chain rule, their gradients: a function of the inputs, differentiated a few rows at a time
    rows = max(1, (1 << 24) // c["H"])
    parts = []
    sums = {}
    for i in range(0, c["b"], rows):
        j = min(c["b"], i + rows)
        x, r = s["x"][i:j].to(F64), s["residual"][i:j].to(F64)
        post = None if s["post"] is None else s["post"].to(F64)
        pre = s["pre"].to(F64)
        token = None if s["token"] is None else s["token"][i:j].to(F64)
        channel = None if s["channel"] is None else s["channel"].to(F64)
        leaves = {"d_x": x, "d_residual": r, "d_post": post, "d_pre": pre, "d_token": token, "d_channel": channel}
        leaves = {k: v.requires_grad_(op == "gradient") for k, v in leaves.items() if v is not None}
        root1 = torch.sqrt((x ** 2).sum(1, keepdim=True) / c["H"] + EPS)
        n = x if post is None else x / root1 * (GAIN_CENTER + post)
        n = n if token is None else token[:, None] * n
        n = n if channel is None else n * channel[None, :]
        h = n + r * s["scale"]
        root2 = torch.sqrt((h ** 2).sum(1, keepdim=True) / c["H"] + EPS)
        y = h / root2 * (GAIN_CENTER + pre)
        if op == "norm":
            rstd = torch.cat([1.0 / root1, 1.0 / root2] if post is not None else [1.0 / root2], dim=1)
            parts.append({"residual": h, "y": y, "rstd": rstd})
            continue
        grads = torch.autograd.grad([h, y], list(leaves.values()), [s["d_residual_out"][i:j].to(F64), s["d_y"][i:j].to(F64)])
        got = dict(zip(leaves, grads))
        parts.append({k: v for k, v in got.items() if k in ("d_x", "d_residual", "d_token")})
        for k in ("d_post", "d_pre", "d_channel"):
            if k in got:
                sums[k] = sums.get(k, 0) + got[k]
    joined = {k: torch.cat([p[k] for p in parts]) for k in parts[0]} | sums
    return {k: joined[k] for k in ("residual", "y", "rstd", "d_x", "d_residual", "d_post", "d_pre", "d_token", "d_channel") if k in joined}
