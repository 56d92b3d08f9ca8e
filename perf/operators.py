"""Workloads of the operators around the decode tail: what a Mixture-of-Experts layer with 8-bit experts does
before and after the finalize calls.

    norm       residual addition, RMS norm, 8-bit rows with scales           moe_tail_norm_quant
    silu       silu(gate) * up in 8-bit rows with scales                     moe_tail_silu_quant
    dispatch   routes sorted by expert, the tokens' rows copied in order     moe_tail_sort_routes, moe_tail_dispatch_rows
    combine    route rows weighted and summed per token, and the gradients   moe_tail_combine_rows, moe_tail_combine_grad
    product    8-bit integer product, a scale per row and per channel        moe_tail_expert_product

Each case has a plain form (elementary torch operations in 32 bits) and, with `own` set, the library's calls.  Rows in
8 bits are returned as the BF16 values they stand for, by the same torch operation in both forms.
"""
import math

import torch

own = False

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
KINDS = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
GAIN_CENTER, EPS = 1.0, 1e-6


def listed():
    return [
        # the residual and norm between two layers for the one token of a single conversation: a latency
        {"name": "norm, one token", "op": "norm", "b": 1, "H": 7168, "kind": "int8", "group": 0},
        # the same over the tokens of a batch of prompts: bandwidth
        {"name": "norm, prompts", "op": "norm", "b": 16384, "H": 4096, "kind": "int8", "group": 0},
        # between an expert's two products, for the 512 routes of a decode step with 64 tokens
        {"name": "silu, decode", "op": "silu", "b": 64, "K": 8, "E": 128, "I": 1024, "kind": "int8", "group": 0,
         "local": 1.0, "skew": 0.0},
        # over prompts, e4m3 with a scale for every 128 columns; an eighth of the routes are another GPU's
        {"name": "silu, prompts", "op": "silu", "b": 4096, "K": 8, "E": 128, "I": 2048, "kind": "e4m3", "group": 128,
         "local": 0.875, "skew": 0.5},
        # a decode step's routes sorted, and its 8-bit rows with their scales copied into the experts' order
        {"name": "dispatch, decode", "op": "dispatch", "b": 64, "K": 8, "E": 128, "H": 4096, "kind": "int8",
         "local": 1.0, "skew": 0.0},
        # a training batch's, in BF16
        {"name": "dispatch, training", "op": "dispatch", "b": 8192, "K": 8, "E": 128, "H": 4096, "kind": "bf16",
         "local": 1.0, "skew": 0.5},
        # the weighted sum of a decode step's route rows
        {"name": "combine, decode", "op": "combine", "b": 64, "K": 8, "E": 128, "H": 4096, "weights": "f32",
         "local": 1.0, "skew": 0.0},
        # the dispatch's gradient (unit weights) for an odd batch, some routes on another GPU
        {"name": "combine, dispatch gradient", "op": "combine", "b": 8191, "K": 16, "E": 256, "H": 3584, "weights": "none",
         "local": 0.5, "skew": 0.0},
        # the gradients of the weighted sum over a training batch
        {"name": "combine gradients, training", "op": "gradient", "b": 4096, "K": 8, "E": 128, "H": 4096, "weights": "f32",
         "local": 1.0, "skew": 0.5},
        # one dense 8-bit weight with the tokens of a small decode batch: weight streaming on few tiles
        {"name": "product, dense decode", "op": "product", "b": 8, "K": 1, "E": 1, "N": 7168, "D": 3584, "local": 1.0,
         "skew": 0.0},
        # the gate and up weights of 128 experts in a decode step with 64 tokens: nearly every expert has a few rows
        {"name": "product, experts decode", "op": "product", "b": 64, "K": 8, "E": 128, "N": 2048, "D": 4096, "local": 1.0,
         "skew": 0.0},
        # the same over prompts: about 256 rows for each expert, unevenly: tensor-core work
        {"name": "product, experts prompts", "op": "product", "b": 4096, "K": 8, "E": 128, "N": 2048, "D": 4096,
         "local": 1.0, "skew": 0.5},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    n = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step))
    return n if n != 3072 else n + step  # in no configuration of this library


def draw(rng):
    op = rng.choice(["norm", "silu", "dispatch", "combine", "gradient", "product", "product"])
    E = rng.choice([8, 60, 128, 256])
    routing = {"K": rng.choice([1, 2, 4, 6, 8]), "E": E, "local": rng.choice([1.0, 1.0, 0.875, 0.25]),
               "skew": rng.choice([0.0, 0.5, 1.5])}
    kind, group = rng.choice([("int8", 0), ("int8", 128), ("e4m3", 0), ("e4m3", 128)])
    if op == "norm":
        H = _spread(rng, 512, 8192, 8)
        return {"op": op, "b": _spread(rng, 1, 16384 * 4096 // H), "H": H, "kind": kind, "group": group}
    if op == "silu":
        I = _spread(rng, 256, 8192, 8)
        return {"op": op, "b": _spread(rng, 1, 2048 * 4096 // I), "I": I, "kind": kind, "group": group, **routing}
    if op == "product":
        D, N = _spread(rng, 512, 4096, 16), _spread(rng, 512, 2048, 8)
        if rng.random() < 0.4:  # one dense weight
            return {"op": op, "b": _spread(rng, 1, 8192), "K": 1, "E": 1, "N": 4 * N, "D": D, "local": 1.0, "skew": 0.0}
        return {"op": op, "b": _spread(rng, 1, 4096), "N": N, "D": D, **routing}
    H = _spread(rng, 512, 7168, 16)
    b = _spread(rng, 1, 4096 * 4096 // H)
    if op == "dispatch":
        return {"op": op, "b": b, "H": H, "kind": rng.choice(["int8", "e4m3", "bf16"]), **routing}
    return {"op": op, "b": b, "H": H, "weights": rng.choice(["f32", "bf16", "none"] if op == "combine" else ["f32", "bf16"]),
            **routing}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _expert_ids(g, b, K, E, local, skew):
    """[b, K] int32: distinct experts for each token, the lower ones more likely with `skew`; a route is -1 (another
    GPU's expert) with probability 1 - local."""
    scores = torch.empty((b, E), device="cuda").exponential_(generator=g).log_().neg_()
    scores -= skew * torch.log1p(torch.arange(E, device="cuda", dtype=F32))
    ids = scores.topk(K, dim=1).indices.to(I32)
    if local < 1.0:
        ids[torch.rand((b, K), device="cuda", generator=g) >= local] = -1
    return ids


def _sorted_routes(ids, E):
    """The routes in the order of (expert, route number): expert_offsets [E + 1], permuted_idx [b, K] (a route's place,
    -1 without one), source [b * K] (the route at a place, -1 past the last)."""
    flat = ids.reshape(-1)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    place = torch.arange(n, device=flat.device)
    inverse = torch.empty_like(order).scatter_(0, order, place)
    offsets = (key[None, :] < torch.arange(E + 1, device=flat.device)[:, None]).sum(1)
    permuted_idx = torch.where(key < E, inverse, -1).reshape(ids.shape)
    source = torch.where(place < offsets[E], order, -1)
    return offsets.to(I32), permuted_idx.to(I32), source.to(I32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.empty(shape, dtype=BF16, device="cuda").normal_(0.0, scale, generator=g)

    def eight_bit(*shape):
        t = torch.empty(shape, dtype=torch.int8, device="cuda")
        for part in t.view(-1).split(1 << 28):  # values of a quantised normal distribution
            part.copy_(torch.empty(part.shape, dtype=BF16, device="cuda").normal_(0.0, 36.0, generator=g).round_().clamp_(-127, 127))
        return t

    def positive(*shape, scale):
        return torch.rand(shape, device="cuda", generator=g).mul_(scale).add_(0.5 * scale)

    def new(dtype, *shape):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    s = {"case": c}
    op, b = c["op"], c["b"]
    if "K" in c:
        R = b * c["K"]
        ids = _expert_ids(g, b, c["K"], c["E"], c["local"], c["skew"])
        offsets, permuted_idx, _ = _sorted_routes(ids, c["E"])
    if op in ("norm", "silu"):
        rows, width = (b, c["H"]) if op == "norm" else (R, c["I"])
        groups = (rows, -(-width // c["group"])) if c["group"] else (rows,)
        s["q"], s["scale"] = new(KINDS[c["kind"]][0], rows, width), new(F32, *groups)
        s["values"] = new(BF16, rows, width)
    if op == "norm":
        s["x"], s["residual"], s["gamma"] = normal(b, c["H"]), normal(b, c["H"], scale=4.0), normal(c["H"], scale=0.1)
        s["residual_out"] = new(BF16, b, c["H"])
    elif op == "silu":
        s["gate_up"], s["used"] = normal(R, 2 * c["I"], scale=2.0), offsets[c["E"]:]
    elif op == "dispatch":
        s["ids"] = ids
        if c["kind"] == "bf16":
            s["x"], s["scale"], s["row_scale"] = normal(b, c["H"]), None, None
        else:
            s["x"] = eight_bit(b, c["H"]) if c["kind"] == "int8" else normal(b, c["H"], scale=100.0).clamp_(-448, 448).to(KINDS["e4m3"][0])
            s["scale"], s["row_scale"] = positive(b, scale=0.02), new(F32, R)
        s["offsets"], s["permuted_idx"], s["source"] = new(I32, c["E"] + 1), new(I32, b, c["K"]), new(I32, R)
        s["rows"], s["values"] = new(s["x"].dtype, R, c["H"]), new(BF16, R, c["H"])
        s["workspace"] = new(torch.uint8, 4096 + 4 * c["E"] * (R // 512 + 2))  # at least what the library asks for
    elif op in ("combine", "gradient"):
        s["idx"], s["rows"] = permuted_idx, normal(R, c["H"])
        if c["weights"] == "none":
            s["w"] = None
        else:
            w = torch.softmax(torch.empty((b, c["K"]), device="cuda").normal_(generator=g), dim=1)
            s["w"] = w if c["weights"] == "f32" else w.to(BF16)
        if op == "combine":
            s["out"] = new(BF16, b, c["H"])
        else:
            s["d_out"], s["d_rows"], s["d_w"] = normal(b, c["H"]), new(BF16, R, c["H"]), new(F32, b, c["K"])
    else:
        s["x"], s["x_scale"] = eight_bit(R, c["D"]), positive(R, scale=0.02)
        s["w"], s["w_scale"] = eight_bit(c["E"], c["N"], c["D"]), positive(c["E"], c["N"], scale=0.0005)
        s["offsets"], s["out"] = offsets, new(BF16, R, c["N"])
        s["most"] = int((offsets[1:] - offsets[:-1]).max())  # the plain form's padded batch
        s["workspace"] = new(torch.uint8, 2 * (R + 256) * (c["D"] + 64) + (64 << 20))  # at least what the library asks for
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------


def _lib():
    import moe_decode_tail_gb300

    return moe_decode_tail_gb300


def _columns(scale, group, width):
    """[rows, width] or [rows, 1]: the scale of every column."""
    return scale.repeat_interleave(group, 1)[:, :width] if group else scale[:, None]


def _stand_for(s):
    """The BF16 values that the state's 8-bit rows stand for."""
    q, c = s["q"], s["case"]
    q = q if q.dtype == torch.int8 else q.to(BF16)
    return torch.mul(q, _columns(s["scale"], c["group"], q.shape[1]), out=s["values"])


def _quantise(s, y, live=None):
    """The plain 8-bit form of y (FP32 [rows, width]) into the state's q and scale; rows not `live` stay as they are."""
    c = s["case"]
    dtype, most = KINDS[c["kind"]]
    rows, width = y.shape
    if c["group"]:
        padded = torch.nn.functional.pad(y.abs(), (0, -width % c["group"]))
        top = padded.view(rows, -1, c["group"]).amax(2)
    else:
        top = y.abs().amax(1)
    scale = top / most
    step = _columns(scale, c["group"], width)
    q = torch.where(step > 0, y / step, 0.0).clamp(-most, most)
    q = (torch.round(q) if dtype == torch.int8 else q).to(dtype)
    if live is not None:
        q = torch.where(live[:, None], q.to(BF16), 0.0).to(dtype)
        scale = torch.where(live[:, None] if c["group"] else live, scale, 0.0)
    s["q"].copy_(q)
    s["scale"].copy_(scale)


def _norm(s):
    if own:
        _lib().moe_tail_norm_quant(s["x"], s["residual"], s["gamma"], s["q"], s["scale"], residual_out=s["residual_out"],
                                    gain_center=GAIN_CENTER, eps=EPS, group=s["case"]["group"])
        return {"residual": s["residual_out"], "scale": s["scale"], "values": _stand_for(s)}
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * (s["gamma"].float() + GAIN_CENTER)
    _quantise(s, y)
    return {"residual": h.to(BF16), "scale": s["scale"], "values": _stand_for(s)}


def _silu(s):
    if own:
        _lib().moe_tail_silu_quant(s["gate_up"], s["q"], s["scale"], used_rows=s["used"], group=s["case"]["group"])
    else:
        gate, up = s["gate_up"].float().chunk(2, dim=1)
        live = torch.arange(gate.shape[0], device=gate.device) < s["used"]
        _quantise(s, gate / (1.0 + torch.exp(-gate)) * up, live)
    return {"scale": s["scale"], "values": _stand_for(s)}


def _dispatch(s):
    c = s["case"]
    if own:
        mt = _lib()
        mt.moe_tail_sort_routes(s["ids"], s["offsets"], s["permuted_idx"], s["source"], s["workspace"])
        mt.moe_tail_dispatch_rows(s["x"], s["permuted_idx"], s["rows"], scale=s["scale"], row_scale=s["row_scale"])
        offsets, permuted_idx, source, rows, row_scale = s["offsets"], s["permuted_idx"], s["source"], s["rows"], s["row_scale"]
    else:
        offsets, permuted_idx, source = _sorted_routes(s["ids"], c["E"])
        token = source.clamp_min(0).long() // c["K"]
        live = source >= 0
        x = s["x"].view(torch.int16 if c["kind"] == "bf16" else torch.int8)
        rows = torch.where(live[:, None], x[token], 0).view(s["x"].dtype)
        row_scale = None if s["scale"] is None else torch.where(live, s["scale"][token], 0.0)
    if row_scale is not None:  # the values that the 8-bit rows stand for
        rows = torch.mul(rows if rows.dtype == torch.int8 else rows.to(BF16), row_scale[:, None], out=s["values"])
    return {"offsets": offsets, "permuted_idx": permuted_idx, "source": source, "row_scale": row_scale, "rows": rows}


def _combine(s):
    if own:
        return _lib().moe_tail_combine_rows(s["rows"], s["idx"], s["w"], s["out"])
    live = s["idx"] >= 0
    picked = s["rows"][s["idx"].clamp_min(0).long()].float()
    w = live.float() if s["w"] is None else torch.where(live, s["w"].float(), 0.0)
    return (picked * w[:, :, None]).sum(1).to(BF16)


def _gradient(s):
    if own:
        _lib().moe_tail_combine_grad(s["d_out"], s["rows"], s["idx"], s["w"], s["d_rows"], s["d_w"])
        return {"d_rows": s["d_rows"], "d_w": s["d_w"]}
    live = s["idx"] >= 0
    place = s["idx"].clamp_min(0).long()
    d = s["d_out"].float()
    d_w = torch.where(live, (s["rows"][place].float() * d[:, None, :]).sum(2), 0.0)
    # the route at every place, to write each row once
    route = torch.full((s["rows"].shape[0] + 1,), -1, dtype=torch.long, device=d.device)
    route.scatter_(0, torch.where(live, place, s["rows"].shape[0]).reshape(-1),
                   torch.arange(place.numel(), device=d.device))
    route = route[:-1]
    w = torch.where(route >= 0, s["w"].float().reshape(-1)[route.clamp_min(0)], 0.0)
    d_rows = d[route.clamp_min(0) // s["idx"].shape[1]] * w[:, None]
    return {"d_rows": d_rows.to(BF16), "d_w": d_w}


def _product(s):
    c = s["case"]
    if own:
        return _lib().moe_tail_expert_product(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], s["workspace"],
                                               expert_offsets=s["offsets"] if c["E"] > 1 else None)
    first, count = s["offsets"][:-1].long(), s["offsets"].diff().long()
    column = torch.arange(s["most"], device="cuda")
    inside = column[None, :] < count[:, None]
    at = torch.where(inside, first[:, None] + column[None, :], s["x"].shape[0])  # past the rows: the padding
    padded = torch.nn.functional.pad(s["x"].float(), (0, 0, 0, 1))[at]
    scale = torch.nn.functional.pad(s["x_scale"], (0, 1))[at]
    d = torch.bmm(padded, s["w"].float().transpose(1, 2)) * scale[:, :, None] * s["w_scale"][:, None, :]
    out = torch.zeros((s["x"].shape[0] + 1, c["N"]), dtype=BF16, device="cuda")
    out.index_copy_(0, at.reshape(-1), d.reshape(-1, c["N"]).to(BF16))
    return out[:-1]


def run(state):
    return {"norm": _norm, "silu": _silu, "dispatch": _dispatch, "combine": _combine, "gradient": _gradient,
            "product": _product}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------


def work(case):
    c = case
    op, b = c["op"], c["b"]
    if op == "norm":
        n = b * c["H"]
        scales = 4 * b * (-(-c["H"] // c["group"]) if c["group"] else 1)
        # x and residual read, the new residual, the 8-bit row and its values written, the 8-bit row read for them
        return {"bytes": n * (2 + 2 + 2 + 1 + 1 + 2) + 2 * scales + 2 * c["H"], "flops": 8 * n}
    live = b * c["K"] * c["local"]  # expected
    if op == "silu":
        scales = 4 * live * (-(-c["I"] // c["group"]) if c["group"] else 1)
        return {"bytes": live * c["I"] * (4 + 1 + 1 + 2) + 2 * scales, "flops": 10 * live * c["I"]}
    if op == "dispatch":
        size = 2 if c["kind"] == "bf16" else 1
        # the rows are copied as they are, and read and written again as BF16 numbers where they are 8 bits wide
        again = 0 if c["kind"] == "bf16" else b * c["K"] * c["H"] * 3
        return {"bytes": size * c["H"] * (b + live) + again + 12 * b * c["K"] + 4 * (b + live), "flops": b * c["K"]}
    size = 0 if c.get("weights") == "none" else 2 if c.get("weights") == "bf16" else 4
    if op == "combine":
        return {"bytes": 2 * c["H"] * (live + b) + b * c["K"] * (4 + size), "flops": 2 * live * c["H"]}
    if op == "gradient":
        return {"bytes": 2 * c["H"] * (2 * live + b) + b * c["K"] * (4 + size + 4), "flops": 3 * live * c["H"]}
    hit = c["E"] * (1.0 - (1.0 - c["K"] * c["local"] / c["E"]) ** b) if c["E"] > 1 else 1  # experts with a row
    return {"bytes": hit * c["N"] * (c["D"] + 4) + live * (c["D"] + 4 + 2 * c["N"]), "flops": 2.0 * live * c["N"] * c["D"]}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------


def _exact_quantised(y, kind, group):
    """(values, scales) of y (FP64) in 8 bits, from the definition."""
    most = KINDS[kind][1]
    width = y.shape[1]
    size = group or width
    parts = [y[:, i:i + size] for i in range(0, width, size)]
    scales = torch.stack([p.abs().max(dim=1).values / most for p in parts], dim=1)
    values = []
    for p, sc in zip(parts, scales.unbind(1)):
        ratio = p / sc.clamp_min(1e-300)[:, None]
        if kind == "int8":
            rounded = ratio.round()
        else:  # three bits after the leading one, down to 2^-9
            exponent = torch.floor(torch.log2(ratio.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
            unit = torch.exp2(exponent - 3.0)
            rounded = (ratio / unit).round() * unit
        values.append(rounded * sc[:, None])
    return torch.cat(values, dim=1), scales if group else scales[:, 0]


def _in_chunks(fn, rows, cost):
    """fn(first, last) over row ranges of at most 2^26 values, its results joined."""
    step = max(1, (1 << 26) // cost)
    parts = [fn(i, min(rows, i + step)) for i in range(0, rows, step)]
    return [torch.cat(p) for p in zip(*parts)]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op, b = c["op"], c["b"]
    f64 = torch.float64
    if op == "norm":
        def part(i, j):
            h = s["x"][i:j].to(f64) + s["residual"][i:j].to(f64)
            root = torch.sqrt((h * h).sum(1) / c["H"] + EPS)
            values, scales = _exact_quantised(h / root[:, None] * (s["gamma"].to(f64) + GAIN_CENTER), c["kind"], c["group"])
            return h, scales, values

        h, scales, values = _in_chunks(part, b, c["H"])
        return {"residual": h, "scale": scales, "values": values}
    if op == "silu":
        used = int(s["used"][0])

        def part(i, j):
            gate, up = s["gate_up"][i:j, :c["I"]].to(f64), s["gate_up"][i:j, c["I"]:].to(f64)
            values, scales = _exact_quantised(gate * torch.sigmoid(gate) * up, c["kind"], c["group"])
            values[max(0, used - i):] = 0
            scales[max(0, used - i):] = 0
            return scales, values

        scales, values = _in_chunks(part, s["gate_up"].shape[0], 2 * c["I"])
        return {"scale": scales, "values": values}
    if op == "dispatch":
        lists = [[] for _ in range(c["E"])]
        for route, e in enumerate(s["ids"].reshape(-1).tolist()):
            if e >= 0:
                lists[e].append(route)
        order = torch.tensor([r for one in lists for r in one], dtype=torch.long, device="cuda")
        rows = torch.zeros(s["rows"].shape, dtype=f64, device="cuda")
        rows[:len(order)] = s["x"].to(F32)[order // c["K"]].to(f64)
        row_scale = None
        if s["scale"] is not None:
            row_scale = torch.zeros(rows.shape[0], dtype=f64, device="cuda")
            row_scale[:len(order)] = s["scale"][order // c["K"]].to(f64)
            rows *= row_scale[:, None]
        return {"offsets": None, "permuted_idx": None, "source": None, "row_scale": row_scale, "rows": rows}
    if op in ("combine", "gradient"):
        w = torch.ones((b, c["K"]), dtype=f64, device="cuda") if s["w"] is None else s["w"].to(f64)
        if op == "combine":
            out = torch.zeros((b, c["H"]), dtype=f64, device="cuda")
            for k in range(c["K"]):
                t = torch.nonzero(s["idx"][:, k] >= 0)[:, 0]
                out[t] += w[t, k, None] * s["rows"][s["idx"][t, k].long()].to(f64)
            return out
        d_rows = torch.zeros(s["rows"].shape, dtype=f64, device="cuda")
        d_w = torch.zeros((b, c["K"]), dtype=f64, device="cuda")
        for k in range(c["K"]):
            t = torch.nonzero(s["idx"][:, k] >= 0)[:, 0]
            place = s["idx"][t, k].long()
            d_rows[place] = w[t, k, None] * s["d_out"][t].to(f64)
            d_w[t, k] = torch.einsum("th,th->t", s["d_out"][t].to(f64), s["rows"][place].to(f64))
        return {"d_rows": d_rows, "d_w": d_w}
    if 2.0 * b * c["K"] * c["N"] * c["D"] > 1e13:  # over about 20 seconds of FP64
        return None
    out = torch.zeros((b * c["K"], c["N"]), dtype=f64, device="cuda")
    ends = s["offsets"].tolist()
    for e in range(c["E"]):
        i, j = ends[e], ends[e + 1]
        if j > i:
            d = s["x"][i:j].to(f64) @ s["w"][e].to(f64).T
            out[i:j] = d * s["x_scale"][i:j].to(f64)[:, None] * s["w_scale"][e].to(f64)[None, :]
    return out
