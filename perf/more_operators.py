"""What is measured of decoding and training through the expert layer: cases, inputs, plain forms and 64-bit values.

The operators: the whole mixture-of-experts layer for a few tokens; the norm after a block joined, with
its gate and the scaled residual, to the norm before the next block, and the gradient of that; SwiGLU that keeps
its input in 8 bits, and its gradient from there; the weights' gradient from rows kept in 8 bits.

`run` computes a case with elementary torch operations in FP32 where `own` is false and with the
package's operators where it is true.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
HALF = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # one decoded token through its eight experts: latency and the weights' bytes
        {"name": "few_token", "op": "few", "rows": 1, "topk": 8, "experts": 32, "all_experts": 32, "hidden": 7168,
         "inner": 2048, "x": "fp8", "dtype": "bf16", "dropped": 0.0},
        # a small speculative batch of 16-bit rows with sizes that end inside blocks, some slots dropped
        {"name": "few_ragged", "op": "few", "rows": 13, "topk": 6, "experts": 24, "all_experts": 24, "hidden": 2064,
         "inner": 1040, "x": "fp16", "dtype": "fp16", "dropped": 0.125},
        # a decode step's tokens on one of eight ranks: 32 of 256 experts live here
        {"name": "few_batch", "op": "few", "rows": 64, "topk": 8, "experts": 32, "all_experts": 256, "hidden": 7168,
         "inner": 2048, "x": "fp8", "dtype": "bf16", "dropped": 0.0},
        # one decoded token after the experts, gated by its router, ahead of the next FP8 dispatch: latency alone
        {"name": "join_token", "op": "join", "rows": 1, "hidden": 7168, "dtype": "bf16", "gate": "row", "fp8": True},
        # every token of eight ranks at 4096 tokens per rank: the prefill join with a learned gate per channel
        {"name": "join_prefill", "op": "join", "rows": 32768, "hidden": 7168, "dtype": "bf16", "gate": "channel",
         "fp8": True},
        # training, ragged: gates per element, 16-bit norms
        {"name": "join_backward_ragged", "op": "join_backward", "rows": 1021, "hidden": 2064, "dtype": "fp16",
         "gate": "element", "fp8": False},
        # training: a step's tokens, gradients of both norms' weights and of the channels' gate
        {"name": "join_backward_train", "op": "join_backward", "rows": 8192, "hidden": 7168, "dtype": "bf16",
         "gate": "channel", "fp8": False},
        # training: the activation between the projections of one rank's experts, its input kept in 8 bits
        {"name": "swiglu_train", "op": "swiglu", "rows": 32768, "inner": 2048, "dtype": "bf16", "fp8": False},
        # training, ragged: the gradient of it where blocks of gate and up straddle
        {"name": "swiglu_backward_ragged", "op": "swiglu_backward", "rows": 777, "inner": 1040, "dtype": "fp16",
         "fp8": False},
        # training: the gradient of it, also as FP8 rows for the product with the transposed weights
        {"name": "swiglu_backward_train", "op": "swiglu_backward", "rows": 32768, "inner": 2048, "dtype": "bf16",
         "fp8": True},
        # ragged groups, columns that fill no tile
        {"name": "weights_ragged", "op": "weights", "rows": 1777, "inner": 1040, "columns": 520, "groups": 6,
         "dtype": "fp16"},
        # training: the first projection's gradient of one rank's 32 experts
        {"name": "weights_train", "op": "weights", "rows": 32768, "inner": 7168, "columns": 4096, "groups": 32,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _odd(rng, lo, hi):
    """An odd whole number of lo..hi, spread over the logarithm."""
    return min(hi, int(_log(rng, lo, hi))) // 2 * 2 + 1


def _size(rng, lo, hi, step):
    """A width: one of the common ones, or an odd multiple of step, spread over the logarithm."""
    if rng.random() < 0.4:
        return rng.choice([v for v in (256, 512, 1024, 2048, 4096, 7168) if lo <= v <= hi])
    return _odd(rng, max(1, lo // step), hi // step - 1) * step


def draw(rng):
    op = rng.choice(["few", "few", "join", "join_backward", "swiglu", "swiglu_backward", "weights", "weights"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "few":
        experts, topk = int(_log(rng, 4, 32)), rng.choice([1, 2, 4, 6, 8])
        ranks = rng.choice([1, 1, 4, 8]) if experts >= 8 else 1
        return {"op": op, "rows": _odd(rng, 1, 62), "topk": min(topk, experts * ranks), "experts": experts,
                "all_experts": experts * ranks, "hidden": _size(rng, 256, 7168, 16), "inner": _size(rng, 256, 2048, 16),
                "x": rng.choice(["fp8", "fp8", dtype]), "dtype": dtype, "dropped": rng.choice([0.0, 0.05, 0.25])}
    if op in ("join", "join_backward"):
        fp8 = op == "join" and rng.random() < 0.6
        return {"op": op, "rows": _odd(rng, 1, 16384 if op == "join" else 8190), "hidden": _size(rng, 256, 7168, 16),
                "dtype": dtype, "gate": rng.choice(["none", "row", "channel", "element"]), "fp8": fp8}
    if op in ("swiglu", "swiglu_backward"):
        return {"op": op, "rows": _odd(rng, 1, 32766), "inner": _size(rng, 256, 2048, 16), "dtype": dtype,
                "fp8": op == "swiglu_backward" and rng.random() < 0.5}
    return {"op": op, "rows": _odd(rng, 16, 16384), "inner": _size(rng, 256, 7168, 16),
            "columns": _size(rng, 136, 4096, 8), "groups": rng.choice([0, int(_log(rng, 2, 24)), int(_log(rng, 2, 24))]),
            "dtype": dtype}


# ------------------------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // 128)


def _quantise(y):
    """e4m3 codes and FP32 scales (one per 128 elements of a row) of FP32 rows."""
    n, width = y.shape
    blocks = torch.nn.functional.pad(y, (0, _blocks(width) * 128 - width)).view(n, -1, 128)
    top = blocks.abs().amax(-1)
    scales = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (blocks / scales[..., None]).clamp(-448.0, 448.0).view(n, -1)[:, :width].to(FP8)
    return q.contiguous(), scales.contiguous()


def _dequantised(q, scales):
    return q.float() * scales.repeat_interleave(128, 1)[:, :q.shape[1]]


def _quantised_weights(w):
    """e4m3 codes and FP32 scales (one per 128 x 128 block) of FP32 weights [N][K]."""
    n, k = w.shape
    p = torch.nn.functional.pad(w, (0, _blocks(k) * 128 - k, 0, _blocks(n) * 128 - n))
    p = p.view(_blocks(n), 128, _blocks(k), 128)
    scale = p.abs().amax((1, 3)).clamp_min(1e-12) / 448.0
    p = (p / scale[:, None, :, None]).clamp(-448.0, 448.0).to(FP8)
    return p.view(_blocks(n) * 128, _blocks(k) * 128)[:n, :k], scale


def _dequantised_weights(q, scales):
    s = scales.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.float() * s


def _gate_of(s):
    return 1.0 if s["gate"] is None else s["gate"].float()


def _join_forward(s):
    """The join in FP32: h, the next block's norm, and both roots."""
    y = s["y"].float()
    post = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    h = s["residual_scale"] * s["residual"].float() + _gate_of(s) * (y * post * s["post_weight"].float())
    pre = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    return h, h * pre * s["pre_weight"].float(), post[:, 0].contiguous(), pre[:, 0].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    op, rows = case["op"], case["rows"]
    if op == "few":
        topk, experts, hidden, inner = case["topk"], case["experts"], case["hidden"], case["inner"]
        everywhere = case["all_experts"]
        noise = -torch.log(-torch.log(torch.rand(rows, everywhere, generator=gen, device=dev).clamp(1e-7, 1 - 1e-6)))
        idx = (noise + 0.5 * randn(everywhere)).topk(topk, dim=1).indices.to(torch.int32)
        lost = torch.rand(rows, topk, generator=gen, device=dev) < case["dropped"]
        first = experts * ((everywhere // experts) // 2)
        idx = torch.where(lost, torch.full_like(idx, -1), idx)
        idx[0, 0] = first
        idx[0, 1:] = torch.where(idx[0, 1:] == first, torch.full_like(idx[0, 1:], -1), idx[0, 1:])
        x, x_scales = randn(rows, hidden), None
        if case["x"] == "fp8":
            x, x_scales = _quantise(x)
        else:
            x = x.to(HALF[case["x"]])
        up = torch.empty((experts, 2 * inner, hidden), dtype=FP8, device=dev)
        down = torch.empty((experts, hidden, inner), dtype=FP8, device=dev)
        up_scales = torch.empty((experts, _blocks(2 * inner), _blocks(hidden)), device=dev)
        down_scales = torch.empty((experts, _blocks(hidden), _blocks(inner)), device=dev)
        for e in range(experts):
            up[e], up_scales[e] = _quantised_weights(randn(2 * inner, hidden) * hidden ** -0.5)
            down[e], down_scales[e] = _quantised_weights(randn(hidden, inner) * inner ** -0.5)
        return {"op": op, "x": x, "x_scales": x_scales, "indices": idx.contiguous(), "first": first,
                "weights": torch.softmax(randn(rows, topk), 1).contiguous(), "up": up, "up_scales": up_scales,
                "down": down, "down_scales": down_scales, "dtype": case["dtype"]}
    t = HALF[case["dtype"]]
    if op in ("join", "join_backward"):
        hidden = case["hidden"]
        gate = {"none": lambda: None, "row": lambda: torch.sigmoid(randn(rows, 1)),
                "channel": lambda: (0.5 + 0.2 * randn(hidden)).to(t),
                "element": lambda: (1 + 0.3 * randn(rows, hidden)).to(t)}[case["gate"]]()
        s = {"op": op, "y": randn(rows, hidden).to(t), "residual": (3 * randn(rows, hidden)).to(t), "gate": gate,
             "post_weight": (1 + 0.1 * randn(hidden)).to(t), "pre_weight": (1 + 0.1 * randn(hidden)).to(t),
             "residual_scale": 0.875, "fp8": case["fp8"]}
        if op == "join_backward":
            h, _, s["post_rstd"], s["pre_rstd"] = _join_forward(s)
            s["h"] = h.to(t)
            s["dh"], s["dn"] = randn(rows, hidden).to(t), randn(rows, hidden).to(t)
        return s
    if op in ("swiglu", "swiglu_backward"):
        inner = case["inner"]
        gate_up = torch.cat([1.5 * randn(rows, inner), randn(rows, inner)], 1)
        if op == "swiglu":
            return {"op": op, "gate_up": gate_up.to(t)}
        saved, saved_scales = _quantise(gate_up)
        return {"op": op, "saved": saved, "saved_scales": saved_scales, "dz": randn(rows, inner).to(t),
                "fp8": case["fp8"]}
    inner, columns, groups = case["inner"], case["columns"], max(1, case["groups"])
    a, a_scales = _quantise(randn(rows, inner) * torch.exp(0.5 * randn(rows, 1)))
    state = {"op": op, "a": a, "a_scales": a_scales, "dy": randn(rows, columns).to(t), "offsets": None,
             "longest": rows, "dtype": case["dtype"]}
    if case["groups"]:
        group = torch.multinomial(torch.exp(0.3 * randn(groups)), rows, replacement=True, generator=gen)
        counts = (group[:, None] == torch.arange(groups, device=dev)).sum(0)
        state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        state["longest"] = int(counts.max())
    return state


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import combine_ep_dispatch_02_gb300 as ep
    op = s["op"]
    if op == "few":
        return {"out": ep.moe_few_rows(s["x"], s["x_scales"], s["indices"], s["weights"], s["up"], s["up_scales"],
                                       s["down"], s["down_scales"], first_expert=s["first"], out_dtype=s["dtype"])}
    if op == "join":
        j = ep.rms_norm_join(s["y"], s["residual"], post_weight=s["post_weight"], gate=s["gate"],
                             pre_weight=s["pre_weight"], residual_scale=s["residual_scale"], eps=EPS, fp8=s["fp8"])
        return {"h": j.h, "n": j.n, "q": j.q, "scales": j.scales, "post_rstd": j.post_rstd, "pre_rstd": j.pre_rstd}
    if op == "join_backward":
        joined = ep.Joined(h=s["h"], post_rstd=s["post_rstd"], pre_rstd=s["pre_rstd"])
        g = ep.rms_norm_join_backward(joined, s["y"], dh=s["dh"], dn=s["dn"], post_weight=s["post_weight"],
                                      gate=s["gate"], pre_weight=s["pre_weight"], residual_scale=s["residual_scale"])
        return {"dy": g.dy, "dresidual": g.dresidual, "dpost_weight": g.dpost_weight, "dgate": g.dgate,
                "dpre_weight": g.dpre_weight}
    if op == "swiglu":
        q, scales, saved, saved_scales = ep.swiglu_saved(s["gate_up"])
        return {"q": q, "scales": scales, "saved": saved, "saved_scales": saved_scales}
    if op == "swiglu_backward":
        d, q, scales = ep.swiglu_saved_backward(s["saved"], s["saved_scales"], s["dz"], fp8=s["fp8"])
        return {"d": d, "q": q, "scales": scales}
    return {"dw": ep.matmul_fp8_weight_gradient(s["dy"], s["a"], s["a_scales"], offsets=s["offsets"],
                                                out_dtype=s["dtype"])}


def _plain(s):
    return {"few": _plain_few, "join": _plain_join, "join_backward": _plain_join_backward, "swiglu": _plain_swiglu,
            "swiglu_backward": _plain_swiglu_backward, "weights": _plain_weights}[s["op"]](s)


def _plain_few(s):
    """Every local expert over every row, weighted by what the row gives it."""
    x = s["x"].float() if s["x_scales"] is None else _dequantised(s["x"], s["x_scales"])
    out = torch.zeros_like(x)
    for e in range(s["up"].shape[0]):
        w = torch.where(s["indices"] == s["first"] + e, s["weights"], torch.zeros_like(s["weights"])).sum(1)
        gate, up = (x @ _dequantised_weights(s["up"][e], s["up_scales"][e]).t()).chunk(2, dim=1)
        z = gate * torch.sigmoid(gate) * up
        out = out + w[:, None] * (z @ _dequantised_weights(s["down"][e], s["down_scales"][e]).t())
    return {"out": out.to(HALF[s["dtype"]])}


def _plain_join(s):
    h, n, post, pre = _join_forward(s)
    t = s["y"].dtype
    q, scales = _quantise(n) if s["fp8"] else (None, None)
    return {"h": h.to(t), "n": None if s["fp8"] else n.to(t), "q": q, "scales": scales, "post_rstd": post,
            "pre_rstd": pre}


def _plain_join_backward(s):
    t, gate = s["y"].dtype, _gate_of(s)
    dn, pre = s["dn"].float(), s["pre_rstd"][:, None]
    xh = s["h"].float() * pre
    g = dn * s["pre_weight"].float()
    d = s["dh"].float() + pre * (g - xh * (g * xh).mean(-1, keepdim=True))
    post = s["post_rstd"][:, None]
    yh = s["y"].float() * post
    du = d * gate
    g = du * s["post_weight"].float()
    dy = post * (g - yh * (g * yh).mean(-1, keepdim=True))
    dgate = None
    if s["gate"] is not None:
        dgate = d * (yh * s["post_weight"].float())
        if s["gate"].dim() == 1:
            dgate = dgate.sum(0)
        elif s["gate"].shape[1] == 1:
            dgate = dgate.sum(1, keepdim=True)
        else:
            dgate = dgate.to(t)
    return {"dy": dy.to(t), "dresidual": (s["residual_scale"] * d).to(t), "dpost_weight": (du * yh).sum(0),
            "dgate": dgate, "dpre_weight": (dn * xh).sum(0)}


def _plain_swiglu(s):
    x = s["gate_up"].float()
    gate, up = x.chunk(2, dim=1)
    q, scales = _quantise(gate * torch.sigmoid(gate) * up)
    saved, saved_scales = _quantise(x)
    return {"q": q, "scales": scales, "saved": saved, "saved_scales": saved_scales}


def _plain_swiglu_backward(s):
    gate, up = _dequantised(s["saved"], s["saved_scales"]).chunk(2, dim=1)
    dz, sig = s["dz"].float(), torch.sigmoid(gate)
    d = torch.cat([dz * up * sig * (1 + gate * (1 - sig)), dz * gate * sig], 1)
    q, scales = _quantise(d) if s["fp8"] else (None, None)
    return {"d": d.to(s["dz"].dtype), "q": q, "scales": scales}


def _plain_weights(s):
    """FP32 product of the dequantised rows: every group's rows padded to the longest group."""
    a, dy = _dequantised(s["a"], s["a_scales"]), s["dy"].float()
    t = HALF[s["dtype"]]
    if s["offsets"] is None:
        return {"dw": (dy.t() @ a).to(t)}
    offsets = s["offsets"].long()
    row = torch.arange(a.shape[0], device=a.device)
    group = torch.searchsorted(offsets[1:], row, right=True)
    at = row - offsets[group]
    left = dy.new_zeros(len(offsets) - 1, s["longest"], dy.shape[1])
    right = a.new_zeros(len(offsets) - 1, s["longest"], a.shape[1])
    left[group, at], right[group, at] = dy, a
    return {"dw": torch.bmm(left.transpose(1, 2), right).to(t)}


# ------------------------------------------------------------------------------------ work and 64-bit values

def work(case):
    rows, op = case["rows"], case["op"]
    if op == "few":
        hidden, inner, experts = case["hidden"], case["inner"], case["experts"]
        pairs = rows * case["topk"] * (1 - case["dropped"]) * experts / case["all_experts"]
        hit = min(pairs, experts * (1 - (1 - 1 / experts) ** pairs)) if rows > 1 else pairs
        row = hidden + 4 * _blocks(hidden) if case["x"] == "fp8" else 2 * hidden
        weights = 3 * inner * hidden + 4 * _blocks(hidden) * (_blocks(2 * inner) + _blocks(inner))
        return {"bytes": hit * weights + rows * (row + 2 * hidden + 8 * case["topk"]),
                "flops": 6 * pairs * inner * hidden}
    if op in ("join", "join_backward"):
        hidden = case["hidden"]
        n, per_row, per_channel = rows * hidden, 8, 4
        gate = {"none": (0, 0, 0), "row": (0, 4, 0), "channel": (0, 0, 2), "element": (2, 0, 0)}[case["gate"]]
        if op == "join":
            per = 4 + 2 + (1 if case["fp8"] else 2) + gate[0]
            per_row += 4 * _blocks(hidden) if case["fp8"] else 0
            return {"bytes": n * per + rows * (per_row + gate[1]) + hidden * (per_channel + gate[2]), "flops": 16 * n}
        return {"bytes": n * (8 + 4 + 2 * gate[0]) + rows * (8 + 2 * gate[1]) + hidden * (12 + 3 * gate[2]),
                "flops": 30 * n}
    if op in ("swiglu", "swiglu_backward"):
        n, inner = rows * case["inner"], case["inner"]
        if op == "swiglu":
            return {"bytes": n * 7 + 4 * rows * (_blocks(inner) + _blocks(2 * inner)), "flops": 20 * n}
        fp8 = 1 if case["fp8"] else 0
        return {"bytes": n * (8 + 2 * fp8) + 4 * rows * (1 + fp8) * _blocks(2 * inner), "flops": 20 * n}
    inner, columns, groups = case["inner"], case["columns"], max(1, case["groups"])
    return {"bytes": rows * (inner + 4 * _blocks(inner) + 2 * columns) + 2 * groups * columns * inner,
            "flops": 2 * rows * inner * columns}


def _codes64(v):
    """Values over their block's scale, and the scales."""
    q, scales = torch.empty_like(v), []
    for c in range(0, v.shape[1], 128):
        top = v[:, c:c + 128].abs().max(1).values
        top = torch.where(top == 0, torch.full_like(top, 448.0), top) / 448.0
        q[:, c:c + 128] = v[:, c:c + 128] / top[:, None]
        scales.append(top)
    return q, torch.stack(scales, 1)


def _values64(q, scales):
    v = q.double()
    for b in range(scales.shape[1]):
        v[:, 128 * b:128 * b + 128] *= scales[:, b:b + 1].double()
    return v


def _weights64(q, scales):
    v = q.double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            v[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= scales[i, j].double()
    return v


def exact(case, seed):
    """The case's outputs in 64 bits, from the definitions, element codes before their rounding."""
    s = prepare(case, seed)
    op = s["op"]
    if op == "few":
        rows, hidden = s["x"].shape
        x = s["x"].double() if s["x_scales"] is None else _values64(s["x"], s["x_scales"])
        out = torch.zeros(rows, hidden, dtype=torch.float64, device=x.device)
        inner = s["down"].shape[2]
        chosen = s["indices"].tolist()
        for e in sorted({i - s["first"] for r in chosen for i in r if 0 <= i - s["first"] < s["up"].shape[0]}):
            here = [(t, j) for t, r in enumerate(chosen) for j, i in enumerate(r) if i - s["first"] == e]
            h = _weights64(s["up"][e], s["up_scales"][e]) @ x[[t for t, _ in here]].T
            h = h[:inner] / (1 + torch.exp(-h[:inner])) * h[inner:]
            o = _weights64(s["down"][e], s["down_scales"][e]) @ h
            for c, (t, j) in enumerate(here):
                out[t] += s["weights"][t, j].double() * o[:, c]
        return {"out": out}
    if op in ("join", "join_backward"):
        width = s["y"].shape[1]
        y, wp, wq = s["y"].double(), s["post_weight"].double(), s["pre_weight"].double()
        gate = torch.ones((), dtype=torch.float64, device=y.device) if s["gate"] is None else s["gate"].double()
        if op == "join":
            post = 1 / (y.pow(2).sum(1) / width + EPS).sqrt()
            h = s["residual_scale"] * s["residual"].double() + gate * wp * y * post[:, None]
            pre = 1 / (h.pow(2).sum(1) / width + EPS).sqrt()
            n = wq * h * pre[:, None]
            q, scales = _codes64(n) if s["fp8"] else (None, None)
            return {"h": h, "n": None if s["fp8"] else n, "q": q, "scales": scales, "post_rstd": post, "pre_rstd": pre}
        dn, pre, post = s["dn"].double(), s["pre_rstd"].double()[:, None], s["post_rstd"].double()[:, None]
        h = s["h"].double()
        along = (dn * wq * h).sum(1, keepdim=True)
        d = s["dh"].double() + pre * dn * wq - pre ** 3 / width * along * h
        u = gate * d * wp
        dy = post * u - post ** 3 / width * (u * y).sum(1, keepdim=True) * y
        dgate = None
        if s["gate"] is not None:
            dgate = d * wp * y * post
            if s["gate"].dim() == 1:
                dgate = dgate.sum(0)
            elif s["gate"].shape[1] == 1:
                dgate = dgate.sum(1)[:, None]
        return {"dy": dy, "dresidual": s["residual_scale"] * d, "dpost_weight": (d * gate * y * post).sum(0),
                "dgate": dgate, "dpre_weight": (dn * h * pre).sum(0)}
    if op == "swiglu":
        x = s["gate_up"].double()
        half = x.shape[1] // 2
        q, scales = _codes64(x[:, :half] / (1 + torch.exp(-x[:, :half])) * x[:, half:])
        saved, saved_scales = _codes64(x)
        return {"q": q, "scales": scales, "saved": saved, "saved_scales": saved_scales}
    if op == "swiglu_backward":
        x, dz = _values64(s["saved"], s["saved_scales"]), s["dz"].double()
        half = x.shape[1] // 2
        gate, up = x[:, :half], x[:, half:]
        e = torch.exp(-gate)
        d = torch.cat([dz * up * (1 + e + gate * e) / (1 + e) ** 2, dz * gate / (1 + e)], 1)
        q, scales = _codes64(d) if s["fp8"] else (None, None)
        return {"d": d, "q": q, "scales": scales}
    edges = [0, case["rows"]] if s["offsets"] is None else s["offsets"].tolist()
    dw = [s["dy"][lo:hi].double().T @ _values64(s["a"][lo:hi], s["a_scales"][lo:hi])
          for lo, hi in zip(edges[:-1], edges[1:])]
    return {"dw": dw[0] if s["offsets"] is None else torch.stack(dw)}
