"""What is measured of the expert-layer operators: cases, inputs, plain forms and 64-bit values.

The operators are the steps of a mixture-of-experts layer around dispatch and combine: the RMS norm
that adds the residual and writes e4m3 rows with one FP32 scale per 128 elements, the sort of rows by
expert with its weighted return and both gradients, and the block-scaled e4m3 matrix product, dense
or by expert, with a 16-bit output or with SwiGLU and an e4m3 output.

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
        # one decoded token's hidden row ahead of dispatch: latency alone
        {"name": "norm_token", "op": "norm", "rows": 1, "hidden": 7168, "dtype": "bf16", "residual": True, "y": True},
        # a ragged prompt chunk whose hidden size ends inside a scale block
        {"name": "norm_ragged", "op": "norm", "rows": 1021, "hidden": 2064, "dtype": "fp16", "residual": False,
         "y": False},
        # every token of eight ranks at 4096 tokens per rank: the prefill norm
        {"name": "norm_prefill", "op": "norm", "rows": 32768, "hidden": 7168, "dtype": "bf16", "residual": True,
         "y": True},
        # one decode step's FP8 tokens brought into expert order
        {"name": "sort_decode", "op": "sort", "rows": 64, "topk": 8, "experts": 256, "hidden": 7168, "dtype": "fp8",
         "dropped": 0.0},
        # a prefill batch in expert order (the widest rows)
        {"name": "sort_prefill", "op": "sort", "rows": 8192, "topk": 8, "experts": 256, "hidden": 7168,
         "dtype": "bf16", "dropped": 0.0},
        # back from expert order with routing weights; an eighth of the slots was dropped over capacity
        {"name": "return_ragged", "op": "return", "rows": 1531, "topk": 6, "experts": 96, "hidden": 2056,
         "dtype": "fp16", "dropped": 0.125},
        # training: gradients of the weighted return for the expert outputs and the routing weights
        {"name": "return_backward", "op": "return_backward", "rows": 4096, "topk": 8, "experts": 64, "hidden": 7168,
         "dtype": "bf16", "dropped": 0.0},
        # training: gradient of the sort, the sum of a token's expert copies
        {"name": "sort_backward", "op": "sort_backward", "rows": 2048, "topk": 8, "experts": 32, "hidden": 2048,
         "dtype": "bf16", "dropped": 0.05},
        # one token through one projection: the weights' bytes alone
        {"name": "product_token", "op": "product", "rows": 1, "inner": 7168, "columns": 2048, "groups": 0,
         "swiglu": False, "dtype": "bf16"},
        # decode: a handful of tokens per expert through the first projection of 32 experts
        {"name": "product_decode", "op": "product", "rows": 256, "inner": 7168, "columns": 4096, "groups": 32,
         "swiglu": True, "dtype": "bf16"},
        # odd sizes: ragged groups, a last scale block of 16, columns that fill no tile
        {"name": "product_ragged", "op": "product", "rows": 1777, "inner": 1040, "columns": 520, "groups": 6,
         "swiglu": False, "dtype": "fp16"},
        # prefill: the first projection of one rank's 32 experts
        {"name": "product_prefill", "op": "product", "rows": 32768, "inner": 7168, "columns": 4096, "groups": 32,
         "swiglu": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _odd(rng, lo, hi):
    """An odd whole number of lo..hi, spread over the logarithm."""
    return min(hi, int(_log(rng, lo, hi))) // 2 * 2 + 1


def _size(rng, lo, hi, step):
    """A hidden size: one of the common ones, or an odd multiple of step, spread over the logarithm."""
    if rng.random() < 0.4:
        return rng.choice([v for v in (256, 512, 1024, 2048, 4096, 7168) if lo <= v <= hi])
    return _odd(rng, max(1, lo // step), hi // step - 1) * step


def draw(rng):
    op = rng.choice(["norm", "sort", "return", "return_backward", "sort_backward", "product", "product", "product"])
    if op == "norm":
        return {"op": op, "rows": _odd(rng, 1, 32766), "hidden": _size(rng, 256, 7168, 16),
                "dtype": rng.choice(["bf16", "fp16"]), "residual": rng.random() < 0.6, "y": rng.random() < 0.5}
    if op != "product":
        dtype = rng.choice(["bf16", "fp16"] + (["fp8", "fp8"] if op == "sort" else []))
        topk, hidden = rng.choice([1, 2, 4, 6, 8]), _size(rng, 256, 7168, 16 if dtype == "fp8" else 8)
        return {"op": op, "rows": _odd(rng, 1, 8000 if op == "sort" else 4000), "topk": topk,
                "experts": max(topk, int(_log(rng, 8, 256))), "hidden": hidden, "dtype": dtype,
                "dropped": rng.choice([0.0, 0.05, 0.25])}
    groups = rng.choice([0, int(_log(rng, 2, 32)), int(_log(rng, 2, 64))])
    swiglu = rng.random() < 0.5
    return {"op": op, "rows": _odd(rng, 1, 16384), "inner": _size(rng, 256, 7168, 16),
            "columns": 2 * _size(rng, 128, 2048, 16) if swiglu else _size(rng, 136, 4096, 8), "groups": groups,
            "swiglu": swiglu, "dtype": "bf16" if swiglu else rng.choice(["bf16", "fp16"])}


# ------------------------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // 128)


def _quantised_rows(x):
    """e4m3 rows and FP32 scales (one per 128 elements of a row) of FP32 rows."""
    n, width = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(width) * 128 - width)).view(n, -1, 128)
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (x / scale[..., None]).clamp(-448.0, 448.0).view(n, -1)[:, :width]
    return q.to(FP8).contiguous(), scale.contiguous()


def _quantised_weights(w):
    """e4m3 weights and FP32 scales (one per 128 x 128 block) of FP32 weights [G][N][K]."""
    g, n, k = w.shape
    p = torch.nn.functional.pad(w, (0, _blocks(k) * 128 - k, 0, _blocks(n) * 128 - n))
    p = p.view(g, _blocks(n), 128, _blocks(k), 128)
    scale = p.abs().amax((2, 4)).clamp_min(1e-12) / 448.0
    p = (p / scale[:, :, None, :, None]).clamp(-448.0, 448.0).to(FP8)
    return p.view(g, _blocks(n) * 128, _blocks(k) * 128)[:, :n, :k].contiguous(), scale.contiguous()


def _routing(case, gen, dev):
    """Distinct experts of each token under a mildly uneven popularity, some slots dropped (-1)."""
    rows, topk, experts = case["rows"], case["topk"], case["experts"]
    noise = -torch.log(-torch.log(torch.rand(rows, experts, generator=gen, device=dev).clamp(1e-7, 1 - 1e-6)))
    popular = 0.5 * torch.randn(experts, generator=gen, device=dev)
    idx = (noise + popular).topk(topk, dim=1).indices.to(torch.int32)
    dropped = torch.rand(rows, topk, generator=gen, device=dev) < case["dropped"]
    dropped[0, 0] = False
    return torch.where(dropped, torch.full_like(idx, -1), idx).contiguous()


def _order(idx, experts, kept):
    """offsets, pos, src of the rows sorted by expert (stable): see run()."""
    flat = idx.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    sorted_key, by = torch.sort(key, stable=True)
    at = torch.empty_like(flat)
    at[by] = torch.arange(flat.numel(), dtype=torch.int32, device=idx.device)
    pos = torch.where(key < experts, at, torch.full_like(at, -1)).view(idx.shape)
    edges = torch.arange(experts + 1, dtype=torch.int32, device=idx.device)
    offsets = torch.searchsorted(sorted_key, edges).to(torch.int32)
    return offsets, pos, by[:kept].to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    op, rows = case["op"], case["rows"]
    if op == "norm":
        hidden, t = case["hidden"], HALF[case["dtype"]]
        return {"op": op, "x": randn(rows, hidden).to(t), "weight": (1 + 0.1 * randn(hidden)).to(t),
                "residual": (3 * randn(rows, hidden)).to(t) if case["residual"] else None, "y": case["y"]}
    if op == "product":
        inner, columns, groups = case["inner"], case["columns"], max(1, case["groups"])
        a, a_scales = _quantised_rows(randn(rows, inner) * torch.exp(0.5 * randn(rows, 1)))
        b = torch.empty((groups, columns, inner), dtype=FP8, device=dev)
        b_scales = torch.empty((groups, _blocks(columns), _blocks(inner)), device=dev)
        for g in range(groups):
            q, s = _quantised_weights(randn(1, columns, inner) * inner ** -0.5)
            b[g], b_scales[g] = q[0], s[0]
        state = {"op": op, "a": a, "a_scales": a_scales, "b": b, "b_scales": b_scales, "swiglu": case["swiglu"],
                 "dtype": case["dtype"], "offsets": None, "longest": rows}
        if case["groups"]:
            popular = torch.exp(0.3 * randn(groups))
            group = torch.multinomial(popular, rows, replacement=True, generator=gen)
            counts = (group[:, None] == torch.arange(groups, device=dev)).sum(0)
            state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            state["longest"] = int(counts.max())
        else:
            state["b"], state["b_scales"] = b[0], b_scales[0]
        return state
    hidden, topk, experts = case["hidden"], case["topk"], case["experts"]
    idx = _routing(case, gen, dev)
    kept = int((idx >= 0).sum())
    state = {"op": op, "indices": idx, "experts": experts, "max_rows": kept}
    if op == "sort":
        x, scales = randn(rows, hidden), None
        if case["dtype"] == "fp8":
            x, scales = _quantised_rows(x)
        else:
            x = x.to(HALF[case["dtype"]])
        return {**state, "x": x, "scales": scales}
    t = HALF[case["dtype"]]
    state["order"] = _order(idx, experts, kept)
    state["y"] = randn(kept, hidden).to(t)
    state["weights"] = torch.softmax(randn(rows, topk), 1).contiguous()
    if op == "return_backward":
        state["dout"] = randn(rows, hidden).to(t)
    return state


# ------------------------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import combine_ep_dispatch_02_gb300 as ep
    op = s["op"]
    if op == "norm":
        q, scales, h, y = ep.rms_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=EPS, want_y=s["y"])
        return {"q": q, "scales": scales, "h": h, "y": y}
    if op == "product":
        if s["swiglu"]:
            q, scales = ep.matmul_fp8_swiglu(s["a"], s["a_scales"], s["b"], s["b_scales"], offsets=s["offsets"])
            return {"q": q, "scales": scales}
        return {"out": ep.matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], offsets=s["offsets"],
                                     out_dtype=s["dtype"])}
    if op == "sort":
        order = ep.sort_by_expert(s["indices"], s["experts"], max_rows=s["max_rows"])
        x, scales = ep.sorted_rows(order, s["x"], s["scales"])
        return {"offsets": order.offsets, "pos": order.pos, "src": order.src, "x": x, "scales": scales}
    order = ep.ExpertOrder(*s["order"])
    if op == "return":
        return {"out": ep.return_rows(order, s["y"], s["weights"])}
    if op == "sort_backward":
        return {"dx": ep.sorted_rows_backward(order, s["y"])}
    dy, dweights = ep.return_rows_backward(order, s["y"], s["weights"], s["dout"])
    return {"dy": dy, "dweights": dweights}


def _quantise(y):
    n, width = y.shape
    blocks = torch.nn.functional.pad(y, (0, _blocks(width) * 128 - width)).view(n, -1, 128)
    top = blocks.abs().amax(-1)
    scales = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (blocks / scales[..., None]).clamp(-448.0, 448.0).view(n, -1)[:, :width].to(FP8)
    return q.contiguous(), scales


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scales = _quantise(y)
        t = s["x"].dtype
        return {"q": q, "scales": scales, "h": None if s["residual"] is None else h.to(t),
                "y": y.to(t) if s["y"] else None}
    if op == "product":
        z = _plain_product(s)
        if not s["swiglu"]:
            return {"out": z.to(HALF[s["dtype"]])}
        gate, up = z.chunk(2, dim=1)
        q, scales = _quantise(gate * torch.sigmoid(gate) * up)
        return {"q": q, "scales": scales}
    if op == "sort":
        offsets, pos, src = _order(s["indices"], s["experts"], s["max_rows"])
        rows = src.long() // s["indices"].shape[1]
        x = s["x"].view(torch.uint8)[rows].view(s["x"].dtype)
        return {"offsets": offsets, "pos": pos, "src": src, "x": x,
                "scales": None if s["scales"] is None else s["scales"][rows]}
    offsets, pos, src = s["order"]
    here = pos >= 0
    at, t = pos.clamp_min(0).long(), s["y"].dtype
    if op == "return_backward":
        rows, w, dout = src.long() // pos.shape[1], s["weights"], s["dout"].float()
        dy = (w.reshape(-1)[src.long()][:, None] * dout[rows]).to(t)
        dots = (s["y"].float()[at] * dout[:, None]).sum(-1)
        return {"dy": dy, "dweights": torch.where(here, dots, torch.zeros_like(dots))}
    w = s["weights"] if op == "return" else torch.ones_like(s["weights"])
    w = torch.where(here, w, torch.zeros_like(w))
    out = (s["y"][at].float() * w[..., None]).sum(1).to(t)
    return {"out": out} if op == "return" else {"dx": out}


def _plain_product(s):
    """FP32 product of the dequantised values: every group's rows padded to the longest group."""
    a, b = s["a"].float(), s["b"].float()
    a = a * s["a_scales"].repeat_interleave(128, 1)[:, :a.shape[1]]
    bs = s["b_scales"].repeat_interleave(128, -1)[..., :b.shape[-1]]
    b = b * bs.repeat_interleave(128, -2)[..., :b.shape[-2], :]
    if s["offsets"] is None:
        return a @ b.t()
    offsets = s["offsets"].long()
    row = torch.arange(a.shape[0], device=a.device)
    group = torch.searchsorted(offsets[1:], row, right=True)
    at = row - offsets[group]
    padded = a.new_zeros(b.shape[0], s["longest"], a.shape[1])
    padded[group, at] = a
    return torch.bmm(padded, b.transpose(1, 2))[group, at]


# ------------------------------------------------------------------------------------ work and 64-bit values

def work(case):
    rows, op = case["rows"], case["op"]
    if op == "norm":
        n = rows * case["hidden"]
        per = 2 + 1 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
        return {"bytes": n * per + 4 * rows * _blocks(case["hidden"]) + 2 * case["hidden"], "flops": 8 * n}
    if op == "product":
        inner, columns, groups = case["inner"], case["columns"], max(1, case["groups"])
        hit = groups * (1 - (1 - 1 / groups) ** rows) if groups > 1 else 1
        b = hit * (columns * inner + 4 * _blocks(columns) * _blocks(inner))
        a = rows * (inner + 4 * _blocks(inner))
        half = columns // 2
        out = rows * (half + 4 * _blocks(half)) if case["swiglu"] else 2 * rows * columns
        return {"bytes": a + b + out, "flops": 2 * rows * inner * columns}
    hidden, pairs = case["hidden"], rows * case["topk"]
    kept = pairs * (1 - case["dropped"])
    row = hidden + 4 * _blocks(hidden) if case["dtype"] == "fp8" else 2 * hidden
    if op == "sort":
        return {"bytes": 8 * pairs + 4 * kept + 4 * case["experts"] + (rows + kept) * row, "flops": 0}
    if op == "return":
        return {"bytes": 8 * pairs + (rows + kept) * row, "flops": 2 * kept * hidden}
    if op == "sort_backward":
        return {"bytes": 4 * pairs + (rows + kept) * row, "flops": kept * hidden}
    return {"bytes": 12 * pairs + (rows + 2 * kept) * row, "flops": 3 * kept * hidden}


def exact(case, seed):
    """The case's outputs in 64 bits, from the definitions, element codes before their rounding."""
    s = prepare(case, seed)
    op = s["op"]

    def codes(v):
        """Values over their block's scale, and the scales."""
        scales = []
        q = torch.empty_like(v)
        for c in range(0, v.shape[1], 128):
            top = v[:, c:c + 128].abs().max(1).values
            top = torch.where(top == 0, torch.full_like(top, 448.0), top) / 448.0
            q[:, c:c + 128] = v[:, c:c + 128] / top[:, None]
            scales.append(top)
        return q, torch.stack(scales, 1)

    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        y = h / (h.pow(2).sum(1, keepdim=True) / h.shape[1] + EPS).sqrt() * s["weight"].double()
        q, scales = codes(y)
        return {"q": q, "scales": scales, "h": None if s["residual"] is None else h, "y": y if s["y"] else None}
    if op == "product":
        b, b_scales = s["b"], s["b_scales"]
        edges = [0, case["rows"]] if s["offsets"] is None else s["offsets"].tolist()
        if s["offsets"] is None:
            b, b_scales = b[None], b_scales[None]
        outs = []
        for g in range(len(edges) - 1):
            a = s["a"][edges[g]:edges[g + 1]].double()
            scale = s["a_scales"][edges[g]:edges[g + 1]].double()
            z = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device=a.device)
            for n in range(0, b.shape[1], 128):
                w = b[g, n:n + 128].double()
                left, right = torch.empty_like(a), torch.empty_like(w)
                for kb in range(b_scales.shape[2]):
                    cut = slice(128 * kb, 128 * kb + 128)
                    left[:, cut] = a[:, cut] * scale[:, kb:kb + 1]
                    right[:, cut] = w[:, cut] * b_scales[g, n // 128, kb].double()
                z[:, n:n + 128] = left @ right.T
            outs.append(z)
        z = torch.cat(outs)
        if not s["swiglu"]:
            return {"out": z}
        half = z.shape[1] // 2
        z = z[:, :half] / (1 + (-z[:, :half]).exp()) * z[:, half:]
        q, scales = codes(z)
        return {"q": q, "scales": scales}
    topk, n = case["topk"], case["rows"]
    token = torch.div(torch.nonzero(s["indices"].reshape(-1) >= 0)[:, 0], topk, rounding_mode="floor")
    expert = s["indices"].reshape(-1)[s["indices"].reshape(-1) >= 0].long()
    rank = torch.argsort(expert * (n * topk) + torch.arange(len(expert), device=expert.device))
    if op == "sort":
        x = s["x"].double()[token[rank]]
        return {"offsets": None, "pos": None, "src": None, "x": x,
                "scales": None if s["scales"] is None else s["scales"].double()[token[rank]]}
    y = s["y"].double()
    w = s["weights"].double().reshape(-1)[s["indices"].reshape(-1) >= 0][rank]
    if op == "return_backward":
        dout = s["dout"].double()[token[rank]]
        dots = torch.zeros(n * topk, dtype=torch.float64, device=y.device)
        place = torch.nonzero(s["indices"].reshape(-1) >= 0)[:, 0][rank]
        dots[place] = (y * dout).sum(1)
        return {"dy": w[:, None] * dout, "dweights": dots.view(n, topk)}
    total = torch.zeros(n, y.shape[1], dtype=torch.float64, device=y.device)
    total.index_add_(0, token[rank], y * w[:, None] if op == "return" else y)
    return {"out": total} if op == "return" else {"dx": total}
