"""A mixture-of-experts layer from the framework's parts, as a user would put them together.

    python -m combine_ep_dispatch_02_gb300.expert_layer [--tokens-per-rank 256] [--hidden 7168] ...

``ExpertLayer`` holds a plan, the experts' e4m3 weights and the norm's weight; ``forward`` takes the
logical ranks' hidden rows and their routing and runs

    rms_norm_fp8 -> dispatch (FP8) -> sort by expert -> product with SwiGLU -> product
                 -> weighted return -> combine

with the residual kept beside it.  Nothing in it waits for the GPU.  The command builds one layer with
random weights, compares it with the same layer in FP32 and prints the median time of a pass.
"""
from __future__ import annotations

import argparse

import numpy as np
import torch

import combine_ep_dispatch_02_gb300 as ep


def quantise_weights(w: torch.Tensor):
    """e4m3 codes and one FP32 scale per 128 x 128 block of FP32 weights [groups][columns][inner]."""
    g, n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.nn.functional.pad(w, (0, 128 * kb - k, 0, 128 * nb - n)).view(g, nb, 128, kb, 128)
    scale = p.abs().amax((2, 4)).clamp_min(1e-12) / 448.0
    q = (p / scale[:, :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(g, 128 * nb, 128 * kb)[:, :n, :k].contiguous(), scale.contiguous()


class ExpertLayer:
    """W ranks of experts_per_rank experts each: up [W*E][2*inner][hidden] (gate rows, then up rows) and
    down [W*E][hidden][inner] as (codes, scales) pairs, norm_weight [hidden]."""

    def __init__(self, W: int, experts_per_rank: int, topk: int, hidden: int, max_tok_per_rank: int, up, down,
                 norm_weight: torch.Tensor):
        self.plan = ep.Plan(W, experts_per_rank, topk, hidden, "fp8", -(-hidden // 128), max_tok_per_rank,
                            device=norm_weight.device)
        self.up, self.down, self.norm_weight = up, down, norm_weight

    def forward(self, x: torch.Tensor, residual: torch.Tensor, route, n_tok):
        """x, residual [W][M][hidden] BF16; route(y) gives the experts [W][M][k] int32 and weights [W][M][k]
        FP32 of the normed rows y [W][M][hidden].  Returns (the experts' output [W][M][hidden], the sum
        x + residual that the next layer adds); rows at or past n_tok[rank] are padding."""
        p = self.plan
        W, M, H = p.W, p.M, p.H
        q, scales, h, y = ep.rms_norm_fp8(x.view(W * M, H), self.norm_weight, residual=residual.view(W * M, H), want_y=True)
        experts, weights = route(y.view(W, M, H))
        d = p.dispatch(q.view(W, M, H), weights, scales.view(W, M, -1), experts, n_tok)
        order = p.sort_received(d)
        rows, row_scales = ep.sorted_rows(order, d.recv_x, d.recv_scales)
        z, z_scales = ep.matmul_fp8_swiglu(rows, row_scales, *self.up, offsets=order.offsets)
        out = ep.matmul_fp8(z, z_scales, *self.down, offsets=order.offsets)
        out, _ = p.combine(ep.return_rows(order, out, d.recv_w), None, d.epoch)
        return out, h.view(W, M, H)

    def close(self):
        self.plan.close()


def reference(x, residual, experts, weights, n_tok, up, down, norm_weight):
    """The layer in FP32 from the dequantised weights, without quantising the rows between: [W][M][hidden]."""
    def plain(qs):
        q, s = qs
        s = s.repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :q.shape[2]]
        return q.float() * s
    h = x.float() + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * norm_weight.float()
    out = torch.zeros_like(y)
    for e in range(up[0].shape[0]):
        w1, w2 = plain((up[0][e:e + 1], up[1][e:e + 1]))[0], plain((down[0][e:e + 1], down[1][e:e + 1]))[0]
        rank, tok, slot = torch.nonzero(experts == e, as_tuple=True)
        gate, upper = (y[rank, tok] @ w1.t()).chunk(2, -1)
        z = (torch.nn.functional.silu(gate) * upper) @ w2.t()
        out.index_put_((rank, tok), weights[rank, tok, slot][:, None] * z, accumulate=True)
    for r, n in enumerate(n_tok):
        out[r, n:] = 0
    return out


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--ranks", type=int, default=4)
    a.add_argument("--experts-per-rank", type=int, default=8)
    a.add_argument("--topk", type=int, default=4)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--inner", type=int, default=1024)
    a.add_argument("--tokens-per-rank", type=int, default=256)
    a.add_argument("--passes", type=int, default=20)
    a = a.parse_args(argv)
    W, E, k, H, I, M = a.ranks, a.experts_per_rank, a.topk, a.hidden, a.inner, a.tokens_per_rank
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)
    up = quantise_weights(randn(W * E, 2 * I, H) * H ** -0.5)
    down = quantise_weights(randn(W * E, H, I) * I ** -0.5)
    norm_weight = (1 + 0.1 * randn(H)).to(torch.bfloat16)
    router = randn(H, W * E) * H ** -0.5
    x, residual = randn(W, M, H).to(torch.bfloat16), randn(W, M, H).to(torch.bfloat16)
    n_tok = np.array([M - (M // 3) * (r % 2) for r in range(W)], dtype=np.int32)
    chosen = {}

    def route(y):
        value, index = torch.topk(y.float() @ router, k, dim=-1)
        chosen["experts"], chosen["weights"] = index.to(torch.int32), torch.softmax(value, -1)
        return chosen["experts"], chosen["weights"]

    layer = ExpertLayer(W, E, k, H, M, up, down, norm_weight)
    out, h = layer.forward(x, residual, route, n_tok)
    want = reference(x, residual, chosen["experts"].long(), chosen["weights"], n_tok, up, down, norm_weight)
    rel = ((out.float() - want).norm() / want.norm()).item()
    times = []
    for _ in range(a.passes):
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        layer.forward(x, residual, route, n_tok)
        t1.record()
        torch.cuda.synchronize()
        times.append(t0.elapsed_time(t1) * 1e3)
    assert layer.plan.status() == 0 and ep.op_status() == 0
    layer.close()
    print(f"{int(n_tok.sum())} tokens, {W} x {E} experts, top-{k}, hidden {H}, inner {I}: "
          f"{sorted(times)[len(times) // 2]:.0f} us a pass, {rel:.3f} from the layer in FP32")
    return rel


if __name__ == "__main__":
    main()
