"""A training step of a block of experts from the framework's parts, as a user would put them together.

    python -m combine_ep_dispatch_02_gb300.expert_training [--rows 512] [--hidden 1024] [--inner 512] ...

The block is  x -> norm -> experts -> norm, gate -> joined to the residual -> norm of the next block:

    forward   rms_norm_fp8 -> sort by expert -> product -> swiglu_saved -> product -> weighted return -> rms_norm_join
    backward  the gradients in reverse: rms_norm_join_backward, return_rows_backward, products with the transposed
              weights, swiglu_saved_backward, matmul_fp8_weight_gradient, sorted_rows_backward

Between the two only 8-bit rows are kept of the experts' activations: the normed rows, SwiGLU's input and its output.
``ExpertBlock`` holds the weights and their e4m3 copies; ``forward`` returns what ``backward`` takes, and nothing waits
for the GPU.  The command compares every gradient with those of the same block in FP64, from autograd, and prints the
time of a step.
"""
from __future__ import annotations

import argparse

import torch

import combine_ep_dispatch_02_gb300 as ep
from .expert_layer import quantise_weights


def quantise_rows(x: torch.Tensor):
    """e4m3 codes and one FP32 scale per 128 elements of 16-bit rows, as rms_norm_fp8 writes them."""
    n, width = x.shape
    blocks = -(-width // 128)
    v = torch.nn.functional.pad(x.float(), (0, 128 * blocks - width)).view(n, blocks, 128)
    top = v.abs().amax(-1)
    scales = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (v / scales[..., None]).clamp(-448.0, 448.0).view(n, -1)[:, :width].to(torch.float8_e4m3fn)
    return q.contiguous(), scales


def _transposed(codes: torch.Tensor, scales: torch.Tensor):
    """The same weights with rows and columns exchanged: a 128 x 128 block keeps its scale."""
    t = codes.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
    return t, scales.transpose(1, 2).contiguous()


class ExpertBlock:
    """up [E][2*inner][hidden] (gate rows, then up rows) and down [E][hidden][inner] FP32; norm, post, gate and pre
    [hidden] FP32: the weights of the norm before the experts and after, the gate and the next block's norm."""

    def __init__(self, up, down, norm, post, gate, pre, residual_scale: float = 1.0):
        self.up, self.down = quantise_weights(up), quantise_weights(down)
        self.up_t, self.down_t = _transposed(*self.up), _transposed(*self.down)
        self.norm, self.post, self.gate, self.pre, self.residual_scale = norm, post, gate, pre, residual_scale

    def forward(self, x, indices, weights):
        """x [rows][hidden] BF16; indices and weights [rows][k].  Returns (n, kept): the next block's normed input, and
        what backward takes."""
        q, scales, _, _ = ep.rms_norm_fp8(x, self.norm)
        order = ep.sort_by_expert(indices, self.up[0].shape[0])
        rows, row_scales = ep.sorted_rows(order, q, scales)
        gate_up = ep.matmul_fp8(rows, row_scales, *self.up, offsets=order.offsets)
        z, z_scales, saved, saved_scales = ep.swiglu_saved(gate_up, offsets=order.offsets)
        out = ep.matmul_fp8(z, z_scales, *self.down, offsets=order.offsets)
        y = ep.return_rows(order, out, weights)
        joined = ep.rms_norm_join(y, x, post_weight=self.post, gate=self.gate, pre_weight=self.pre,
                                  residual_scale=self.residual_scale)
        return joined.n, (x, order, weights, rows, row_scales, z, z_scales, saved, saved_scales, out, y, joined)

    def backward(self, kept, dn):
        """Gradients from that of n, [rows][hidden] BF16: of x, the experts' weights (FP32), the routing weights, and the
        vectors along the channels.  The norm before the experts is differentiated with its own input as residual."""
        x, order, weights, rows, row_scales, z, z_scales, saved, saved_scales, out, y, joined = kept
        join = ep.rms_norm_join_backward(joined, y, dn=dn, post_weight=self.post, gate=self.gate, pre_weight=self.pre,
                                         residual_scale=self.residual_scale)
        dout, dweights = ep.return_rows_backward(order, out, weights, join.dy)
        ddown = ep.matmul_fp8_weight_gradient(dout, z, z_scales, offsets=order.offsets, out_dtype="fp32")
        dz = ep.matmul_fp8(*quantise_rows(dout), *self.down_t, offsets=order.offsets)
        d, dq, dq_scales = ep.swiglu_saved_backward(saved, saved_scales, dz, offsets=order.offsets, fp8=True)
        dup = ep.matmul_fp8_weight_gradient(d, rows, row_scales, offsets=order.offsets, out_dtype="fp32")
        dsorted = ep.matmul_fp8(dq, dq_scales, *self.up_t, offsets=order.offsets)
        dnormed = ep.sorted_rows_backward(order, dsorted)
        # the first norm is the join's second one over h = x: its gradient, with the residual's for dh
        root = torch.rsqrt(x.float().square().mean(1) + 1e-6)
        first = ep.rms_norm_join_backward(ep.Joined(h=x, pre_rstd=root), x, dh=join.dresidual, dn=dnormed, pre_weight=self.norm)
        return {"x": first.dresidual, "up": dup, "down": ddown, "weights": dweights, "norm": first.dpre_weight,
                "post": join.dpost_weight, "gate": join.dgate, "pre": join.dpre_weight}


def reference(block: ExpertBlock, x, indices, weights, dn):
    """The gradients in FP64 by autograd, from the dequantised weights, without quantising the rows between."""
    def plain(qs):
        q, s = qs
        s = s.repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :q.shape[2]]
        return q.double() * s.double()
    leaves = {"x": x.double(), "up": plain(block.up), "down": plain(block.down), "weights": weights.double(),
              **{k: getattr(block, k).double() for k in ("norm", "post", "gate", "pre")}}
    for v in leaves.values():
        v.requires_grad_()

    def norm(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w
    v = leaves["x"]
    rows = norm(v, leaves["norm"])
    y = torch.zeros_like(rows)
    for e in range(leaves["up"].shape[0]):
        t, slot = torch.nonzero(indices == e, as_tuple=True)
        gate, up = (rows[t] @ leaves["up"][e].t()).chunk(2, -1)
        o = (torch.nn.functional.silu(gate) * up) @ leaves["down"][e].t()
        y = y.index_add(0, t, leaves["weights"][t, slot][:, None] * o)
    h = block.residual_scale * v + leaves["gate"] * norm(y, leaves["post"])
    n = norm(h, leaves["pre"])
    n.backward(dn.double())
    return n.detach(), {k: v.grad for k, v in leaves.items()}


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rows", type=int, default=512)
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--topk", type=int, default=2)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--inner", type=int, default=512)
    p.add_argument("--steps", type=int, default=10)
    a = p.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)
    E, H, I = a.experts, a.hidden, a.inner
    block = ExpertBlock(randn(E, 2 * I, H) * H ** -0.5, randn(E, H, I) * I ** -0.5, *(1 + 0.1 * randn(H) for _ in range(4)), 0.75)
    x, dn = randn(a.rows, H).to(torch.bfloat16), randn(a.rows, H).to(torch.bfloat16)
    indices = torch.rand(a.rows, E, generator=gen, device=dev).topk(a.topk, 1).indices.int()
    weights = torch.softmax(randn(a.rows, a.topk), 1)
    n, kept = block.forward(x, indices, weights)
    grads = block.backward(kept, dn)
    want_n, want = reference(block, x, indices.long(), weights, dn)
    off = {"n": ((n.double() - want_n).norm() / want_n.norm()).item()}
    off.update({k: ((grads[k].double() - want[k]).norm() / want[k].norm()).item() for k in want})
    times = []
    for _ in range(a.steps):
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        block.backward(block.forward(x, indices, weights)[1], dn)
        t1.record()
        torch.cuda.synchronize()
        times.append(t0.elapsed_time(t1) * 1e3)
    assert ep.op_status() == 0
    print(f"{a.rows} rows, {E} experts, top-{a.topk}, hidden {H}, inner {I}: {sorted(times)[len(times) // 2]:.0f} us a step; off by "
          + ", ".join(f"{k} {v:.3f}" for k, v in off.items()))
    return off


if __name__ == "__main__":
    main()
