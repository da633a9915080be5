"""Calls of the expert layer for a few rows at the edges of what it takes (bounds: see test_experts_gpu.py)."""
import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from test_experts_gpu import DEV, F8, HALF, U, _built, _gen, _half_bound, _no_status, _randn, _within  # noqa: F401
from test_few_rows_gpu import _layer, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 9, 33])
@pytest.mark.parametrize("kind", ["fp8", "fp16", "bf16"])
def test_columns_far_below_their_block_keep_their_values(rows, kind):
    """One 128-block of z holds groups of 8 columns from 2^16 down to 2^-22 (negative gates), and each output takes one of the
    small groups alone: the large group's down codes are 0.  The products with up are exact: x is 1/128 everywhere and a
    weight row one value, so all partial sums are whole multiples of a step of few bits.  z is then off by the sigmoid's 2^-16
    and FP16's half step 2^-11, below FP16's normal numbers by half its smallest step, 2^-25, where the block's largest is 2^14
    or more; that may happen twice, the second time to what the first left halved at least: 1.5 * 2^-39 of the largest."""
    g, hidden, inner = _gen(rows), 128, 256
    gates = torch.tensor([256.0, 0.5, -1, -4, -6, -8, -9, -10, -11, -12, -13, -14, -15, -16, -18, -20], device=DEV)
    group = torch.arange(inner, device=DEV) % 128 // 8
    gate = gates[group]
    up = 1 + torch.randint(0, 8, (inner,), generator=g, device=DEV) / 8
    up[group == 0] = 256.0
    own = group[None] == 1 + torch.arange(hidden, device=DEV)[:, None] % 15
    down = torch.where(own, _randn(g, hidden, inner), 0.0).to(F8)
    layer = (torch.cat([gate, up])[:, None].expand(-1, hidden).to(F8).contiguous()[None], torch.ones(1, 4, 1, device=DEV),
             down[None], torch.full((1, 1, 2), 1024.0, device=DEV))
    x = torch.full((rows, hidden), 1.0 if kind == "fp8" else 2.0 ** -7, device=DEV).to(F8 if kind == "fp8" else HALF[kind])
    xs = torch.full((rows, 1), 2.0 ** -7, device=DEV) if kind == "fp8" else None
    out = ep.moe_few_rows(x, xs, torch.zeros(rows, 1, dtype=torch.int32, device=DEV), torch.ones(rows, 1, device=DEV), *layer,
                          out_dtype="fp16" if kind == "fp16" else "bf16")
    z = gate.double() * torch.sigmoid(gate.double()) * up.double()
    err = z.abs() * (2.0 ** -16 + 2.0 ** -11) * (1 + 2.0 ** -10) + 1.5 * 2.0 ** -39 * z.abs().max()
    d = down.double() * 1024
    want, bound = d @ z, d.abs() @ (err + (inner + 8) * 2 * U * z.abs())
    # half of either output type's smallest step near 0 is within _half_bound's 2^-25 (FP16) and far below these values (BF16)
    _within(out, want.expand(rows, -1), (_half_bound(out.dtype, want) + bound * 1.01).expand(rows, -1), "out")


@pytest.mark.parametrize("first", [-1, -3, -4, -7, -(2 ** 31)])
def test_negative_ids_are_left_out_whatever_the_first_expert(first):
    """-1 marks a dropped slot also where first_expert is negative, as on a rank whose range starts before the experts do."""
    g = _gen(20)
    layer = _layer(g, 4, 256, 128)
    x, xs = _rows(g, 20, 256, "fp8")
    idx = torch.randint(-5, 6, (20, 6), generator=g, device=DEV, dtype=torch.int32)
    idx[0] = -1
    idx[1, :] = torch.tensor([-1, 0, -2, -(2 ** 31), 1, -1], device=DEV)
    w = torch.softmax(_randn(g, 20, 6), 1)
    out = ep.moe_few_rows(x, xs, idx, w, *layer, first_expert=first)
    assert torch.equal(out, ep.moe_few_rows(x, xs, torch.where(idx < 0, 1000, idx), w, *layer, first_expert=first))
    assert not out[0].any()


def test_example_layer_decodes_with_more_experts_than_the_one_call_takes():
    """1040 experts: within what the sorted calls take, above moe_few_rows's 1024.  The bound is that of the example layer's
    other tests."""
    from combine_ep_dispatch_02_gb300 import expert_layer
    assert expert_layer.main(["--ranks", "4", "--experts-per-rank", "260", "--topk", "4", "--tokens-per-rank", "8", "--hidden", "128",
                              "--inner", "32", "--passes", "1", "--decode-rows", "5"]) <= 2.0 ** -3
