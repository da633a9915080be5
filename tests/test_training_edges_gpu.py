"""Calls of the training operators that the other files leave out (bounds: see test_training_gpu.py)."""
import copy
import os

import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from combine_ep_dispatch_02_gb300 import build
from test_experts_gpu import DEV, F8, HALF, _built, _gen, _no_status, _randn  # noqa: F401
from test_training_gpu import FORMS, _check_join, _inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------- join

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gate,post,pre", [f for f in FORMS if f[2]])
@pytest.mark.parametrize("rows,hidden", [(1, 16), (7, 144), (300, 272), (33, 1040), (4, 2064), (5, 528), (9, 7184), (3, 4112), (2, 8176),
                                         (2, 8208), (2, 16400), (1, 32752)])
def test_join_codes_with_a_short_last_block(rows, hidden, gate, post, pre, dtype):
    """Widths whose last 128-block has 16 to 112 columns, in a thread's first vector and in its last."""
    _check_join(_inputs(rows, hidden, HALF[dtype], gate, post, pre, rows * 1019 + hidden), 0.75, 1e-6, fp8=True)


def test_join_codes_follow_one_rule_at_every_width():
    """A row and the same row twice over have the same mean square: here exactly, because y is a small whole number of 1/8
    and widths are powers of two, so that every sum is exact.  So the codes of both are bit for bit those of the row, though
    another kernel makes them."""
    g, rows, hidden = _gen(30), 1024, 8192
    y = (torch.randint(-16, 17, (rows, hidden), generator=g, device=DEV) / 8).to(torch.bfloat16)
    w = _randn(g, hidden)
    zero = torch.zeros_like(y)
    one = ep.rms_norm_join(y, zero, pre_weight=w, fp8=True, want_n=True)
    two = ep.rms_norm_join(torch.cat([y, y], 1), torch.cat([zero, zero], 1), pre_weight=torch.cat([w, w]), fp8=True, want_n=True)
    assert torch.equal(two.pre_rstd, one.pre_rstd)
    for half in (0, 1):
        assert torch.equal(two.n[:, half * hidden:(half + 1) * hidden], one.n)
        assert torch.equal(two.scales[:, half * hidden // 128:(half + 1) * hidden // 128], one.scales)
        assert torch.equal(two.q.view(torch.uint8)[:, half * hidden:(half + 1) * hidden], one.q.view(torch.uint8))


# ------------------------------------------------------------------------------------------- weights

def test_weight_gradient_of_a_tile_that_takes_longer_than_one_wait(tmp_path, monkeypatch):
    """A tile's sums come after all of its stages.  A test build lets a wait last 4 million cycles; a million rows take some
    14 million, of which every single wait but the sums' is a few thousand: the call is right and reports nothing.  Whole
    numbers, so that the sum is exact."""
    d = str(tmp_path)
    lib = ep.load_library(build.build(force=True, defines=["EP_WAIT_CYCLES=4000000"], lib_path=os.path.join(d, "libep.so"),
                                      build_dir=d))
    rows, columns, inner = 1 << 20, 8, 16
    dy = torch.ones(rows, columns, dtype=torch.bfloat16, device=DEV)
    a = torch.full((rows, inner), 0x38, dtype=torch.uint8, device=DEV).view(F8)      # 1.0
    s = torch.full((rows, 1), 0.5, device=DEV)
    offsets = torch.tensor([0, 5, rows - 7, rows], dtype=torch.int32, device=DEV)
    with monkeypatch.context() as m:
        m.setattr(ep, "_lib", lib)
        for _ in range(3):
            whole = ep.matmul_fp8_weight_gradient(dy, a, s, out_dtype="fp32")
            parts = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets, out_dtype="fp32")
        assert ep.op_status(DEV) == 0
    assert (whole == rows / 2).all()
    assert torch.equal(parts[:, 0, 0].cpu(), torch.tensor([2.5, rows / 2 - 6, 3.5])) and (parts == parts[:, :1, :1]).all()


# ------------------------------------------------------------------------------------------- together

@pytest.mark.parametrize("rows,E,k,H,inner", [(97, 8, 2, 512, 256), (33, 5, 3, 272, 144), (200, 4, 1, 1024, 512)])
def test_a_training_step_against_the_block_and_blocks_that_differ(rows, E, k, H, inner):
    """Gradients by their norms, closely enough that a forgotten factor or term shows.  A code is off by up to 2^-4, evenly
    spread over its step of 2^-3 of the power of two below the value v: 2^-4 / sqrt(3) of that power, so, with v's place
    between two powers evenly spread over its logarithm, (3 / 8 / ln 2)^(1/2) of 2^-4 / sqrt(3) of v, 2.7 %, in the root
    mean square, which is what a norm of many values shows.  The rows pass five such roundings, forward and back, whose
    errors have nothing to do with each other: the root of 5 of them, 6 %, and twice that where SwiGLU's slope or the norms
    raise it.  16-bit roundings are 2^-8 each.  So 2^-3.

    With one expert to a row the block does not depend on the row's routing weight, but for eps: y = w * out, and the norm
    after the experts drops y's scale.  So dy is at right angles to y, and that weight's gradient, dy * out, is 0 up to eps:
    its error is held against the two vectors' norms, not against itself."""
    from combine_ep_dispatch_02_gb300.expert_training import ExpertBlock, reference
    g = _gen(rows + H)
    block = ExpertBlock(_randn(g, E, 2 * inner, H) * H ** -0.5, _randn(g, E, H, inner) * inner ** -0.5,
                        *(1 + 0.3 * _randn(g, H) for _ in range(4)), 0.75)
    x, dn = _randn(g, rows, H).to(torch.bfloat16), _randn(g, rows, H).to(torch.bfloat16)
    idx = torch.rand(rows, E, generator=g, device=DEV).topk(k, 1).indices.int()
    w = 0.25 + torch.rand(rows, k, generator=g, device=DEV)
    n, kept = block.forward(x, idx, w)
    got = {"n": n, **block.backward(kept, dn)}

    y, joined = kept[10], kept[11]
    dy = ep.rms_norm_join_backward(joined, y, dn=dn, post_weight=block.post, gate=block.gate, pre_weight=block.pre,
                                   residual_scale=0.75).dy
    sizes = {"weights": (dy.double().norm(dim=1) * y.double().norm(dim=1) / w[:, 0].double()).norm()} if k == 1 else {}

    def off(weights=w, **change):
        other = copy.copy(block)
        for name, v in change.items():
            setattr(other, name, v)
        want_n, want = reference(other, x, idx.long(), weights, dn)
        want["n"] = want_n
        return {name: ((got[name].double() - want[name]).norm() / sizes.get(name, want[name].norm())).item() for name in got}
    for name, v in off().items():
        assert v <= 2.0 ** -3, (name, v)
    # the same measure tells the block from one with another factor
    one = torch.ones_like(block.gate)
    for change in [dict(residual_scale=1.0), dict(gate=one), dict(post=one), dict(pre=one), dict(norm=one),
                   dict(up=(block.up[0], 0.75 * block.up[1])),
                   dict(down=(block.down[0].view(torch.uint8).roll(1, 0).view(F8), block.down[1].roll(1, 0)))] + \
                  [dict(weights=torch.ones_like(w))] * (k > 1):
        assert max(off(**change).values()) > 2.0 ** -3, list(change)


def test_calls_on_two_streams_at_once():
    """Products, norms and gradients of two streams share the SMs; each result is that of the call alone."""
    g, rows, H, inner = _gen(40), 777, 1040, 528
    x, r = _randn(g, rows, 2 * inner).to(torch.bfloat16), _randn(g, rows, H).to(torch.bfloat16)
    w = (1 + 0.1 * _randn(g, H)).to(torch.bfloat16)
    offsets = torch.tensor([0, 300, 300, 777], dtype=torch.int32, device=DEV)
    q, s, saved, saved_s = ep.swiglu_saved(x, offsets=offsets)
    joined = ep.rms_norm_join(r, r, post_weight=w, gate=w, pre_weight=w, fp8=True, want_n=True)

    def fields(o):
        return tuple(v for v in (getattr(o, f) for f in o.__dataclass_fields__) if v is not None)
    calls = [lambda: ep.swiglu_saved(x, offsets=offsets),
             lambda: ep.swiglu_saved_backward(saved, saved_s, q.to(torch.bfloat16), offsets=offsets, fp8=True),
             lambda: (ep.matmul_fp8_weight_gradient(r, q, s, offsets=offsets),),
             lambda: fields(ep.rms_norm_join(r, r, post_weight=w, gate=w, pre_weight=w, fp8=True, want_n=True)),
             lambda: fields(ep.rms_norm_join_backward(joined, r, dh=r, dn=r, post_weight=w, gate=w, pre_weight=w))]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(40):
        outs = []
        for k in range(len(calls)):
            for n, st in enumerate(streams):
                j = (k + i * n) % len(calls)
                with torch.cuda.stream(st):
                    outs.append((j, calls[j]()))
        torch.cuda.synchronize()
        for j, out in outs:
            for a, b in zip(out, want[j]):
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), j
        del outs
