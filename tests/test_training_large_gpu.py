"""The training operators and the layer for a few rows where an array passes 2^32 bytes: the last rows, or the last experts,
are bit for bit those of a call on them alone."""
import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from test_experts_gpu import DEV, F8, _blocks, _built, _gen, _no_status, _randn  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS, HIDDEN = 300000, 7200      # 4.3 GB of 16 bits, the last block of scales short
LAST = slice(ROWS - 5, ROWS)


def _equal(a, b):
    return torch.equal(a.view(torch.uint8) if a.dtype == F8 else a, b.view(torch.uint8) if b.dtype == F8 else b)


def _rows(seed):
    return torch.randn(ROWS, HIDDEN, dtype=torch.bfloat16, device=DEV, generator=_gen(seed))


@pytest.fixture(autouse=True)
def _memory_back():
    yield
    torch.cuda.empty_cache()


def test_join_past_32_bits():
    y, r, w = _rows(1), _rows(2), 1 + 0.2 * _randn(_gen(3), HIDDEN)
    kw = dict(post_weight=w, pre_weight=w)
    j = ep.rms_norm_join(y, r, gate=r, fp8=True, want_n=True, **kw)
    k = ep.rms_norm_join(y[LAST], r[LAST], gate=r[LAST], fp8=True, want_n=True, **kw)
    for name in ("h", "n", "q", "scales", "post_rstd", "pre_rstd"):
        assert _equal(getattr(j, name)[LAST], getattr(k, name)), name
    a = ep.rms_norm_join_backward(j, y, dh=r, dn=y, gate=r, **kw)
    b = ep.rms_norm_join_backward(k, y[LAST], dh=r[LAST], dn=y[LAST], gate=r[LAST], **kw)
    for name in ("dy", "dresidual", "dgate"):
        assert _equal(getattr(a, name)[LAST], getattr(b, name)), name


def test_swiglu_past_32_bits():
    x, inner = _rows(4), HIDDEN // 2
    got, want = ep.swiglu_saved(x), ep.swiglu_saved(x[LAST])
    for a, b in zip(got, want):
        assert _equal(a[LAST], b)
    dz = x[:, inner:]
    back, last = ep.swiglu_saved_backward(got[2], got[3], dz, fp8=True), ep.swiglu_saved_backward(want[2], want[3], dz[LAST], fp8=True)
    for a, b in zip(back, last):
        assert _equal(a[LAST], b)


def test_weight_gradient_past_32_bits():
    """A gradient of 8 GB, groups of up to 90 rows and of none; and rows of 4.3 GB in one group, of which only the last 9 are
    not zero."""
    g, groups, columns, inner = _gen(5), 72, 4096, 7168
    counts = torch.randint(0, 90, (groups,), generator=g, device=DEV)
    counts[5], counts[groups - 1] = 0, 77
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    rows = int(offsets[-1])
    dy = _randn(g, rows, columns).to(torch.bfloat16)
    a = (100 * _randn(g, rows, inner)).clamp(-448, 448).to(F8)
    s = torch.rand(rows, _blocks(inner), generator=g, device=DEV)
    dw = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets, out_dtype="fp32")
    assert dw.numel() * 4 > 2 ** 32 and not dw[5].any()
    last = slice(rows - 77, rows)
    assert torch.equal(dw[groups - 1], ep.matmul_fp8_weight_gradient(dy[last], a[last], s[last], out_dtype="fp32"))
    del dw
    columns, inner, last = 64, 7168, slice(ROWS * 2 - 9, ROWS * 2)
    dy = torch.zeros(ROWS * 2, columns, dtype=torch.bfloat16, device=DEV)
    dy[last] = _randn(g, 9, columns).to(torch.bfloat16)
    a = torch.randint(0, 127, (ROWS * 2, inner), dtype=torch.uint8, device=DEV, generator=g).view(F8)
    s = torch.rand(ROWS * 2, _blocks(inner), generator=g, device=DEV)
    got = ep.matmul_fp8_weight_gradient(dy, a, s, out_dtype="fp32")
    v = (a[last].float() * s[last].repeat_interleave(128, 1)).to(torch.bfloat16).double()
    want = dy[last].double().T @ v
    assert (got.double() - want).abs().max() <= 2.0 ** -20 * (dy[last].double().abs().T @ v.abs()).max()


def test_few_rows_past_32_bits():
    """Weights of 6 GB and 3 GB: the last experts' part of a layer is that of a layer of theirs alone."""
    g, experts, hidden, inner, rows = _gen(6), 210, 7168, 2048, 3
    up = torch.randint(0, 127, (experts, 2 * inner, hidden), dtype=torch.uint8, device=DEV, generator=g).view(F8)
    down = torch.randint(0, 127, (experts, hidden, inner), dtype=torch.uint8, device=DEV, generator=g).view(F8)
    scales = [1e-4 * torch.rand(experts, n, k, generator=g, device=DEV) for n, k in ((2 * inner // 128, hidden // 128),
                                                                                    (hidden // 128, inner // 128))]
    assert up.numel() > 2 ** 32 - 1
    x = _randn(g, rows, hidden).to(torch.bfloat16)
    idx = torch.tensor([[209, 0], [208, 207], [206, 209]], dtype=torch.int32, device=DEV)
    w = torch.rand(rows, 2, generator=g, device=DEV)
    last = slice(204, 210)      # as many experts as pairs: the order of sums goes by the fewer of the two
    got = ep.moe_few_rows(x, None, torch.where(idx < 204, -1, idx), w, up, scales[0], down, scales[1])
    want = ep.moe_few_rows(x, None, idx - 204, w, up[last], scales[0][last], down[last], scales[1][last])
    assert torch.equal(got, want) and torch.isfinite(got).all() and (got != 0).any(1).all()
