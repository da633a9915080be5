"""The training operators of the expert layer on the GPU against their definitions in 64 bits.

Bounds are derived as in test_experts_gpu.py: u = 2^-24 per FP32 operation, n * u * sum|terms| for a sum, half a step for
each rounding to fewer bits.  Each gradient's 64-bit formula is itself compared with differences of the forward definition.
"""
import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from test_experts_gpu import (DEV, F8, HALF, U, _blocks, _built, _check_codes, _gen, _half_bound, _no_status,  # noqa: F401
                              _randn, _within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------- join

def _join64(y, r, post, gate, pre, alpha, eps):
    y, r = y.double(), r.double()
    py = 1 / (y.pow(2).mean(1, keepdim=True) + eps).sqrt()
    u = y if post is None else y * py * post.double()
    h = alpha * r + (u if gate is None else gate.double() * u)
    ph = 1 / (h.pow(2).mean(1, keepdim=True) + eps).sqrt()
    return u, h, None if pre is None else h * ph * pre.double(), py, ph


def _inputs(rows, hidden, t, gate, post, pre, seed):
    g = _gen(seed)
    made = {"y": _randn(g, rows, hidden).to(t), "residual": (2 * _randn(g, rows, hidden)).to(t),
            "gate": {"none": lambda: None, "row": lambda: torch.rand(rows, 1, generator=g, device=DEV),
                     "channel": lambda: (0.5 + 0.3 * _randn(g, hidden)).to(t), "channel32": lambda: _randn(g, hidden),
                     "element": lambda: _randn(g, rows, hidden).to(t)}[gate]()}
    for name, kind in (("post_weight", post), ("pre_weight", pre)):
        made[name] = None if kind is None else (1 + 0.2 * _randn(g, hidden)).to(t if kind == "half" else torch.float32)
    return made


SHAPES = [(1, 16), (3, 128), (1, 7168), (7, 144), (129, 256), (5, 1024), (33, 1040), (4, 2064), (257, 2048), (2, 8192)]
FORMS = [("none", None, "half"), ("row", "half", "half"), ("channel", "half", None), ("channel32", "fp32", "fp32"),
         ("element", "half", "half"), ("element", None, None), ("row", None, "fp32")]


def _check_join(m, alpha, eps, fp8):
    t, hidden = m["y"].dtype, m["y"].shape[1]
    j = ep.rms_norm_join(m["y"], m["residual"], post_weight=m["post_weight"], gate=m["gate"], pre_weight=m["pre_weight"],
                         residual_scale=alpha, eps=eps, fp8=fp8, want_n=m["pre_weight"] is not None)
    u, h, n, py, ph = _join64(m["y"], m["residual"], m["post_weight"], m["gate"], m["pre_weight"], alpha, eps)
    norm = (hidden / 2 + 8) * U                  # the squares' sum, halved by the root; root, division, products
    gu = u.abs() if m["gate"] is None else (m["gate"].double() * u).abs()
    h_err = gu * (norm + 3 * U) + 2 * U * (alpha * m["residual"].double()).abs() + U * h.abs()
    _within(j.h, h, _half_bound(t, h) + h_err, "h")
    if m["post_weight"] is not None:
        _within(j.post_rstd, py[:, 0], norm * py[:, 0], "post_rstd")
    else:
        assert j.post_rstd is None
    if m["pre_weight"] is None:
        assert j.n is None and j.q is None and j.pre_rstd is None
        return j
    shift = norm + h_err.norm(dim=1, keepdim=True) / h.norm(dim=1, keepdim=True)
    _within(j.pre_rstd, ph[:, 0], (shift * ph)[:, 0], "pre_rstd")
    n_err = n.abs() * shift + h_err * ph * m["pre_weight"].double().abs()
    _within(j.n, n, _half_bound(t, n) + n_err, "n")
    if fp8:
        _check_codes(j.q, j.scales, n, n_err)
    else:
        assert j.q is None and j.scales is None
    return j


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gate,post,pre", FORMS)
@pytest.mark.parametrize("rows,hidden", SHAPES + [(2, 16400), (1, 32768), (3000, 272), (3000, 256), (2000, 512), (999, 528)])
def test_join(rows, hidden, gate, post, pre, dtype):
    m = _inputs(rows, hidden, HALF[dtype], gate, post, pre, rows * 1009 + hidden)
    _check_join(m, 0.75, 1e-6, fp8=pre is not None and hidden % 32 == 0)


def _backward64(m, h, py, ph, dh, dn, alpha):
    """The gradients, and bounds of what FP32 leaves of each: (value, bound) by name."""
    y, hidden, rows = m["y"].double(), m["y"].shape[1], m["y"].shape[0]
    one = torch.ones((), dtype=torch.float64, device=DEV)
    gate = one if m["gate"] is None else m["gate"].double()
    wpost = one if m["post_weight"] is None else m["post_weight"].double()
    v = y if m["post_weight"] is None else y * py
    d = torch.zeros_like(y) if dh is None else dh.double()
    d_err = torch.zeros_like(y)
    out = {}
    if dn is not None:
        x, g = h.double() * ph, dn.double() * m["pre_weight"].double()
        mean = (g * x).mean(1, keepdim=True)
        mean_err = (hidden + 4) * U * (g * x).abs().mean(1, keepdim=True)
        d = d + ph * (g - x * mean)
        d_err = ph * (3 * U * g.abs() + x.abs() * (5 * U * mean.abs() + mean_err)) + 2 * U * d.abs()
        out["dpre_weight"] = ((dn.double() * x).sum(0), (rows + 4) * U * (dn.double() * x).abs().sum(0))
    out["dresidual"] = (alpha * d, abs(alpha) * (d_err + U * d.abs()))
    p = d * gate * wpost
    p_err = d_err * (gate * wpost).abs() + 4 * U * p.abs()
    u = v * wpost
    each, each_err = d * u, d_err * u.abs() + 5 * U * (d * u).abs()
    if m["gate"] is not None:
        if m["gate"].dim() == 1:
            out["dgate"] = (each.sum(0), each_err.sum(0) + rows * U * each.abs().sum(0))
        elif m["gate"].shape[1] == 1:
            out["dgate"] = (each.sum(1, keepdim=True), each_err.sum(1, keepdim=True) + hidden * U * each.abs().sum(1, keepdim=True))
        else:
            out["dgate"] = (each, each_err)
    if m["post_weight"] is not None:
        mean = (p * v).mean(1, keepdim=True)
        mean_err = (p_err * v.abs() + (hidden + 6) * U * (p * v).abs()).mean(1, keepdim=True)
        q = d * gate * v
        out["dpost_weight"] = (q.sum(0), (d_err * (gate * v).abs() + (rows + 5) * U * q.abs()).sum(0))
        dy = py * (p - v * mean)
        out["dy"] = (dy, py * (p_err + v.abs() * (mean_err + 5 * U * mean.abs())) + 2 * U * dy.abs())
    else:
        out["dy"] = (p, p_err)
    return out


def _call_backward(m, j, dh, dn, alpha):
    return ep.rms_norm_join_backward(j, m["y"], dh=dh, dn=dn, post_weight=m["post_weight"], gate=m["gate"],
                                     pre_weight=m["pre_weight"], residual_scale=alpha)


def _check_backward(m, j, dh, dn, alpha):
    got = _call_backward(m, j, dh, dn, alpha)
    py = None if j.post_rstd is None else j.post_rstd.double()[:, None]
    ph = None if j.pre_rstd is None else j.pre_rstd.double()[:, None]
    want = _backward64(m, j.h, py, ph, dh, dn, alpha)
    for name in ("dy", "dresidual", "dpost_weight", "dgate", "dpre_weight"):
        value = getattr(got, name)
        if name not in want:
            assert value is None, name
            continue
        assert value.shape == want[name][0].shape, name
        half = _half_bound(value.dtype, want[name][0]) if value.dtype != torch.float32 else 0.0
        _within(value, want[name][0], want[name][1] * 1.01 + half + 2.0 ** -140, name)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gate,post,pre", FORMS)
@pytest.mark.parametrize("rows,hidden", SHAPES + [(1500, 272), (1500, 256), (900, 512), (641, 7168)])
def test_join_backward(rows, hidden, gate, post, pre, dtype):
    t = HALF[dtype]
    m = _inputs(rows, hidden, t, gate, post, pre, rows * 1013 + hidden)
    g = _gen(rows + hidden)
    j = ep.rms_norm_join(m["y"], m["residual"], post_weight=m["post_weight"], gate=m["gate"], pre_weight=m["pre_weight"],
                         residual_scale=0.75)
    dh, dn = _randn(g, rows, hidden).to(t), _randn(g, rows, hidden).to(t) if pre else None
    _check_backward(m, j, dh, dn, 0.75)
    if pre:
        _check_backward(m, j, None, dn, 0.75)


@pytest.mark.parametrize("gate,post,pre", FORMS)
def test_join_gradient_against_differences(gate, post, pre):
    """The formula that the kernel is held to, against central differences of the definition, both in 64 bits."""
    rows, hidden, alpha, eps = 5, 48, 0.75, 1e-6
    m = {k: None if v is None else v.double() for k, v in _inputs(rows, hidden, torch.bfloat16, gate, post, pre, 3).items()}
    g = _gen(4)
    dh, dn = _randn(g, rows, hidden).double(), _randn(g, rows, hidden).double() if pre else None

    def loss(v):
        _, h, n, _, _ = _join64(v["y"], v["residual"], v["post_weight"], v["gate"], v["pre_weight"], alpha, eps)
        return (dh * h).sum() + (0 if dn is None else (dn * n).sum())
    _, h, _, py, ph = _join64(m["y"], m["residual"], m["post_weight"], m["gate"], m["pre_weight"], alpha, eps)
    formula = _backward64(m, h, py, ph, dh, dn, alpha)
    for name, grad in (("y", "dy"), ("residual", "dresidual"), ("post_weight", "dpost_weight"), ("gate", "dgate"),
                       ("pre_weight", "dpre_weight")):
        if m[name] is None:
            continue
        v = _randn(g, *m[name].shape).double()
        step = 1e-5
        ahead, back = ({**m, name: m[name] + s * step * v} for s in (1, -1))
        by = (loss(ahead) - loss(back)) / (2 * step)
        along = (formula[grad][0] * v).sum()
        # the third derivative's step^2 = 1e-10 times a factor of order hidden, and 2^-53 of the loss over the step
        assert abs(by - along) <= 1e-7 * (1 + formula[grad][0].norm() * v.norm()), name


def test_join_strides_and_streams():
    g, t = _gen(7), torch.bfloat16
    wide = _randn(g, 37, 6 * 512).to(t)
    part = [wide[:, 512 * i:512 * i + 512] for i in range(6)]
    w = (1 + 0.1 * _randn(g, 512)).to(t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kw = dict(post_weight=w, gate=part[2], pre_weight=w, fp8=True, want_n=True)
    a = ep.rms_norm_join(part[0], part[1], stream=s, **kw)
    s.synchronize()
    kw["gate"] = part[2].contiguous()
    b = ep.rms_norm_join(part[0].contiguous(), part[1].contiguous(), **kw)
    for name in ("h", "n", "scales", "post_rstd", "pre_rstd"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
    kw = dict(post_weight=w, pre_weight=w)
    torch.cuda.synchronize()
    x = ep.rms_norm_join_backward(a, part[0], dh=part[3], dn=part[4], gate=part[2], stream=s, **kw)
    s.synchronize()
    z = ep.rms_norm_join_backward(b, *(part[i].contiguous() for i in (0, 3, 4)), gate=part[2].contiguous(), **kw)
    for name in ("dy", "dresidual", "dpost_weight", "dgate", "dpre_weight"):
        assert torch.equal(getattr(x, name), getattr(z, name)), name


@pytest.mark.parametrize("over", ["y", "residual"])
@pytest.mark.parametrize("gate,post,pre", [FORMS[2], FORMS[3], FORMS[4]])
@pytest.mark.parametrize("rows,hidden", [(700, 256), (700, 512), (700, 2064), (320, 8192), (3, 16400)])
def test_join_writes_h_over_its_input(rows, hidden, gate, post, pre, over):
    lib, m = ep.load_library(), _inputs(rows, hidden, torch.bfloat16, gate, post, pre, rows + hidden)
    want = ep.rms_norm_join(**m, residual_scale=0.5)
    m = {k: v if v is None else v.clone() for k, v in m.items()}
    w, v, g = m["post_weight"], m["pre_weight"], m["gate"]
    at = [None if t is None else t.data_ptr() for t in (w, g, v)]
    j = ep.JoinArgs(m["y"].data_ptr(), hidden, at[0], at[1], hidden, at[2], rows, hidden, ep.EP_BF16,
                    int(w is not None and w.dtype == torch.float32), int(v is not None and v.dtype == torch.float32),
                    ep.GATE_KINDS[gate.rstrip("32")], int(g.dtype == torch.float32), 0.5, 1e-6)
    n, root, pre_root = torch.empty_like(want.h), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    rc = lib.ep_rms_norm_join(j, m["residual"].data_ptr(), hidden, m[over].data_ptr(), None if v is None else n.data_ptr(), None,
                              None, root.data_ptr(), pre_root.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == ep.EP_OK and torch.equal(m[over], want.h)
    assert v is None or torch.equal(n, want.n)


def test_join_of_no_rows_and_of_rows_of_zeros():
    t = torch.bfloat16
    w = torch.ones(256, dtype=t, device=DEV)
    x = torch.zeros(3, 256, dtype=t, device=DEV)
    for n in (0, 3):
        j = ep.rms_norm_join(x[:n], x[:n], post_weight=w, gate=w, pre_weight=w, fp8=True, want_n=True)
        assert j.h.shape == (n, 256) and not j.h.any() and not j.n.any() and (j.scales == 1).all()
        b = ep.rms_norm_join_backward(j, x[:n], dh=x[:n], dn=x[:n], post_weight=w, gate=w, pre_weight=w)
        assert not b.dy.any() and not b.dresidual.any()
        assert not b.dpost_weight.any() and not b.dgate.any() and not b.dpre_weight.any()


def test_join_keeps_what_is_not_a_number_in_its_row():
    t = torch.float16
    m = _inputs(4, 272, t, "row", "half", "half", 5)
    m["y"][1, 3] = float("nan")
    m["residual"][2, 100] = float("inf")
    kw = {k: m[k] for k in ("post_weight", "gate", "pre_weight")}
    j = ep.rms_norm_join(m["y"], m["residual"], **kw)
    assert torch.isnan(j.h[1]).all() and torch.isinf(j.h[2, 100]) and torch.isnan(j.n[2, 100])
    assert torch.isfinite(j.n[0]).all() and torch.isfinite(j.n[3]).all()
    b = ep.rms_norm_join_backward(j, m["y"], dn=m["residual"].clamp(-2, 2), **kw)
    assert torch.isfinite(b.dy[0]).all() and torch.isfinite(b.dy[3]).all() and torch.isnan(b.dpre_weight).any()


def test_join_gradients_are_the_same_every_time():
    m = _inputs(3001, 1040, torch.bfloat16, "channel", "half", "half", 6)
    kw = {k: m[k] for k in ("post_weight", "gate", "pre_weight")}
    j = ep.rms_norm_join(m["y"], m["residual"], **kw)
    first = _call_backward(m, j, m["residual"], m["y"], 1.0)
    for _ in range(5):
        again = _call_backward(m, j, m["residual"], m["y"], 1.0)
        for name in ("dy", "dresidual", "dpost_weight", "dgate", "dpre_weight"):
            assert torch.equal(getattr(first, name), getattr(again, name)), name


# ------------------------------------------------------------------------------------------- SwiGLU

def _values(q, scales):
    return q.double() * scales.double().repeat_interleave(128, 1)[:, :q.shape[1]]


SWIGLU_SHAPES = [(1, 16), (1, 2048), (3, 128), (7, 144), (33, 1040), (129, 256), (5, 272), (257, 1024), (1000, 80)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,inner", SWIGLU_SHAPES)
def test_swiglu_saved(rows, inner, dtype):
    g, t = _gen(rows + inner), HALF[dtype]
    x = torch.cat([3 * _randn(g, rows, inner), _randn(g, rows, inner)], 1).to(t)
    q, s, saved, saved_s = ep.swiglu_saved(x)
    gate, up = x.double().chunk(2, 1)
    z = gate * torch.sigmoid(gate) * up
    assert q.shape == z.shape and s.shape == (rows, _blocks(inner)) and saved.dtype == F8
    _check_codes(q, s, z, z.abs() * 2.0 ** -17)
    _check_codes(saved, saved_s, x.double(), torch.zeros_like(x, dtype=torch.float64))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,inner", SWIGLU_SHAPES)
def test_swiglu_saved_backward(rows, inner, dtype):
    g, t = _gen(rows + inner), HALF[dtype]
    x = torch.cat([3 * _randn(g, rows, inner), _randn(g, rows, inner)], 1).to(t)
    dz = _randn(g, rows, inner).to(t)
    _, _, saved, saved_s = ep.swiglu_saved(x)
    gate, up = _values(saved, saved_s).chunk(2, 1)
    sig, d64 = torch.sigmoid(gate), dz.double()
    want = torch.cat([d64 * up * sig * (1 + gate * (1 - sig)), d64 * gate * sig], 1)
    # a sigmoid off by 2^-17 at the most, in a sum of terms of both signs
    err = torch.cat([(d64 * up * sig).abs() * (1 + (gate * (1 - sig)).abs()), (d64 * gate * sig).abs()], 1) * 2.0 ** -16
    for fp8 in (False, True):
        d, q, s = ep.swiglu_saved_backward(saved, saved_s, dz, fp8=fp8)
        _within(d, want, _half_bound(t, want) + err, "d")
        if fp8:
            assert q.shape == want.shape and s.shape == (rows, _blocks(2 * inner))
            _check_codes(q, s, want, err)
        else:
            assert q is None and s is None
    # the formula against differences of the definition, in 64 bits
    v, step = _randn(g, rows, 2 * inner).double(), 1e-5
    vg, vu = v.chunk(2, 1)
    loss = lambda c: (d64 * (gate + c * vg) * torch.sigmoid(gate + c * vg) * (up + c * vu)).sum()  # noqa: E731
    by = (loss(step) - loss(-step)) / (2 * step)
    assert abs(by - (want * v).sum()) <= 1e-7 * (1 + want.norm() * v.norm())


def test_swiglu_rows_past_the_last_stay_as_they_were():
    rows, inner = 40, 144
    g = _gen(8)
    x, dz = _randn(g, rows, 2 * inner).half(), _randn(g, rows, inner).half()
    offsets = torch.tensor([0, 5, 5, 23], dtype=torch.int32, device=DEV)
    whole = ep.swiglu_saved(x)
    d_whole = ep.swiglu_saved_backward(whole[2], whole[3], dz, fp8=True)
    x[23:], dz[23:] = float("nan"), float("nan")
    lib, stream = ep.load_library(), torch.cuda.current_stream().cuda_stream
    end = offsets.data_ptr() + 12
    out = [torch.full_like(t.view(torch.uint8), 0x55) for t in whole]
    assert lib.ep_swiglu_saved(x.data_ptr(), 2 * inner, ep.EP_FP16, rows, inner, end, *(t.data_ptr() for t in out), stream) == 0
    d_out = [torch.full_like(t.view(torch.uint8), 0x55) for t in d_whole]
    assert lib.ep_swiglu_saved_backward(whole[2].data_ptr(), whole[3].data_ptr(), dz.data_ptr(), inner, ep.EP_FP16, rows,
                                        inner, end, *(t.data_ptr() for t in d_out), stream) == 0
    for got, want in zip(out + d_out, list(whole) + list(d_whole)):
        assert torch.equal(got[:23], want.view(torch.uint8)[:23]) and (got[23:] == 0x55).all()
    again = ep.swiglu_saved(x, offsets=offsets)
    assert torch.equal(again[0][:23].view(torch.uint8), whole[0][:23].view(torch.uint8))
    for last in (-7, 0, 99):                                # an end outside the buffer is held inside it
        ep.swiglu_saved(x, offsets=torch.tensor([last], dtype=torch.int32, device=DEV))


def test_swiglu_strides_extremes_and_no_rows():
    g = _gen(9)
    wide = _randn(g, 9, 1000).to(torch.bfloat16)
    x = wide[:, 8:8 + 512]
    for a, b in zip(ep.swiglu_saved(x), ep.swiglu_saved(x.contiguous())):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    _, _, saved, s = ep.swiglu_saved(x)
    for a, b in zip(ep.swiglu_saved_backward(saved, s, wide[:, 16:272], fp8=True),
                    ep.swiglu_saved_backward(saved, s, wide[:, 16:272].contiguous(), fp8=True)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    e = ep.swiglu_saved(x[:0])
    assert [t.shape[0] for t in e] == [0] * 4
    assert ep.swiglu_saved_backward(e[2], e[3], x[:0, :256])[0].shape == (0, 512)
    # gates at which the sigmoid is 1 or leaves FP32's normal numbers, and what is not a number stays in its block
    x = torch.ones(2, 256, dtype=torch.bfloat16, device=DEV)
    x[0, :4] = torch.tensor([300.0, -300.0, -80.0, 1e30], device=DEV)
    x[1, 5] = float("nan")
    q, s, saved, ss = ep.swiglu_saved(x)
    z = _values(q, s)
    assert z[0, 1] == 0 and abs(z[0, 3] / 1e30 - 1) < 0.01 and torch.isnan(z[1, 5]) and torch.isfinite(z[1, 6:]).all()
    d, _, _ = ep.swiglu_saved_backward(saved, ss, torch.ones(2, 128, dtype=torch.bfloat16, device=DEV))
    lost = torch.zeros(256, dtype=torch.bool, device=DEV)
    lost[5] = lost[133] = True                # both gradients at a gate that is not a number have it as a factor
    assert torch.isfinite(d[0]).all() and torch.equal(torch.isnan(d[1]), lost)


# ------------------------------------------------------------------------------------------- weights

def _gradient_inputs(g, rows, columns, inner, t):
    a, s, _, _ = ep.rms_norm_fp8(_randn(g, rows, inner).to(torch.bfloat16), 1 + 0.2 * _randn(g, inner))
    return _randn(g, rows, columns).to(t), a, s * torch.rand(s.shape, generator=g, device=DEV)


def _check_gradient(dy, a, s, offsets=None, out_dtype=None):
    t, rows = dy.dtype, dy.shape[0]
    got = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets, out_dtype=out_dtype)
    edges = [0, rows] if offsets is None else offsets.tolist()
    assert got.shape == ((len(edges) - 1,) if offsets is not None else ()) + (dy.shape[1], a.shape[1])
    for i, (lo, hi) in enumerate(zip(edges[:-1], edges[1:])):
        out = got if offsets is None else got[i]
        if hi <= lo:
            assert not out.any()
            continue
        d, v = dy[lo:hi].double(), _values(a[lo:hi], s[lo:hi])
        want = d.T @ v
        # each value's rounding to dy's type (FP16's smallest step is 2^-24), and the sum in FP32
        per = v.abs() * (2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -11) + (2.0 ** -25 if t == torch.float16 else 0.0)
        bound = d.abs().T @ (per * (1 + 2.0 ** -10) + 2 * U * (hi - lo + 8) * v.abs())
        half = _half_bound(out.dtype, want) if out.dtype != torch.float32 else U * want.abs()
        _within(out, want, half + bound * 1.01, f"group {i}")
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,columns,inner", [(64, 256, 256), (128, 128, 128), (1, 8, 16), (16, 256, 256), (63, 264, 272),
                                                (65, 8, 1040), (300, 520, 144), (1000, 1024, 512), (777, 2056, 16),
                                                (4099, 136, 2064)])
def test_weight_gradient(rows, columns, inner, dtype):
    g = _gen(rows + columns + inner)
    dy, a, s = _gradient_inputs(g, rows, columns, inner, HALF[dtype])
    _check_gradient(dy, a, s)
    _check_gradient(dy, a, s, out_dtype="fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("columns,inner,edges", [
    (264, 272, [0, 1, 1, 65, 128, 128, 400, 419]), (512, 256, [0, 0, 0, 33]), (128, 1040, [5, 64, 200, 200]),
    (1024, 2048, [0, 64, 192, 448, 449, 1000]), (8, 16, list(range(0, 260, 4)))])
def test_weight_gradient_by_group(columns, inner, edges, dtype):
    g, rows = _gen(columns + inner), edges[-1] + 7
    dy, a, s = _gradient_inputs(g, rows, columns, inner, HALF[dtype])
    # rows outside every group, and what is not a number next to a group's rows, do not enter
    dy[edges[-1]:] = float("nan")
    a.view(torch.uint8)[edges[-1]:] = 0x7F
    dy[:edges[0]] = float("inf")
    offsets = torch.tensor(edges, dtype=torch.int32, device=DEV)
    got = _check_gradient(dy, a, s, offsets)
    for _ in range(3):
        assert torch.equal(ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets), got)
    poisoned, last = dy.clone(), len(edges) - 2
    if edges[-1] > edges[-2]:
        poisoned[edges[-2]:] = float("nan")
        other = ep.matmul_fp8_weight_gradient(poisoned, a, s, offsets=offsets)
        assert torch.equal(other[:last], got[:last]) and torch.isnan(other[last]).all()


def test_weight_gradient_of_no_rows_and_of_offsets_outside_the_buffer():
    g = _gen(12)
    dy, a, s = _gradient_inputs(g, 40, 64, 128, torch.bfloat16)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert ep.matmul_fp8_weight_gradient(dy[:0], a[:0], s[:0], offsets=offsets).shape == (3, 64, 128)
    assert not ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets).any()
    assert not ep.matmul_fp8_weight_gradient(dy[:0], a[:0], s[:0]).any()
    wide = torch.tensor([-9, 20, 10, 99], dtype=torch.int32, device=DEV)     # held inside; a group that ends before it starts
    got = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=wide)
    held = torch.tensor([0, 20, 20, 40], dtype=torch.int32, device=DEV)
    want = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=held)
    assert torch.equal(got[:2], want[:2])
    assert torch.equal(got[2], ep.matmul_fp8_weight_gradient(dy[10:].contiguous(), a[10:].contiguous(), s[10:].contiguous()))


def test_weight_gradient_with_many_tiles_to_a_pair():
    """More tiles than pairs of CTAs, groups of no and of few rows among them: both accumulators are used again."""
    g = _gen(13)
    counts = torch.randint(0, 150, (64,), generator=g, device=DEV)
    counts[::7] = 0
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    dy, a, s = _gradient_inputs(g, int(offsets[-1]), 640, 528, torch.bfloat16)
    _check_gradient(dy, a, s, offsets)


@pytest.mark.parametrize("rows,columns,inner,groups", [(8192, 4096, 7168, 8), (16384, 1024, 2048, 8), (6000, 2048, 2064, 7)])
def test_weight_gradients_are_the_same_every_time(rows, columns, inner, groups):
    """Many stages one after another, random codes: one that met another stage's rows, codes or scales would differ."""
    g = _gen(rows)
    dy = _randn(g, rows, columns).to(torch.bfloat16)
    a = (100 * _randn(g, rows, inner)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.rand(rows, _blocks(inner), generator=g, device=DEV)
    offsets = torch.linspace(0, rows, groups + 1, device=DEV).int()
    want = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets)
    for _ in range(60):
        assert torch.equal(ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets), want)
    # the first and the last group against products of the values as the kernel rounds them: see test_weight_gradient
    for e in (0, groups - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        v = (a[lo:hi].float() * s[lo:hi].repeat_interleave(128, 1)[:, :inner]).to(torch.bfloat16).float()
        y = dy[lo:hi].float()
        exact = y.t().double() @ v.double()
        size = y.abs().t().double() @ v.abs().double()
        _within(want[e], exact, _half_bound(torch.bfloat16, exact) + (hi - lo) * U * size, f"group {e}")


def test_weight_gradient_on_a_stream_and_in_a_graph():
    g = _gen(14)
    dy, a, s = _gradient_inputs(g, 200, 256, 384, torch.bfloat16)
    offsets = torch.tensor([0, 77, 200], dtype=torch.int32, device=DEV)
    want = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets)
    graph.replay()
    assert torch.equal(out, want)
    dy.mul_(2)
    graph.replay()
    assert torch.equal(out, 2 * want)


# ------------------------------------------------------------------------------------------- together

@pytest.mark.parametrize("args", [["--rows", "97", "--hidden", "512", "--inner", "256", "--steps", "1"],
                                  ["--rows", "33", "--experts", "5", "--topk", "3", "--hidden", "272", "--inner", "144", "--steps", "1"]])
def test_a_training_step_has_the_gradients_of_the_block(args):
    """Against autograd in FP64, by norms.  Rows pass e4m3 (2^-4 of each element at most, so of any norm) three times on the
    way forward and twice on the way back, and a gradient is a product of one of each: five of them, with what each is
    amplified by in the next kept below 2, leave less than 5 * 2^-4 * 2."""
    from combine_ep_dispatch_02_gb300 import expert_training
    for name, off in expert_training.main(args).items():
        assert off <= 5 * 2.0 ** -3, (name, off)


def test_training_step_replays_in_a_graph_and_back_to_back():
    """Forward and backward as one graph, and as a stream of calls whose memory is reused: as calls one by one."""
    from combine_ep_dispatch_02_gb300.expert_training import ExpertBlock
    g, E, H, inner, rows = _gen(15), 6, 256, 144, 50
    block = ExpertBlock(_randn(g, E, 2 * inner, H) * H ** -0.5, _randn(g, E, H, inner) * inner ** -0.5,
                        *(1 + 0.1 * _randn(g, H) for _ in range(4)), 0.5)
    x, dn = _randn(g, rows, H).to(torch.bfloat16), _randn(g, rows, H).to(torch.bfloat16)
    idx = torch.rand(rows, E, generator=g, device=DEV).topk(2, 1).indices.int()
    w = torch.softmax(_randn(g, rows, 2), 1)

    def step():
        n, kept = block.forward(x, idx, w)
        return {"n": n, **block.backward(kept, dn)}
    first = step()
    torch.cuda.synchronize()
    for _ in range(10):
        again = step()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    for k in first:
        assert torch.equal(first[k], out[k]), k
    x.copy_(_randn(g, rows, H).to(torch.bfloat16))
    graph.replay()
    for k, v in step().items():
        assert torch.equal(v, out[k]), k
