"""The expert-layer operators on the GPU against their definitions in 64 bits.

Error bounds are derived, not fitted.  u = 2^-24 is FP32's unit roundoff; a sum of n terms in any
order is off by at most n * u * sum|terms| (taken twice as large, 2 u, where a matrix unit may
truncate instead of round); a 16-bit output adds half a unit in its last place (2^-8 relative for
BF16, 2^-11 for FP16, or half the smallest subnormal, 2^-25, for FP16); an e4m3 code is within 2^-4
relative or 2^-10 absolute of the value it rounds.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from combine_ep_dispatch_02_gb300 import workloads as wlmod

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
U = 2.0 ** -24
HALF = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    from combine_ep_dispatch_02_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _no_status():
    assert ep.op_status(DEV) == 0
    yield
    assert ep.op_status(DEV) == 0


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _blocks(n):
    return -(-n // 128)


def _within(got, want, bound, what):
    got, want = got.double(), want.double()
    off = (got - want).abs() - bound
    assert not torch.isnan(off).any(), what
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:g} past its bound"


def _half_bound(t, want):
    return HALF_ULP[t] * want.abs() * (1 + 2.0 ** -8) + (2.0 ** -25 if t == torch.float16 else 0.0)


def _check_codes(q, scales, z, z_err):
    """q and scales hold z [rows][n] to e4m3's half step, given |z| off by at most z_err before it."""
    n = z.shape[1]
    pad = _blocks(n) * 128 - n
    zb = torch.nn.functional.pad(z, (0, pad)).view(z.shape[0], -1, 128)
    eb = torch.nn.functional.pad(z_err.expand_as(z), (0, pad)).view(z.shape[0], -1, 128)
    top = zb.abs().amax(-1)
    want = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    _within(scales, want, torch.where(top > 0, eb.amax(-1) / 448.0 + 2 * U * want, torch.zeros_like(want)), "scales")
    s = scales.double().repeat_interleave(128, 1)[:, :n]
    v = z / s
    bound = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) * (1 + 2.0 ** -20) + 1.07 * z_err / s
    # a value just past 448 (its scale was rounded down) saturates
    _within(q.double(), v, bound + (v.abs() - 448).clamp_min(0), "codes")


# ------------------------------------------------------------------------------------------- norm

def _norm64(x, w, r, eps):
    h = x.double() + (r.double() if r is not None else 0)
    return h, h / (h.pow(2).mean(1, keepdim=True) + eps).sqrt() * w.double()


def _check_norm(x, w, r, eps=1e-6, **kw):
    q, s, h, y = ep.rms_norm_fp8(x, w, residual=r, eps=eps, want_y=True, **kw)
    h64, y64 = _norm64(x, w, r, eps)
    if r is None:
        assert h is None
    else:
        assert torch.equal(h, (x.float() + r.float()).to(x.dtype))      # one FP32 add, one rounding
    # the squares' sum: at most hidden terms (halved by the root); h, root, division, two products
    err = y64.abs() * (x.shape[1] / 2 + 6) * U
    _within(y, y64, _half_bound(x.dtype, y64) + 2 * err, "y")
    _check_codes(q, s, y64, err)
    assert s.shape == (x.shape[0], _blocks(x.shape[1])) and q.dtype == F8


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,hidden", [(1, 16), (3, 128), (1, 7168), (7, 144), (129, 256), (5, 1024), (33, 1040),
                                         (4, 2064), (257, 2048), (2, 16384), (2, 16400), (1, 32768)])
def test_norm(rows, hidden, dtype):
    g, t = _gen(rows * 100003 + hidden), HALF[dtype]
    x, r = _randn(g, rows, hidden).to(t), (4 * _randn(g, rows, hidden)).to(t)
    w = 1 + 0.2 * _randn(g, hidden)
    _check_norm(x, w.to(t), r)
    _check_norm(x, w, None)


def test_norm_strides_streams_and_no_optional_outputs():
    g = _gen(5)
    wide = _randn(g, 37, 3 * 512).to(torch.bfloat16)
    x, r = wide[:, 512:1024], wide[:, 1024:]
    w = (1 + 0.2 * _randn(g, 512)).to(torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, sc, h, y = ep.rms_norm_fp8(x, w, residual=r, stream=s)
    s.synchronize()
    q2, sc2, h2, y2 = ep.rms_norm_fp8(x.contiguous(), w, residual=r.contiguous())
    assert y is None and y2 is None
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2) and torch.equal(h, h2)


def test_norm_zeros_tiny_and_non_finite_rows():
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(5, 256, dtype=torch.bfloat16, device=DEV)
    x[1] = 1e-30
    x[2, 7] = float("nan")
    x[3, 200] = float("inf")
    x[4, :128] = 3.0                                           # the second block stays zero
    q, s, h, y = ep.rms_norm_fp8(x, w, want_y=True)
    q = q.float()
    assert not q[0].any() and torch.equal(s[0], torch.ones(2, device=DEV))
    assert torch.isfinite(q[1]).all() and (s[1] > 0).all()
    assert torch.isnan(q[2]).all() and torch.isnan(y[2]).all() and torch.equal(s[2], torch.ones(2, device=DEV))
    assert torch.isnan(q[3, 200]) and not q[3, :200].any()     # inf * 0, and 0 elsewhere
    assert (q[4, :128] == 448).all() and not q[4, 128:].any() and s[4, 1] == 1
    empty = ep.rms_norm_fp8(x[:0], w)
    assert empty[0].shape == (0, 256) and empty[1].shape == (0, 2)


# ------------------------------------------------------------------------------- sort by expert and back

def _sort_np(idx, E, counts, max_rows):
    idx = idx.cpu().numpy()
    W, R, k = idx.shape
    flat = idx.reshape(-1)
    pair = np.arange(flat.size)
    rank, row = pair // (R * k), pair // k % R
    held = np.full(W, R) if counts is None else np.asarray(counts)
    ok = (flat >= rank * E) & (flat < (rank + 1) * E) & (row < held[rank])
    order = pair[ok][np.argsort(flat[ok], kind="stable")]
    offsets = np.searchsorted(flat[order], np.arange(W * E + 1))
    pos = np.full(flat.size, -1)
    order = order[:max_rows]
    pos[order] = np.arange(order.size)
    src = np.full(max_rows, -1)
    src[:order.size] = order
    return np.minimum(offsets, max_rows), pos.reshape(idx.shape), src


def _check_sort(idx, E, counts=None, max_rows=None):
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
    order = ep.sort_by_expert(idx if idx.shape[0] > 1 else idx[0], E, max_rows=max_rows, counts=c)
    want = _sort_np(idx, E, counts, idx.numel() if max_rows is None else max_rows)
    for name, w in zip(("offsets", "pos", "src"), want):
        assert np.array_equal(getattr(order, name).cpu().numpy().reshape(w.shape), w), name
    return order


def _indices(g, W, R, k, E, bad=0.1):
    idx = torch.randint(0, W * E, (W, R, k), generator=g, device=DEV, dtype=torch.int32)
    odd = torch.randint(-3, W * E + 9, (W, R, k), generator=g, device=DEV, dtype=torch.int32)
    return torch.where(torch.rand(W, R, k, generator=g, device=DEV) < bad, odd, idx)


@pytest.mark.parametrize("W,R,k,E", [(1, 1, 1, 1), (1, 3, 8, 256), (1, 1000, 8, 32), (1, 1024, 8, 7), (1, 1025, 8, 7),
                                     (1, 256, 8, 7), (1, 257, 8, 7), (1, 2047, 1, 40),
                                     (1, 1537, 6, 96), (1, 9000, 8, 256), (1, 700, 64, 4096), (1, 64, 2, 4096),
                                     (1, 20000, 1, 1), (2, 64, 2, 4), (4, 999, 9, 64), (8, 2048, 8, 32), (32, 5, 3, 2),
                                     (1, 500, 4, 2048), (1, 500, 4, 2049), (1, 40000, 8, 129), (1, 16384, 8, 300),
                                     (1, 16385, 8, 300), (2, 20001, 4, 700)])
def test_sort_by_expert(W, R, k, E):
    g = _gen(W + 10 * R + k + E)
    idx = _indices(g, W, R, k, E)
    _check_sort(idx, E)
    _check_sort(idx, E, counts=np.random.default_rng(R).integers(0, R + 1, W))


def test_sort_nothing_and_one_expert_for_all():
    _check_sort(torch.full((1, 777, 4), -1, dtype=torch.int32, device=DEV), 16)
    _check_sort(torch.full((1, 5000, 8), 3, dtype=torch.int32, device=DEV), 16)   # every slot names expert 3
    _check_sort(torch.zeros((1, 0, 4), dtype=torch.int32, device=DEV), 16)
    _check_sort(torch.zeros((2, 50, 4), dtype=torch.int32, device=DEV), 16, counts=[0, 0])


@pytest.mark.parametrize("W,E", [(1, 2049), (1, 4096), (2, 1500)])
def test_sort_of_no_rows_with_many_groups(W, E):
    shape = (W, 0, 4) if W > 1 else (0, 4)
    order = ep.sort_by_expert(torch.zeros(shape, dtype=torch.int32, device=DEV), E, max_rows=37)
    assert order.offsets.shape == (W * E + 1,) and not order.offsets.any()
    assert order.pos.shape == shape and (order.src == -1).all()


@pytest.mark.parametrize("R", [100, 4000])
def test_sort_past_capacity_is_recorded_and_left_out(R):
    idx = _indices(_gen(R), 1, R, 8, 16, bad=0)
    order = _check_sort(idx, 16, max_rows=R * 3)
    assert ep.op_status(DEV) == ep.EP_ERR_CAPACITY
    x = _randn(_gen(1), R, 64).to(torch.bfloat16)
    xs, _ = ep.sorted_rows(order, x)
    assert torch.equal(xs, x[(order.src // 8).long()])
    _check_sort(idx, 16, max_rows=0)
    assert ep.op_status(DEV) == ep.EP_ERR_CAPACITY


@pytest.mark.parametrize("dtype,hidden,sd", [("bf16", 8, 0), ("fp16", 2056, 0), ("fp8", 7168, 56), ("fp8", 16, 1),
                                             ("f32", 68, 3), ("bf16", 7168, 0)])
@pytest.mark.parametrize("W,R,k,E", [(1, 1, 8, 16), (1, 301, 6, 40), (4, 77, 33, 8)])
def test_sorted_rows(W, R, k, E, dtype, hidden, sd):
    g = _gen(hidden + R)
    t = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": F8, "f32": torch.float32}[dtype]
    x = _randn(g, W, R, hidden).to(t)
    scales = torch.rand(W, R, sd, generator=g, device=DEV) if sd else None
    idx = _indices(g, W, R, k, E)
    if W == 1:
        x, idx1, scales = x[0], idx[0], scales[0] if sd else None
    else:
        idx1 = idx
    order = ep.sort_by_expert(idx1, E)
    n = int(order.offsets[-1])
    xs, ss = ep.sorted_rows(order, x, scales)
    rows = (order.src[:n] // k).long()
    raw = x.reshape(W * R, hidden).contiguous().view(torch.uint8).view(W * R, -1)
    assert torch.equal(xs.view(torch.uint8).view(len(xs), -1)[:n], raw[rows])
    if sd:
        assert torch.equal(ss[:n], scales.reshape(W * R, sd)[rows])
    else:
        assert ss is None


def _return64(y, w, pos):
    here = pos >= 0
    v = y.double()[pos.clamp_min(0).long()] * torch.where(here, w.double(), 0.0)[..., None]
    return torch.where(here[..., None], v, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,k,E,hidden", [(1100, 8, 24, 1040), (1, 1, 4, 8), (1, 8, 64, 7168), (513, 6, 96, 2056), (130, 33, 40, 264),
                                          (64, 64, 100, 1000), (1531, 2, 8, 512)])
def test_return_rows_and_gradients(R, k, E, hidden, dtype):
    g, t = _gen(R + hidden), HALF[dtype]
    order = ep.sort_by_expert(_indices(g, 1, R, k, E, bad=0.3)[0], E)
    n = int(order.offsets[-1])
    y = _randn(g, R * k, hidden).to(t)
    y[n:] = float("nan")                                 # rows past the last are not read
    w = _randn(g, R, k)
    w[order.pos < 0] = float("inf")                      # nor the weights of slots without a row
    terms = _return64(y, w, order.pos)
    want = terms.sum(1)
    _within(ep.return_rows(order, y, w), want, _half_bound(t, want) + 2 * (k + 1) * U * terms.abs().sum(1), "return")
    ones = _return64(y, torch.ones_like(w), order.pos)
    want = ones.sum(1)
    _within(ep.sorted_rows_backward(order, y), want, _half_bound(t, want) + 2 * (k + 1) * U * ones.abs().sum(1), "sum")

    dout = _randn(g, R, hidden).to(t)
    dy, dw = ep.return_rows_backward(order, y, w, dout)
    src = order.src[:n].long()
    assert torch.equal(dy[:n], (w.reshape(-1)[src][:, None] * dout.float()[src // k]).to(t))
    here = order.pos >= 0
    prod = torch.where(here[..., None], y.double()[order.pos.clamp_min(0).long()], 0.0) * dout.double()[:, None]
    _within(dw, prod.sum(-1), hidden * U * prod.abs().sum(-1), "dweights")
    assert not dw[~here].any()

    # differences of the 64-bit definition along a random direction; it is linear in y and in w
    vy, vw = _randn(g, n, hidden).double(), torch.where(here, _randn(g, R, k).double(), 0.0)
    loss = lambda yy, ww: (_return64(yy, ww, order.pos).sum(1) * dout.double()).sum()  # noqa: E731
    y64, w64 = y.double(), torch.where(here, w.double(), 0.0)
    y64[n:] = 0
    step = torch.zeros_like(y64)
    step[:n] = vy
    by = (loss(y64 + step, w64) - loss(y64 - step, w64)) / 2
    bw = (loss(y64, w64 + vw) - loss(y64, w64 - vw)) / 2
    slack = 1e-9 * (y64.abs().sum() * dout.abs().double().sum()).sqrt()
    _within((dy[:n].double() * vy).sum(), by, (_half_bound(t, dy[:n].double()) * vy.abs()).sum() * 1.01 + slack, "by y")
    _within((dw.double() * vw).sum(), bw, (hidden * U * prod.abs().sum(-1) * vw.abs()).sum() + slack, "by w")


def test_rows_past_counts_are_not_written():
    W, R, k, E, H = 4, 50, 4, 8, 64
    g = _gen(9)
    counts = torch.tensor([50, 0, 17, 1], dtype=torch.int32, device=DEV)
    order = ep.sort_by_expert(_indices(g, W, R, k, E), E, counts=counts)
    n = int(order.offsets[-1])
    y = _randn(g, W * R * k, H).to(torch.bfloat16)
    w = torch.rand(W, R, k, generator=g, device=DEV)
    out = torch.zeros(W, R, H, dtype=torch.bfloat16, device=DEV)
    lib = ep.load_library()
    s = ep.experts._status_word(DEV)
    rc = lib.ep_return_rows(y.data_ptr(), w.data_ptr(), order.pos.data_ptr(), counts.data_ptr(), W, R, k, y.shape[0], H,
                            ep.EP_BF16, out.data_ptr(), s.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    terms = _return64(y, w, order.pos)
    for r in range(W):
        c = int(counts[r])
        want = terms[r, :c].sum(1)
        _within(out[r, :c], want, _half_bound(y.dtype, want) + 2 * 5 * U * terms[r, :c].abs().sum(1), "return")
        assert not out[r, c:].any()
    assert n == int((order.pos >= 0).sum())


def test_positions_outside_the_buffer_are_recorded_and_skipped():
    pos = torch.tensor([[0, 7], [-2, 1]], dtype=torch.int32, device=DEV)
    order = ep.ExpertOrder(torch.zeros(1, dtype=torch.int32, device=DEV), pos,
                           torch.zeros(2, dtype=torch.int32, device=DEV))
    y = torch.ones(2, 16, dtype=torch.bfloat16, device=DEV)
    out = ep.return_rows(order, y)
    assert ep.op_status(DEV) == ep.EP_ERR_DEVICE_BOUNDS
    assert torch.equal(out, y)


# ------------------------------------------------------------------------------------------- product

def _fp8_rows(g, rows, width, spread=0.5):
    x = _randn(g, rows, width) * torch.exp(spread * _randn(g, rows, 1))
    xb = torch.nn.functional.pad(x, (0, _blocks(width) * 128 - width)).view(rows, -1, 128)
    s = (xb.abs().amax(-1) / 448).clamp_min(1e-20)
    return (xb / s[..., None]).view(rows, -1)[:, :width].to(F8).contiguous(), s.contiguous()


def _product_inputs(g, rows, K, N, groups):
    a, sa = _fp8_rows(g, rows, K)
    b = (100 * _randn(g, groups, N, K)).clamp(-448, 448).to(F8)
    sb = torch.rand(groups, _blocks(N), _blocks(K), generator=g, device=DEV) * 1e-3
    return a, sa, b, sb


def _product64(a, sa, b, sb):
    """(product, sum of |terms|) of one group in 64 bits."""
    K, N = a.shape[1], b.shape[0]
    a64 = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    b64 = b.double() * sb.double().repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]
    return a64 @ b64.t(), a64.abs() @ b64.abs().t()


def _edges(rows, groups, g):
    """Ragged offsets with empty groups among them."""
    if groups == 1:
        return [0, rows]
    cut = torch.randint(0, rows + 1, (groups - 1,), generator=g, device=DEV).sort().values.tolist()
    cut[len(cut) // 2] = cut[len(cut) // 2 - 1] if len(cut) > 1 else cut[0]
    return [0, *cut, rows]


def _check_product(a, sa, b, sb, edges, dtype="bf16", swiglu=False, stream=None):
    K, N = a.shape[1], b.shape[1]
    if edges is None:
        offsets, bb, ss, edges = None, b[0], sb[0], [0, a.shape[0]]
    else:
        offsets, bb, ss = torch.tensor(edges, dtype=torch.int32, device=DEV), b, sb
    # products of codes are exact; their sums take at most 128 additions a block and one FMA per
    # block, each off by 2 u at most where a matrix unit truncates; the scales' product by u
    rel = 2 * (128 + _blocks(K) + 2) * U
    if swiglu:
        q, s = ep.matmul_fp8_swiglu(a, sa, bb, ss, offsets=offsets, stream=stream)
    else:
        out = ep.matmul_fp8(a, sa, bb, ss, offsets=offsets, out_dtype=dtype, stream=stream)
    torch.cuda.synchronize()
    for i in range(len(edges) - 1):
        lo, hi = edges[i], edges[i + 1]
        if lo == hi:
            continue
        z, mag = _product64(a[lo:hi], sa[lo:hi], b[i], sb[i])
        if not swiglu:
            _within(out[lo:hi], z, _half_bound(out.dtype, z) + 1.01 * rel * mag, f"group {i}")
            continue
        half = N // 2
        gate, up = z[:, :half], z[:, half:]
        sig = 1 / (1 + torch.exp(-gate))
        want = gate * sig * up
        # d silu <= 1.1 d gate; the exponential, quotient and products: under 16 u in all
        err = rel * (1.1 * mag[:, :half] * up.abs() + (gate * sig).abs() * mag[:, half:]) * 1.01 + 16 * U * want.abs()
        _check_codes(q[lo:hi], s[lo:hi], want, err)


SHAPES = [(1, 16, 8, 0), (1, 7168, 512, 0), (3, 144, 24, 0), (65, 128, 129, 0), (128, 256, 256, 0), (129, 272, 264, 0),
          (300, 1040, 520, 0), (1000, 512, 384, 0), (257, 2048, 1024, 0), (5, 1040, 130, 3), (40, 512, 272, 7),
          (64, 2048, 512, 64), (700, 1040, 520, 6), (1500, 512, 640, 5), (2100, 1024, 768, 3), (33, 256, 96, 40),
          (4000, 256, 512, 9), (17, 4096, 7, 0), (520, 144, 1, 2), (50, 640, 288, 0), (64, 2064, 1184, 0),
          (100, 272, 192, 8), (96, 128, 2048, 0), (31, 1024, 20000, 0), (700, 64, 40, 600), (12000, 32, 16, 600),
          (9000, 16, 32, 4096), (66, 4096, 512, 0), (130, 3088, 1000, 0), (200, 7168, 2048, 0), (300, 3600, 1312, 0),
          (90, 4096, 544, 5), (129, 3200, 257, 2), (1000, 4096, 96, 0), (20, 1536, 528, 0), (40, 3200, 640, 0), (64, 1536, 96, 8),
          (2000, 1040, 712, 0), (777, 144, 300, 3)]


@pytest.mark.parametrize("rows,K,N,groups", SHAPES)
def test_product(rows, K, N, groups):
    g = _gen(rows + K + N)
    args = _product_inputs(g, rows, K, N, max(1, groups))
    edges = _edges(rows, groups, g) if groups else None
    for dtype in ("bf16", "fp16"):
        _check_product(*args, edges, dtype)


@pytest.mark.parametrize("rows,K,N,groups", [s for s in SHAPES if s[2] % 32 == 0] + [(77, 400, 160, 0), (900, 256, 544, 4)])
def test_product_swiglu(rows, K, N, groups):
    g = _gen(rows + K + N + 1)
    args = _product_inputs(g, rows, K, N, max(1, groups))
    _check_product(*args, _edges(rows, groups, g) if groups else None, swiglu=True)


@pytest.mark.parametrize("rows", [5, 700])
def test_product_swiglu_of_gates_far_from_zero(rows):
    """Gates from single digits to past 1000, where the sigmoid is 0 or 1 to every digit."""
    g = _gen(rows)
    a, sa, b, sb = _product_inputs(g, rows, 256, 256, 1)
    sa *= torch.logspace(0, 2.5, rows, device=DEV)[:, None]
    z, _ = _product64(a, sa, b[0], sb[0])
    assert z[:, :128].max() > 100 and z[:, :128].min() < -100
    _check_product(a, sa, b, sb, None, swiglu=True)


@pytest.mark.parametrize("rows,K", [(6, 256), (700, 256), (256, 4096)])
def test_product_swiglu_of_small_sigmoids_times_large_values(rows, K):
    """gate * up alone would pass FP32's range; with the sigmoid between them the product does not."""
    one = torch.full((1, 1), 0x38, dtype=torch.uint8, device=DEV)                 # 1.0
    a, b = one.expand(rows, K).contiguous().view(F8), one.expand(256, K).contiguous()
    b[:128] = 0xB8                                                                # -1.0
    sb = torch.full((2, K // 128), 80.0 / K, device=DEV)
    sb[1] = 3e37 / K
    f = torch.linspace(0.25, 1.05, rows, device=DEV)
    sa = f[:, None].expand(rows, K // 128).contiguous()
    q, s = ep.matmul_fp8_swiglu(a, sa, b.view(F8), sb)
    z, _ = _product64(a, sa, b.view(F8), sb)
    gate, up = z[:, :128], z[:, 128:]
    assert (gate * up).abs().max() > 3.5e38 and gate.min() < -80
    want = gate / (1 + torch.exp(-gate)) * up
    # the sums' error in the gate enters by its own size (the exponential), the exponential's argument is off
    # by less than 2^-25 |gate| (log2 e in FP32), and the rest by less than 32 u
    err = want.abs() * (2 * (130 + K // 128) * U * (gate.abs() + 1) + 2.0 ** -25 * gate.abs() + 32 * U) * 1.01
    _check_codes(q, s, want, err)
    # a sigmoid below FP32's smallest normal number counts as zero
    sa[:] = 1.25
    q, s = ep.matmul_fp8_swiglu(a, sa, b.view(F8), sb)
    assert not q.float().any() and (s == 1).all()


def test_product_swiglu_codes_do_not_depend_on_the_number_of_rows():
    """With one block of K and whole-number codes every kernel has the same sums, so the same codes."""
    for seed in range(16):
        g = _gen(seed)
        a = torch.randint(-8, 9, (200, 128), generator=g, device=DEV).float().to(F8)
        b = torch.randint(-8, 9, (131072, 128), generator=g, device=DEV).float().to(F8)
        sa = 0.002 * torch.rand(200, 1, generator=g, device=DEV)
        sb = torch.rand(1024, 1, generator=g, device=DEV)
        q, s = ep.matmul_fp8_swiglu(a, sa, b, sb)
        few, s_few = ep.matmul_fp8_swiglu(a[:32].contiguous(), sa[:32].contiguous(), b, sb)
        assert torch.equal(s[:32], s_few)
        assert torch.equal(q[:32].view(torch.uint8), few.view(torch.uint8)), seed


@pytest.mark.parametrize("rows", [2, 20, 60, 100, 140, 1000])
def test_product_all_rows_in_one_of_many_groups(rows):
    g = _gen(rows)
    args = _product_inputs(g, rows, 256, 256, 12)
    _check_product(*args, [0] * 8 + [rows] * 5)
    _check_product(*args, [0] * 8 + [rows] * 5, swiglu=True)


@pytest.mark.parametrize("rows", [30, 1200])
def test_product_leaves_rows_outside_the_groups_alone(rows):
    g = _gen(rows)
    a, sa, b, sb = _product_inputs(g, rows, 256, 192, 3)
    lo, mid, hi = rows // 5, rows // 2, rows - 3
    offsets = torch.tensor([lo, mid, mid, hi], dtype=torch.int32, device=DEV)
    out = torch.full((rows, 192), 7.0, dtype=torch.bfloat16, device=DEV)
    word = ep.experts._status_word(DEV)
    rc = ep.load_library().ep_matmul_fp8(
        a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), offsets.data_ptr(), rows, 3, 192, 256, 0, ep.EP_BF16,
        out.data_ptr(), None, word.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert (out[:lo] == 7).all() and (out[hi:] == 7).all()
    for i, (m0, m1) in enumerate([(lo, mid), (mid, mid), (mid, hi)]):
        z, mag = _product64(a[m0:m1], sa[m0:m1], b[i], sb[i])
        _within(out[m0:m1], z, _half_bound(out.dtype, z) + 2.02 * 132 * U * mag, f"group {i}")


@pytest.mark.parametrize("rows", [6, 400])
def test_product_non_finite_codes_stay_in_their_row(rows):
    """A NaN code makes its row's outputs NaN (and a weight's NaN its column's), and no others."""
    g = _gen(rows)
    a, sa, b, sb = _product_inputs(g, rows, 384, 160, 2)
    a.view(torch.uint8)[rows // 2, 300] = 0x7F
    b.view(torch.uint8)[1, 77, 5] = 0x7F
    offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
    out = ep.matmul_fp8(a, sa, b, sb, offsets=offsets)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[rows // 2] = True
    want[rows // 3:, 77] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("rows", [9, 600])
def test_product_on_another_stream_and_empty(rows):
    g = _gen(2)
    args = _product_inputs(g, rows, 512, 256, 1)
    torch.cuda.synchronize()
    _check_product(*args, None, stream=torch.cuda.Stream())
    a, sa, b, sb = args
    assert ep.matmul_fp8(a[:0], sa[:0], b[0], sb[0]).shape == (0, 256)
    q, s = ep.matmul_fp8_swiglu(a[:0], sa[:0], b[0], sb[0])
    assert q.shape == (0, 128) and s.shape == (0, 1)


@pytest.mark.parametrize("rows", [8, 900])
def test_product_is_deterministic(rows):
    g = _gen(3)
    a, sa, b, sb = _product_inputs(g, rows, 7168, 512, 4)
    offsets = torch.tensor(_edges(rows, 4, g), dtype=torch.int32, device=DEV)
    one = ep.matmul_fp8(a, sa, b, sb, offsets=offsets)
    for _ in range(5):
        assert torch.equal(one, ep.matmul_fp8(a, sa, b, sb, offsets=offsets))


# ------------------------------------------------------------------------------------------- past 32 bits

def test_norm_past_32_bits():
    rows, hidden = 300000, 8192                                     # 2.46e9 elements
    x = torch.empty(rows, hidden, dtype=torch.bfloat16, device=DEV)
    x[-3:] = _randn(_gen(1), 3, hidden).to(x.dtype)
    w = torch.ones(hidden, device=DEV)
    q, s, h, _ = ep.rms_norm_fp8(x, w, residual=x)
    q2, s2, h2, _ = ep.rms_norm_fp8(x[-3:], w, residual=x[-3:])
    assert torch.equal(q[-3:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-3:], s2) and torch.equal(h[-3:], h2)


def test_sorted_rows_and_return_past_32_bits():
    R, k, E, H = 40000, 8, 16, 4096                                 # 320000 sorted rows of 8 KB: 2.6 GB
    g = _gen(2)
    idx = torch.rand(R, E, generator=g, device=DEV).topk(k, 1).indices.int()
    x = _randn(g, R, H).to(torch.bfloat16)
    order = ep.sort_by_expert(idx, E)
    xs, _ = ep.sorted_rows(order, x)
    last = order.src[-50:].long()
    assert torch.equal(xs[-50:], x[last // k])
    w = torch.softmax(_randn(g, R, k), 1)
    rows = last // k                                                # rows with a slot at the far end
    out = ep.return_rows(order, xs, w)
    want = (x[rows].double()[:, None] * w[rows].double()[..., None])
    _within(out[rows], want.sum(1), _half_bound(out.dtype, want.sum(1)) + 2 * 9 * U * want.abs().sum(1), "return")
    dout = _randn(g, R, H).to(torch.bfloat16)
    dy, dw = ep.return_rows_backward(order, xs, w, dout)
    assert torch.equal(dy[-50:], (w.reshape(-1)[last][:, None] * dout[rows].float()).to(dy.dtype))
    dots = x[rows].double() * dout[rows].double()
    _within(dw[rows], dots.sum(1)[:, None].expand(-1, k), (H * U * dots.abs().sum(1))[:, None], "dweights")


@pytest.mark.parametrize("swiglu", [False, True])
def test_product_past_32_bits(swiglu):
    rows, K, N = 530000, 64, 8192                                   # 4.3e9 outputs, 2.2e9 with SwiGLU
    g = _gen(3)
    a, sa = _fp8_rows(g, rows, K)
    b = (100 * _randn(g, 2, N, K)).clamp(-448, 448).to(F8)
    sb = torch.rand(2, _blocks(N), 1, generator=g, device=DEV) * 1e-3
    cut = rows - 200                                                # the last group is the last 200 rows
    offsets = torch.tensor([0, cut, rows], dtype=torch.int32, device=DEV)
    one = torch.tensor([0, 200, 200], dtype=torch.int32, device=DEV)
    if swiglu:
        q, s = ep.matmul_fp8_swiglu(a, sa, b, sb, offsets=offsets)
        q2, s2 = ep.matmul_fp8_swiglu(a[cut:], sa[cut:], b.flip(0), sb.flip(0), offsets=one)
        assert torch.equal(q[cut:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[cut:], s2)
        return
    out = ep.matmul_fp8(a, sa, b, sb, offsets=offsets)
    z, mag = _product64(a[cut:], sa[cut:], b[1], sb[1])
    _within(out[cut:], z, _half_bound(out.dtype, z) + 2.02 * 131 * U * mag, "the last group")


# ------------------------------------------------------------------------------------------- refusals

def _zeros(shape, dtype):
    t = torch.zeros(shape, dtype=torch.uint8 if dtype == F8 else dtype, device=DEV)
    return t.view(F8) if dtype == F8 else t


def test_binding_names_the_argument_at_fault():
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x = _zeros((4, 256), bf)
    order = ep.ExpertOrder(_zeros((5,), i32), _zeros((4, 2), i32), _zeros((8,), i32))
    y, w = _zeros((8, 256), bf), _zeros((4, 2), f32)
    a, sa, b, sb = _zeros((4, 128), F8), _zeros((4, 1), f32), _zeros((64, 128), F8), _zeros((1, 1), f32)
    many = (_zeros((3, 64, 128), F8), _zeros((3, 1, 1), f32))
    cases = [
        (lambda: ep.rms_norm_fp8(_zeros((4, 256), f32), _zeros((256,), f32)), "x is Float"),
        (lambda: ep.rms_norm_fp8(x[0], x[0]), "x has 1 dimensions"),
        (lambda: ep.rms_norm_fp8(x.t(), _zeros((4,), bf)), "not consecutive"),
        (lambda: ep.rms_norm_fp8(x, _zeros((128,), bf)), "weight has shape"),
        (lambda: ep.rms_norm_fp8(x, _zeros((256,), torch.float16)), "weight is Half"),
        (lambda: ep.rms_norm_fp8(x, x[0], residual=_zeros((4, 128), bf)), "residual is"),
        (lambda: ep.rms_norm_fp8(x[:, :24].contiguous(), x[0, :24].contiguous()), "hidden=24"),
        (lambda: ep.rms_norm_fp8(x[:, 4:132], x[0, :128].contiguous()), "16-byte aligned"),
        (lambda: ep.sort_by_expert(_zeros((4, 2), torch.int64), 4), "indices is Long"),
        (lambda: ep.sort_by_expert(_zeros((4,), i32), 4), "indices has 1 dimensions"),
        (lambda: ep.sort_by_expert(_zeros((2, 4, 2), i32), 4, counts=_zeros((3,), i32)), "counts has shape"),
        (lambda: ep.sort_by_expert(_zeros((4, 2), i32), 0), "experts_per_rank"),
        (lambda: ep.sort_by_expert(_zeros((4, 2), i32), 5000), "experts_per_rank"),
        (lambda: ep.sort_by_expert(_zeros((4, 2), i32), 4, max_rows=-1), "max_rows"),
        (lambda: ep.sort_by_expert(_zeros((4, 65), i32), 4), "topk=65"),
        (lambda: ep.sort_by_expert(_zeros((4, 2), i32)[:, :1], 4), "indices is not contiguous"),
        (lambda: ep.sorted_rows(order, _zeros((5, 256), bf)), "order.pos has shape"),
        (lambda: ep.sorted_rows(order, _zeros((4, 12), bf)), "row of 24 bytes"),
        (lambda: ep.sorted_rows(order, x, _zeros((4, 2), bf)), "scales is BFloat16"),
        (lambda: ep.return_rows(order, x), "y has shape"),
        (lambda: ep.return_rows(order, y, _zeros((4, 3), f32)), "weights has shape"),
        (lambda: ep.return_rows(order, y.float()), "y is Float"),
        (lambda: ep.return_rows_backward(order, y, None, x), "weights is a NoneType"),
        (lambda: ep.return_rows_backward(order, y, w, x.half()), "dout is Half"),
        (lambda: ep.matmul_fp8(a, sa, _zeros((64, 256), F8), sb), "b has shape"),
        (lambda: ep.matmul_fp8(a, sa, b, _zeros((2, 1), f32)), "b_scales has shape"),
        (lambda: ep.matmul_fp8(a, _zeros((4, 2), f32), b, sb), "a_scales has shape"),
        (lambda: ep.matmul_fp8(a, sa, *many, offsets=_zeros((3,), i32)), "offsets has shape"),
        (lambda: ep.matmul_fp8(a, sa, *many), "b has shape"),
        (lambda: ep.matmul_fp8(a.view(torch.uint8), sa, b, sb), "a is Byte"),
        (lambda: ep.matmul_fp8_swiglu(a, sa, _zeros((48, 128), F8), sb), "columns=48"),
        (lambda: ep.matmul_fp8(a, sa, b.cpu(), sb), "b is on cpu"),
    ]
    for call, words in cases:
        with pytest.raises(ep.EpError) as e:
            call()
        assert e.value.code == ep.EP_ERR_ARG and words in str(e.value), (words, str(e.value))


def test_a_refused_launch_is_reported_by_its_own_call_only():
    """A launch into the legacy stream is refused while another stream captures.  The call returns that error; the
    runtime's record of it, which the next caller's check would read, is clear."""
    rt, lib = ctypes.CDLL("libcudart.so.13"), ep.load_library()
    y, pos, out, word = _zeros((2, 16), torch.bfloat16), _zeros((1, 1), torch.int32), _zeros((1, 16), torch.bfloat16), \
        ep.experts._status_word(DEV)
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    try:
        rc = lib.ep_return_rows(y.data_ptr(), None, pos.data_ptr(), None, 1, 1, 1, 2, 16, ep.EP_BF16, out.data_ptr(),
                                word.data_ptr(), None)
        left = rt.cudaPeekAtLastError()
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaGetLastError()
        rt.cudaStreamDestroy(stream)
    assert rc == ep.EP_ERR_CUDA and b"Capture" in lib.ep_last_error()
    assert left == 0


# ------------------------------------------------------------------------------------------- together

def test_dispatched_rows_through_the_experts():
    """FP8 dispatch, sort, both products, weighted return, combine: against the layer in 64 bits.

    The hidden quantisation rounds to e4m3, so the comparison is by norms: each quantiser is off by at
    most 2^-4 per element, and the two of them (rows and hidden) leave less than 2^-3 of the output."""
    wl = wlmod.custom_workload(W=4, E=6, k=4, H=256, M=48, n_tok=[48, 0, 17, 33], seed=2)
    W, E, k, H, M, inner = wl.W, wl.E, wl.k, wl.H, wl.M, 160
    g = _gen(4)
    x = _randn(g, W * M, H).to(torch.bfloat16)
    q, s, _, y = ep.rms_norm_fp8(x, torch.ones(H, device=DEV), want_y=True)
    idx = torch.from_numpy(wl.indices).to(DEV)
    w = torch.from_numpy(wl.weights).to(DEV)
    b1 = (100 * _randn(g, W * E, 2 * inner, H)).clamp(-448, 448).to(F8)
    s1 = torch.full((W * E, _blocks(2 * inner), _blocks(H)), 1e-3, device=DEV)
    b2 = (100 * _randn(g, W * E, H, inner)).clamp(-448, 448).to(F8)
    s2 = torch.full((W * E, _blocks(H), _blocks(inner)), 1e-3, device=DEV)
    with ep.Plan(W, E, k, H, "fp8", H // 128, M, device=DEV) as plan:
        d = plan.dispatch(q.view(W, M, H), w, s.view(W, M, -1), idx, wl.n_tok)
        order = plan.sort_received(d)
        xs, ss = ep.sorted_rows(order, d.recv_x, d.recv_scales)
        hq, hs = ep.matmul_fp8_swiglu(xs, ss, b1, s1, offsets=order.offsets)
        z = ep.matmul_fp8(hq, hs, b2, s2, offsets=order.offsets)
        out, _ = plan.combine(ep.return_rows(order, z, d.recv_w), None, d.epoch)
        assert plan.status() == 0
    y64 = _norm64(x, torch.ones(H, device=DEV), None, 1e-6)[1].view(W, M, H)
    for r in range(W):
        for t in range(int(wl.n_tok[r])):
            want = torch.zeros(H, dtype=torch.float64, device=DEV)
            for j in range(k):
                e = int(wl.indices[r, t, j])
                h1 = (b1[e].double() * 1e-3) @ y64[r, t]
                h1 = h1[:inner] / (1 + torch.exp(-h1[:inner])) * h1[inner:]
                want += float(wl.weights[r, t, j]) * ((b2[e].double() * 1e-3) @ h1)
            assert (out[r, t].double() - want).norm() <= 2.0 ** -3 * want.norm(), (r, t)
        assert not out[r, int(wl.n_tok[r]):].any()


def test_sort_received_refuses_a_dispatch_that_is_not_live():
    wl = wlmod.custom_workload(W=2, E=4, k=2, H=128, M=16, n_tok=[16, 9], seed=3)
    idx = torch.from_numpy(wl.indices).to(DEV)
    x = _randn(_gen(1), 2, 16, 128).to(torch.bfloat16)

    def refused(plan, d):
        with pytest.raises(ep.EpError) as e:
            plan.sort_received(d)
        assert e.value.code == ep.EP_ERR_STATE
    with ep.Plan(2, 4, 2, 128, "bf16", 0, 16, device=DEV) as plan:
        d = plan.dispatch(x, None, None, idx, wl.n_tok)
        plan.sort_received(d)
        d2 = plan.dispatch(x, None, None, idx, wl.n_tok)
        refused(plan, d)
        plan.sort_received(d2)
        d3 = plan.dispatch_route(idx, wl.n_tok)
        refused(plan, d3)                      # routed, but no row has arrived
        plan.dispatch_scatter(x, None, None, idx)
        plan.sort_received(d3)
        plan.reset()
        refused(plan, d3)


def test_sort_received_of_many_rows():
    """Above 131072 pairs, with the dispatch's own counts."""
    wl = wlmod.custom_workload(W=4, E=8, k=8, H=128, M=1100, n_tok=[1100, 0, 1000, 7], seed=5)
    idx = torch.from_numpy(wl.indices).to(DEV)
    with ep.Plan(4, 8, 8, 128, "bf16", 0, 1100, device=DEV) as plan:
        d = plan.dispatch(_randn(_gen(1), 4, 1100, 128).to(torch.bfloat16), None, None, idx, wl.n_tok)
        assert d.recv_idx.numel() > 131072
        order = plan.sort_received(d)
        want = _sort_np(d.recv_idx, 8, d.recv_count.tolist(), 4 * 1100 * 8)
        for name, w in zip(("offsets", "pos", "src"), want):
            assert np.array_equal(getattr(order, name).cpu().numpy().reshape(w.shape), w), name
        held = wl.indices[np.arange(1100)[None, :] < np.asarray(wl.n_tok)[:, None]]
        assert int(order.offsets[-1]) == (held >= 0).sum()


def test_calls_replay_in_a_graph():
    g = _gen(11)
    R, k, E, H = 40, 4, 8, 256
    x = _randn(g, R, H).to(torch.bfloat16)
    idx = _indices(g, 1, R, k, E, bad=0)[0]
    w = torch.softmax(_randn(g, R, k), 1)
    weight = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    _, _, b, sb = _product_inputs(g, 1, H, 2 * H, E)
    _, _, b2, sb2 = _product_inputs(g, 1, H, H, E)

    def layer():
        q, s, _, _ = ep.rms_norm_fp8(x, weight)
        order = ep.sort_by_expert(idx, E)
        xs, ss = ep.sorted_rows(order, q, s)
        hq, hs = ep.matmul_fp8_swiglu(xs, ss, b, sb, offsets=order.offsets)
        return ep.return_rows(order, ep.matmul_fp8(hq, hs, b2, sb2, offsets=order.offsets), w)

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    x2 = _randn(g, R, H).to(torch.bfloat16)
    graph.replay()
    assert torch.equal(out, want)
    x.copy_(x2)
    graph.replay()
    assert torch.equal(out, layer())


def test_example_layer_agrees_with_fp32():
    """The example's layer quantises the rows twice; see the bound of the test above."""
    from combine_ep_dispatch_02_gb300 import expert_layer
    assert expert_layer.main(["--tokens-per-rank", "33", "--hidden", "512", "--inner", "272", "--passes", "2"]) <= 2.0 ** -3
    assert expert_layer.main(["--ranks", "1", "--experts-per-rank", "4", "--topk", "2", "--tokens-per-rank", "1",
                              "--hidden", "256", "--passes", "1"]) <= 2.0 ** -3


def test_example_layer_with_a_short_last_block_of_scales():
    from combine_ep_dispatch_02_gb300 import expert_layer
    assert expert_layer.main(["--tokens-per-rank", "20", "--hidden", "272", "--inner", "144", "--passes", "1"]) <= 2.0 ** -3


def test_back_to_back_calls_touch_nothing_early():
    """A call's kernels are set up while the kernel before them still runs; their memory is the allocator's
    and so often what that kernel reads.  Results of a stream of calls are those of calls one by one."""
    g = _gen(21)
    H, E, R, k = 512, 8, 24, 4
    w = (1 + 0.1 * _randn(g, H)).to(torch.bfloat16)
    _, _, b, sb = _product_inputs(g, 1, H, 2 * H, E)
    _, _, b2, sb2 = _product_inputs(g, 1, H, H, E)
    base = _randn(g, R, H).to(torch.bfloat16)
    idx = torch.rand(R, E, generator=g, device=DEV).topk(k, 1).indices.int()
    wt = torch.softmax(_randn(g, R, k), 1)

    def passes(wait):
        x, i, done = base.clone(), idx.clone(), []
        step = torch.cuda.synchronize if wait else (lambda: None)
        for _ in range(60):
            q, s, h, y = ep.rms_norm_fp8(x, w, residual=x, want_y=True)
            step()
            i = (i + 1) % E
            order = ep.sort_by_expert(i, E)
            step()
            xs, ss = ep.sorted_rows(order, q, s)
            step()
            z, zs = ep.matmul_fp8_swiglu(xs, ss, b, sb, offsets=order.offsets)
            step()
            o = ep.matmul_fp8(z, zs, b2, sb2, offsets=order.offsets)
            step()
            out = ep.return_rows(order, o, wt)
            dy, dw = ep.return_rows_backward(order, o, wt, y)
            step()
            x = (0.5 * y.float() + 0.05 * out.float().tanh()).to(torch.bfloat16)
            done += [x, dw, dy[:3].clone()]
        torch.cuda.synchronize()
        return done
    for a, c in zip(passes(True), passes(False)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("W,R,k,E", [(1, 1500, 8, 40), (4, 4500, 8, 16)])
def test_sorts_of_several_launches_read_nothing_early(W, R, k, E):
    """The two- and three-launch sorts on indices and counts that the kernels just before them write, in memory
    that an earlier pass has read: as calls one by one."""
    g = _gen(R)
    base = torch.stack([_indices(g, W, R, k, E, bad=0.05) for _ in range(2)])
    held = torch.tensor([[R] * W, [R // (r + 2) for r in range(W)]], dtype=torch.int32, device=DEV)
    idx, counts = torch.empty_like(base[0]), torch.empty_like(held[0])
    view = idx if W > 1 else idx[0]

    def passes(wait):
        step, done = torch.cuda.synchronize if wait else (lambda: None), []
        for i in range(40):
            torch.add(base[i % 2], 0, out=idx)
            torch.add(held[i // 2 % 2], 0, out=counts)
            step()
            order = ep.sort_by_expert(view, E, counts=counts)
            step()
            done += [order.offsets, order.pos, order.src]
        torch.cuda.synchronize()
        return done
    for a, b in zip(passes(False), passes(True)):
        assert torch.equal(a, b)
    order = ep.sort_by_expert(view, E, counts=counts)      # the last pass's
    want = _sort_np(base[1], E, held[1].tolist(), base[1].numel())
    for name, w in zip(("offsets", "pos", "src"), want):
        assert np.array_equal(getattr(order, name).cpu().numpy().reshape(w.shape), w), name


# ------------------------------------------------------------------------------------------- host threads

def _on_two_threads(calls, passes):
    """Each call `passes` times on a thread and a stream of its own: the messages of those that were refused."""
    failed, start = [[] for _ in calls], threading.Barrier(len(calls))

    def work(i):
        with torch.cuda.device(DEV):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                torch.zeros(1, device=DEV)     # the thread has used the device before
            start.wait()
            for _ in range(passes):
                if calls[i](s.cuda_stream) != ep.EP_OK:
                    failed[i].append(ep.load_library().ep_last_error())
            s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed


@pytest.mark.parametrize("dense,grouped,groups,K", [(4, 1600, 400, 2048), (160, 2400, 100, 128)])
def test_products_of_two_host_threads_do_not_disturb_each_other(dense, grouped, groups, K):
    """ctypes releases the interpreter's lock, so the calls run at the same time; their kernel is the same, the
    shared memory that their numbers of groups take is not."""
    lib, calls, keep = ep.load_library(), [], []
    for n, G in ((dense, 1), (grouped, groups)):
        a, sa, b, sb = _product_inputs(_gen(n), n, K, 16, G)
        offsets = torch.linspace(0, n, G + 1, device=DEV).int()
        out, word = torch.empty(n, 16, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        keep.append((a, sa, b, sb, offsets, out, word))
        calls.append(lambda s, p=[t.data_ptr() for t in keep[-1]], n=n, G=G: lib.ep_matmul_fp8(
            p[0], p[1], p[2], p[3], p[4], n, G, 16, K, 0, ep.EP_BF16, p[5], None, p[6], s))
    torch.cuda.synchronize()
    assert _on_two_threads(calls, 4000) == [[], []]


@pytest.mark.parametrize("rows", [64, 4096])
def test_sorts_of_two_host_threads_do_not_disturb_each_other(rows):
    lib, g = ep.load_library(), _gen(rows)
    calls, keep = [], []
    for E in (1600, 2048):
        idx = _indices(g, 1, rows, 4, E)
        n = rows * 4
        ws = max(4, lib.ep_sort_workspace_bytes(1, rows, 4, E))
        bufs = [idx] + [torch.empty(m, dtype=torch.int32, device=DEV) for m in (E + 1, n, n, ws // 4)] + \
            [torch.zeros(1, dtype=torch.int32, device=DEV)]
        keep.append(bufs)
        p = [t.data_ptr() for t in bufs]
        calls.append(lambda s, p=p, E=E, n=n, ws=ws: lib.ep_sort_by_expert(
            p[0], None, 1, rows, 4, E, n, p[1], p[2], p[3], p[4], ws, p[5], s))
    torch.cuda.synchronize()
    assert _on_two_threads(calls, 4000) == [[], []]


@pytest.mark.parametrize("rows", [4, 160])
def test_product_as_the_first_call_of_a_host_thread(rows):
    """The allocator has memory of these sizes at hand, so nothing before the product binds the thread to the device."""
    args = _product_inputs(_gen(rows), rows, 256, 128, 1)
    a, sa, b, sb = args[0], args[1], args[2][0], args[3][0]
    want, got = ep.matmul_fp8(a, sa, b, sb).clone(), []
    torch.cuda.synchronize()

    def work():
        try:
            got.append(ep.matmul_fp8(a, sa, b, sb))
        except ep.EpError as e:
            got.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert isinstance(got[0], torch.Tensor), got[0]
    assert torch.equal(got[0], want)


def test_each_recorded_status_is_read_once():
    order = ep.ExpertOrder(torch.zeros(2, dtype=torch.int32, device=DEV),
                           torch.full((1, 1), 7, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV))
    y = torch.ones(2, 16, dtype=torch.bfloat16, device=DEV)
    done, other = threading.Event(), [0]

    def reader():
        while not done.is_set():
            other[0] += ep.op_status(DEV) != 0
    t = threading.Thread(target=reader)
    t.start()
    mine, passes = 0, 1500
    for _ in range(passes):
        ep.return_rows(order, y)               # one lane of one warp records EP_ERR_DEVICE_BOUNDS
        mine += ep.op_status(DEV) != 0
    done.set()
    t.join()
    assert mine + other[0] == passes


def test_taking_a_status_clears_its_word():
    lib, word, taken = ep.load_library(), torch.full((1,), -5, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    for i in range(2):
        assert lib.ep_take_status(word.data_ptr(), taken[i:].data_ptr(), torch.cuda.current_stream().cuda_stream) == ep.EP_OK
    assert taken.tolist() == [-5, 0] and word.item() == 0
