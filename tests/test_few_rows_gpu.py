"""The whole expert layer for a few rows, on the GPU, against its definition in 64 bits (bounds: see test_experts_gpu.py)."""
import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from combine_ep_dispatch_02_gb300.expert_layer import quantise_weights
from test_experts_gpu import DEV, F8, HALF, U, _blocks, _built, _gen, _half_bound, _no_status, _randn, _within  # noqa: F401

pytestmark = pytest.mark.gpu


def _weights64(q, s):
    s = s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * s


def _layer(g, experts, hidden, inner):
    up = quantise_weights(_randn(g, experts, 2 * inner, hidden) * hidden ** -0.5)
    down = quantise_weights(_randn(g, experts, hidden, inner) * inner ** -0.5)
    return (*up, *down)


def _rows(g, rows, hidden, kind):
    x = _randn(g, rows, hidden)
    if kind == "fp8":
        q, s, _, _ = ep.rms_norm_fp8(x.to(torch.bfloat16), torch.ones(hidden, device=DEV))
        return q, s
    return x.to(HALF[kind]), None


def _check(x, xs, idx, w, layer, first=0, out_dtype="bf16"):
    up, ups, down, downs = layer
    rows, hidden = x.shape
    inner = down.shape[2]
    out = ep.moe_few_rows(x, xs, idx, w, *layer, first_expert=first, out_dtype=out_dtype)
    x64 = x.double() if xs is None else x.double() * xs.double().repeat_interleave(128, 1)[:, :hidden]
    want, bound = torch.zeros(rows, hidden, dtype=torch.float64, device=DEV), torch.zeros(rows, hidden, dtype=torch.float64, device=DEV)
    chosen = idx.long() - first
    for e in range(up.shape[0]):
        t = torch.nonzero((chosen == e).any(1))[:, 0]
        if t.numel() == 0:
            continue
        share = (w[t].double() * (chosen[t] == e)).sum(1, keepdim=True)
        share_err = (w[t].double().abs() * (chosen[t] == e)).sum(1, keepdim=True) * idx.shape[1] * U
        w1, w2 = _weights64(up[e], ups[e]), _weights64(down[e], downs[e])
        h, size = x64[t] @ w1.T, x64[t].abs() @ w1.abs().T
        h_err = (hidden + 8) * 2 * U * size
        gate, upper = h.chunk(2, 1)
        gate_err, upper_err = h_err.chunk(2, 1)
        act = gate * torch.sigmoid(gate)
        z = act * upper
        # |d/dg g sigmoid(g)| <= 1.1; the sigmoid's own error; FP16's half step, and what falls below its range
        z_err = 1.1 * gate_err * upper.abs() + act.abs() * upper_err + 1.1 * gate_err * upper_err + 2.0 ** -16 * z.abs()
        z_err = z_err + 2.0 ** -11 * (z.abs() + z_err) + 2.0 ** -37 * z.abs().amax(1, keepdim=True)
        want[t] += share * (z @ w2.T)
        sums = z.abs() @ w2.abs().T
        bound[t] += share.abs() * (z_err @ w2.abs().T + (inner + 8) * 2 * U * sums) + share_err * sums
        bound[t] += (up.shape[0] + 32) * U * (share * (z @ w2.T)).abs()
    # 2^-134: half of BF16's smallest subnormal, the finest that either output type resolves near 0
    _within(out, want, _half_bound(HALF[out_dtype], want) + bound * 1.01 + 2.0 ** -134, "out")
    assert not out[~((chosen >= 0) & (chosen < up.shape[0])).any(1)].any()
    return out


@pytest.mark.parametrize("kind,out_dtype", [("fp8", "bf16"), ("fp16", "fp16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,k,experts,hidden,inner", [
    (1, 1, 1, 16, 16), (1, 8, 32, 1024, 512), (2, 2, 3, 272, 144), (1, 4, 8, 2048, 1024), (5, 6, 24, 2064, 1040),
    (8, 2, 2, 128, 128), (9, 2, 2, 144, 272), (16, 3, 4, 512, 256), (17, 1, 1, 256, 80), (33, 4, 5, 272, 528),
    (64, 8, 16, 512, 1024), (128, 4, 4, 160, 48), (128, 32, 64, 256, 128), (3, 64, 100, 64, 32), (31, 1, 300, 256, 128)])
def test_few_rows(rows, k, experts, hidden, inner, kind, out_dtype):
    g = _gen(rows * 31 + hidden + inner)
    layer = _layer(g, experts, hidden, inner)
    x, xs = _rows(g, rows, hidden, kind)
    # twice as many experts as are here, and slots that were dropped
    idx = torch.rand(rows, 2 * experts + k, generator=g, device=DEV).topk(k, 1).indices.int()
    idx = torch.where(torch.rand(rows, k, generator=g, device=DEV) < 0.1, -1, idx)
    w = torch.softmax(_randn(g, rows, k), 1)
    w[(idx < 0) | (idx >= experts)] = float("nan")        # the weights of what is left out are not read
    _check(x, xs, idx, w.nan_to_num(0) if k > 1 else w, layer, 0, out_dtype)
    out = ep.moe_few_rows(x, xs, idx, w, *layer, out_dtype=out_dtype)
    assert not torch.isnan(out).any()


def test_few_rows_of_another_rank():
    g = _gen(2)
    layer = _layer(g, 6, 256, 128)
    x, xs = _rows(g, 20, 256, "fp8")
    idx = torch.rand(20, 24, generator=g, device=DEV).topk(4, 1).indices.int()
    w = torch.softmax(_randn(g, 20, 4), 1)
    parts = []
    for first in (0, 6, 12, 18, 100, -3):
        parts.append(_check(x, xs, idx, w, layer, first).double())
    assert not parts[4].any() and parts[0].any()
    far = torch.full_like(idx, 2 ** 31 - 1)
    assert not ep.moe_few_rows(x, xs, far, w, *layer, first_expert=-(2 ** 31)).any()


def test_an_expert_named_twice_counts_once_with_both_weights():
    g = _gen(3)
    layer = _layer(g, 4, 256, 128)
    x, xs = _rows(g, 11, 256, "fp8")
    idx = torch.randint(0, 3, (11, 7), generator=g, device=DEV, dtype=torch.int32)
    idx[0] = 2
    w = _randn(g, 11, 7)
    _check(x, xs, idx, w, layer)


def test_all_rows_on_one_expert_and_on_none():
    g = _gen(4)
    layer = _layer(g, 3, 512, 256)
    for rows in (7, 16, 40, 128):
        x, xs = _rows(g, rows, 512, "bf16")
        w = torch.rand(rows, 2, generator=g, device=DEV)
        _check(x, xs, torch.full((rows, 2), 1, dtype=torch.int32, device=DEV), w, layer)
        assert not ep.moe_few_rows(x, xs, torch.full((rows, 2), -1, dtype=torch.int32, device=DEV), w, *layer).any()
    assert ep.moe_few_rows(x[:0], None, torch.zeros((0, 2), dtype=torch.int32, device=DEV), w[:0], *layer).shape == (0, 512)


def test_results_are_the_same_every_time():
    """The places that rows take among an expert's differ from call to call; what they get does not."""
    g = _gen(5)
    layer = _layer(g, 8, 1024, 528)
    x, xs = _rows(g, 8, 1024, "fp8")
    idx = torch.rand(8, 8, generator=g, device=DEV).topk(4, 1).indices.int()
    w = torch.softmax(_randn(g, 8, 4), 1)
    first = ep.moe_few_rows(x, xs, idx, w, *layer)
    for _ in range(20):
        assert torch.equal(ep.moe_few_rows(x, xs, idx, w, *layer), first)


def test_values_far_from_one():
    """Hidden values whose sizes differ by more than FP16's range from expert to expert, row to row and column to
    column: each block of 8 columns has its own power of two."""
    g = _gen(6)
    up, ups, down, downs = _layer(g, 4, 256, 256)
    x, xs = _rows(g, 6, 256, "fp8")
    idx = torch.rand(6, 4, generator=g, device=DEV).topk(2, 1).indices.int()
    w = torch.softmax(_randn(g, 6, 2), 1)
    # the experts' up rows (of z's columns past 128 too) are scaled far up and down, and down back again
    for e, f in enumerate((1e-20, 1e12, 1.0, 1e-6)):
        ups[e, 2:] *= f
        downs[e] /= f
    ups[:, 3] *= 1e-3
    _check(x, xs, idx, w, (up, ups, down, downs))
    big = (x.float() * 1e30 / 448).to(torch.bfloat16)
    big[0, 3], big[1] = 3e38, 1e-38
    ups[:] = 1e-30
    downs[:] = 1.0
    _check(big, None, idx, w, (up, ups, down, downs))


def test_what_is_not_a_number_stays_in_its_row():
    g = _gen(7)
    layer = _layer(g, 4, 256, 128)
    idx = torch.rand(9, 4, generator=g, device=DEV).topk(2, 1).indices.int()
    w = torch.softmax(_randn(g, 9, 2), 1)
    for kind in ("bf16", "fp16"):
        x, _ = _rows(g, 9, 256, kind)
        clean = ep.moe_few_rows(x, None, idx, w, *layer)
        x[2, 100], x[5, 7] = float("nan"), float("inf")
        out = ep.moe_few_rows(x, None, idx, w, *layer)
        assert torch.isnan(out[2]).all() and not torch.isfinite(out[5]).any()
        keep = [0, 1, 3, 4, 6, 7, 8]
        assert torch.equal(out[keep], clean[keep])


def test_few_rows_on_a_stream_in_a_graph_and_back_to_back():
    g = _gen(8)
    layers = [_layer(g, 8, 512, 272) for _ in range(3)]
    base = _randn(g, 4, 512).to(torch.bfloat16)
    x = base.clone()
    idx = torch.rand(4, 8, generator=g, device=DEV).topk(3, 1).indices.int()
    w = torch.softmax(_randn(g, 4, 3), 1)
    norm = torch.ones(512, device=DEV)

    def passes(wait=False):
        h = x
        for i in range(6):
            q, s, _, _ = ep.rms_norm_fp8(h, norm)
            if wait:
                torch.cuda.synchronize()
            o = ep.moe_few_rows(q, s, (idx + i) % 8, w, *layers[i % 3])
            if wait:
                torch.cuda.synchronize()
            h = ep.rms_norm_join(o, h, post_weight=norm).h
        return h
    want = passes(wait=True)
    for _ in range(20):
        assert torch.equal(passes(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(passes(), want)
    torch.cuda.current_stream().wait_stream(side)
    o = ep.moe_few_rows(x, None, idx, w, *layers[0], stream=side)
    side.synchronize()
    assert torch.equal(o, ep.moe_few_rows(x, None, idx, w, *layers[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = passes()
    for _ in range(5):
        graph.replay()
    assert torch.equal(out, want)
    x.copy_(_randn(g, 4, 512).to(torch.bfloat16))
    graph.replay()
    assert torch.equal(out, passes(wait=True))


def test_two_streams_at_once():
    g = _gen(9)
    layer = _layer(g, 16, 1024, 512)
    made = []
    for rows in (1, 3, 24):
        x, xs = _rows(g, rows, 1024, "fp8")
        idx = torch.rand(rows, 16, generator=g, device=DEV).topk(4, 1).indices.int()
        w = torch.softmax(_randn(g, rows, 4), 1)
        made.append((x, xs, idx, w, ep.moe_few_rows(x, xs, idx, w, *layer)))
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    outs = [[] for _ in made]
    for _ in range(50):
        for s, m, o in zip(streams, made, outs):
            with torch.cuda.stream(s):
                o.append(ep.moe_few_rows(*m[:4], *layer))
    torch.cuda.synchronize()
    for m, o in zip(made, outs):
        assert all(torch.equal(v, m[4]) for v in o)


@pytest.mark.parametrize("rows", [1, 9, 40, 128])
def test_nothing_of_the_workspace_is_read_before_it_is_written(rows):
    lib, g = ep.load_library(), _gen(10)
    layer = _layer(g, 3, 256, 144)
    x, _ = _rows(g, rows, 256, "bf16")
    idx = torch.rand(rows, 6, generator=g, device=DEV).topk(3, 1).indices.int()
    idx[:, 0] = 1
    w = torch.rand(rows, 3, generator=g, device=DEV)
    want = ep.moe_few_rows(x, None, idx, w, *layer)
    need = lib.ep_moe_few_workspace_bytes(rows, 3, 144)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)        # not a number as FP16
    out = torch.empty_like(want)
    assert lib.ep_moe_few_rows(x.data_ptr(), None, ep.EP_BF16, idx.data_ptr(), w.data_ptr(), rows, 3, 0, 3, 256, 144,
                               *(t.data_ptr() for t in layer), ep.EP_BF16, out.data_ptr(), ws.data_ptr(), need,
                               torch.cuda.current_stream().cuda_stream) == ep.EP_OK
    assert torch.equal(out, want) and (ws[need:] == 0xFF).all()


def test_example_layer_decodes():
    """The rows are quantised once; see the bound of the example layer's other tests."""
    from combine_ep_dispatch_02_gb300 import expert_layer
    for rows in (1, 20, 128):
        assert expert_layer.main(["--tokens-per-rank", "20", "--hidden", "512", "--inner", "272", "--passes", "1",
                                  "--decode-rows", str(rows)]) <= 2.0 ** -3
