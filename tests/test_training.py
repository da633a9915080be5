"""Refusals of the training operators and of the layer for a few rows that need no GPU: the C ABI rejects what the host can
check before any CUDA call, and the binding rejects tensors of the wrong kind."""
import ctypes
import os

import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from combine_ep_dispatch_02_gb300 import build as epbuild
from test_experts import P, _refused, lib  # noqa: F401

JOIN = dict(y=P, y_stride=256, post_weight=P, gate=None, gate_stride=0, pre_weight=P, rows=4, hidden=256, dtype=ep.EP_BF16,
            post_fp32=0, pre_fp32=0, gate_kind=0, gate_fp32=0, residual_scale=1.0, eps=1e-6)
FWD = dict(residual=P, rs=256, h=P, n=P, q=None, s=None, post=P, pre=P, stream=None)
BWD = dict(h=P, post=P, pre=P, dh=P, dhs=256, dn=P, dns=256, dy=P, dres=P, dpost=P, dgate=None, dpre=P, ws=P, wsb=1 << 40,
           stream=None)
SAVE = dict(x=P, stride=512, dtype=ep.EP_BF16, rows=4, inner=256, end=None, q=P, s=P, saved=P, ss=P, stream=None)
BACK = dict(saved=P, ss=P, dz=P, stride=256, dtype=ep.EP_BF16, rows=4, inner=256, end=None, d=P, q=None, s=None, stream=None)

GRAD = dict(dy=P, dtype=ep.EP_BF16, a=P, s=P, offsets=None, rows=64, groups=1, columns=128, inner=256, fp32=0, dw=P, status=P,
            stream=None)
FEW = dict(x=P, xs=P, xd=ep.EP_FP8_E4M3, idx=P, w=P, rows=4, k=2, first=0, experts=8, hidden=256, inner=128, up=P, ups=P, down=P,
           downs=P, od=ep.EP_BF16, out=P, ws=P, wsb=1 << 40, stream=None)


def _join(lib, change, call, rest):
    j = ep.JoinArgs(**{**JOIN, **{k: v for k, v in change.items() if k in JOIN}})
    return call(ctypes.byref(j), *{**rest, **{k: v for k, v in change.items() if k not in JOIN}}.values())


SHARED = [(dict(dtype=2), "dtype"), (dict(hidden=0), "hidden"), (dict(hidden=24), "hidden"), (dict(hidden=32784), "hidden"),
          (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
          (dict(gate_kind=4), "gate_kind"), (dict(gate_kind=-1), "gate_kind"), (dict(post_weight=P + 4), "weight"),
          (dict(pre_weight=P + 8), "weight"), (dict(y=None), "y is"), (dict(y=P + 8), "y is"), (dict(y_stride=248), "stride"),
          (dict(y_stride=260), "stride"), (dict(gate_kind=1), "gate"), (dict(gate_kind=1, gate=P + 2), "gate"),
          (dict(gate_kind=2, gate=P + 8), "gate"), (dict(gate_kind=3, gate=P, gate_stride=128), "gate")]


@pytest.mark.parametrize("change,word", SHARED + [
    (dict(residual=None), "residual"), (dict(rs=252), "residual"), (dict(h=None), "h is"), (dict(n=P + 2), "n is"),
    (dict(q=P), "q and scales"), (dict(q=P + 8, s=P), "q and scales"), (dict(pre_weight=None), "pre_weight"),
    (dict(post=None), "rstd"), (dict(pre=P + 1), "rstd")])
def test_join_refusals(lib, change, word):  # noqa: F811
    _refused(lib, _join(lib, change, lib.ep_rms_norm_join, FWD), "ep_rms_norm_join", word)


@pytest.mark.parametrize("change,word", SHARED + [
    (dict(hidden=8208), "hidden"), (dict(dn=None), "dn and pre_weight"), (dict(pre_weight=None), "dn and pre_weight"),
    (dict(dn=None, dh=None, pre_weight=None), "neither"), (dict(dpost=None), "gradient"), (dict(dpre=P + 2), "gradient"),
    (dict(gate_kind=2, gate=P), "gradient"), (dict(dhs=200), "dh or dn"), (dict(dn=P + 4), "dh or dn"), (dict(h=None), "h, dy"),
    (dict(dy=None), "h, dy"), (dict(dres=P + 2), "h, dy"), (dict(gate_kind=1, gate=P), "dgate"),
    (dict(gate_kind=3, gate=P, gate_stride=256, dgate=P + 8), "dgate"), (dict(post=None), "rstd"), (dict(pre=P + 2), "rstd")])
def test_join_backward_refusals(lib, change, word):  # noqa: F811
    _refused(lib, _join(lib, change, lib.ep_rms_norm_join_backward, BWD), "ep_rms_norm_join_backward", word)


def test_join_takes_its_arguments(lib):  # noqa: F811
    _refused(lib, lib.ep_rms_norm_join(None, *FWD.values()), "join is NULL")
    _refused(lib, lib.ep_rms_norm_join_backward(None, *BWD.values()), "join is NULL")
    assert _join(lib, dict(rows=0, y=None), lib.ep_rms_norm_join, {**FWD, "residual": None}) == ep.EP_OK
    for rows, hidden in ((0, 256), (-1, 256), (1 << 31, 256), (4, 8), (4, 24), (4, 8208)):
        assert lib.ep_rms_norm_join_workspace_bytes(rows, hidden) == 0


GLU = [(dict(dtype=2), "dtype"), (dict(inner=0), "inner"), (dict(inner=24), "inner"), (dict(inner=(1 << 20) + 16), "inner"),
       (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(rows=1 << 29), "rows"), (dict(rows=1 << 62), "rows"),
       (dict(end=P + 2), "rows_end"), (dict(stride=248), "stride"), (dict(stride=516), "stride")]


@pytest.mark.parametrize("change,word", GLU + [
    (dict(x=None), "gate_up"), (dict(x=P + 8), "gate_up"), (dict(q=None), "q, saved"), (dict(saved=P + 8), "q, saved"),
    (dict(s=P + 2), "scale"), (dict(ss=None), "scale")])
def test_swiglu_refusals(lib, change, word):  # noqa: F811
    _refused(lib, lib.ep_swiglu_saved(*{**SAVE, **change}.values()), "ep_swiglu_saved", word)


@pytest.mark.parametrize("change,word", GLU + [
    (dict(dz=None), "dz"), (dict(dz=P + 4), "dz"), (dict(saved=None), "saved"), (dict(ss=P + 2), "saved_scales"),
    (dict(d=P + 8), "d_gate_up"), (dict(q=P), "q and scales"), (dict(s=P), "q and scales"), (dict(q=P + 8, s=P), "q and scales")])
def test_swiglu_backward_refusals(lib, change, word):  # noqa: F811
    _refused(lib, lib.ep_swiglu_saved_backward(*{**BACK, **change}.values()), "ep_swiglu_saved_backward", word)


@pytest.mark.parametrize("change,word", [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 31) - 64), "rows"), (dict(groups=0), "groups"), (dict(groups=2), "groups"),
    (dict(groups=4097, offsets=P), "groups"), (dict(inner=0), "inner"), (dict(inner=24), "inner"),
    (dict(inner=(1 << 20) + 16), "inner"), (dict(columns=0), "columns"), (dict(columns=12), "columns"),
    (dict(columns=(1 << 20) + 8), "columns"), (dict(dtype=2), "dtype"), (dict(status=None), "device_status"),
    (dict(dw=None), "dw"), (dict(dw=P + 8), "dw"), (dict(offsets=P + 2), "offsets"), (dict(dy=P + 8), "dy, a"),
    (dict(a=None), "dy, a"), (dict(s=P + 2), "a_scales")])
def test_weight_gradient_refusals(lib, change, word):  # noqa: F811
    _refused(lib, lib.ep_matmul_fp8_weight_gradient(*{**GRAD, **change}.values()), "ep_matmul_fp8_weight_gradient", word)


@pytest.mark.parametrize("change,word", [
    (dict(rows=-1), "rows"), (dict(rows=129), "rows"), (dict(k=0), "topk"), (dict(rows=128, k=33), "topk"),
    (dict(k=2 ** 31 - 1), "topk"), (dict(experts=0), "experts"), (dict(experts=1025), "experts"), (dict(hidden=0), "hidden"),
    (dict(hidden=24), "hidden"), (dict(hidden=(1 << 20) + 16), "hidden"), (dict(inner=0), "inner"), (dict(inner=40), "inner"),
    (dict(inner=(1 << 19) + 16), "inner"), (dict(xd=3), "x_dtype"), (dict(od=2), "out_dtype"), (dict(x=None), "x is"),
    (dict(x=P + 8), "x is"), (dict(xs=None), "x_scales"), (dict(xd=0), "x_scales"), (dict(xs=P + 2), "x_scales"),
    (dict(idx=None), "indices"), (dict(w=P + 2), "weights"), (dict(up=P + 8), "up, down"), (dict(down=None), "up, down"),
    (dict(ups=P + 1), "scale"), (dict(downs=None), "scale"), (dict(out=P + 8), "out"), (dict(ws=None), "workspace"),
    (dict(wsb=100), "workspace")])
def test_few_rows_refusals(lib, change, word):  # noqa: F811
    _refused(lib, lib.ep_moe_few_rows(*{**FEW, **change}.values()), "ep_moe_few_rows", word)


def test_few_rows_workspace(lib):  # noqa: F811
    assert lib.ep_moe_few_workspace_bytes(1, 8, 2048) == 8 * 2048 * 2 + 8 * 256
    assert lib.ep_moe_few_workspace_bytes(3, 1, 16) == 256 + 3 * 2      # 96 bytes of z, rounded up
    for bad in ((0, 8, 16), (129, 1, 16), (128, 33, 16), (1, 0, 16), (1, 1, 24), (1, 1, 0)):
        assert lib.ep_moe_few_workspace_bytes(*bad) == 0
    assert lib.ep_moe_few_rows(*{**FEW, "rows": 0, "x": None, "ws": None}.values()) == ep.EP_OK


def test_empty_calls_succeed_without_a_gpu(lib):  # noqa: F811
    assert lib.ep_swiglu_saved(*{**SAVE, "rows": 0, "x": None, "q": None}.values()) == ep.EP_OK
    assert lib.ep_swiglu_saved_backward(*{**BACK, "rows": 0, "dz": None, "saved": None}.values()) == ep.EP_OK


def test_binding_takes_cuda_tensors_only(lib):  # noqa: F811
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for call in (lambda: ep.rms_norm_join(x, x), lambda: ep.rms_norm_join_backward(ep.Joined(x), x, dh=x),
                 lambda: ep.swiglu_saved(x), lambda: ep.swiglu_saved_backward(x, x, x),
                 lambda: ep.moe_few_rows(x, None, x, x, x, x, x, x), lambda: ep.matmul_fp8_weight_gradient(x, x, x)):
        with pytest.raises(ep.EpError) as e:
            call()
        assert e.value.code == ep.EP_ERR_ARG and "not a CUDA device" in str(e.value)
    with pytest.raises(ep.EpError, match="y is a list, not a tensor"):
        ep.rms_norm_join([1.0], x)


def test_out_types_are_named(lib):  # noqa: F811
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ep.EpError, match="out_dtype"):
        ep.matmul_fp8_weight_gradient(x, x, x, out_dtype="fp64")
    with pytest.raises(ep.EpError, match="out_dtype"):
        ep.moe_few_rows(x, None, x, x, x, x, x, x, out_dtype="fp32")


@pytest.mark.parametrize("name,kernels", [("ep_join.cu", 4), ("ep_swiglu.cu", 2), ("ep_wgrad.cu", 1)])
def test_kernels_read_no_memory_before_their_own_wait(name, kernels):
    """As in test_experts.py: before follow_predecessor() no kernel names an array of its arguments."""
    import re
    with open(os.path.join(epbuild.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    arrays = set()
    for struct in re.findall(r"struct \w+Args \{(.*?)\n\};", text, flags=re.S):
        for line in re.findall(r"[^;]*\*[^;]*;", struct):
            arrays |= set(re.findall(r"\*?\s*(\w+)(?:\[\d+\])?\s*[,;]", line))
    assert arrays
    bodies = re.findall(r"__global__ [^;{]*\{(.*?)\n\}", text, flags=re.S)
    assert len(bodies) == kernels
    for body in bodies:
        before, wait, _ = body.partition("follow_predecessor();")
        assert wait
        assert not set(re.findall(r"\b[ap]\.(\w+)", before)) & (arrays - {"status"}), (name, before[-300:])
