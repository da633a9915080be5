"""Refusals of the expert-layer operators that need no GPU: the C ABI rejects what the host can check
before any CUDA call, and the binding rejects tensors of the wrong kind."""
import ctypes
import os
import re

import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from combine_ep_dispatch_02_gb300 import build as epbuild

P = 1 << 20          # an aligned address that no rejected call dereferences


@pytest.fixture(scope="module")
def lib():
    epbuild.build()
    return ep.load_library()


def _refused(lib, rc, *words):
    assert rc == ep.EP_ERR_ARG
    msg = lib.ep_last_error().decode()
    for w in words:
        assert w in msg, msg


NORM = dict(x=P, xs=256, r=None, rs=0, w=P, w32=0, dtype=ep.EP_BF16, rows=4, hidden=256, eps=1e-6, q=P, s=P, h=None,
            y=None, stream=None)
SORT = dict(idx=P, counts=None, W=1, R=8, k=2, E=4, max_rows=16, offsets=P, pos=P, src=P, ws=None, wsb=0, status=P,
            stream=None)
ROWS = dict(x=P, scales=None, pos=P, counts=None, W=1, R=8, k=2, max_rows=16, row_bytes=32, sd=0, out=P, os=None,
            status=P, stream=None)
RET = dict(y=P, w=P, pos=P, counts=None, W=1, R=8, k=2, max_rows=16, hidden=16, dtype=ep.EP_BF16, out=P, status=P,
           stream=None)
BACK = dict(y=P, w=P, dout=P, pos=P, counts=None, W=1, R=8, k=2, max_rows=16, hidden=16, dtype=ep.EP_BF16, dy=P, dw=P,
            status=P, stream=None)
MUL = dict(a=P, sa=P, b=P, sb=P, offsets=None, rows=4, groups=1, columns=64, inner=128, swiglu=0, dtype=ep.EP_BF16,
           out=P, os=None, status=P, stream=None)


@pytest.mark.parametrize("change,word", [
    (dict(dtype=2), "dtype"), (dict(hidden=0), "hidden"), (dict(hidden=24), "hidden"), (dict(hidden=32784), "hidden"),
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(x=None), "x is"), (dict(x=P + 8), "x is"), (dict(xs=248), "stride"), (dict(xs=260), "stride"),
    (dict(r=P + 2, rs=256), "residual"), (dict(r=P, rs=128), "residual"), (dict(w=None), "weight"),
    (dict(w=P + 4), "weight"), (dict(q=None), "q or scales"), (dict(s=P + 2), "q or scales"), (dict(h=P + 8), "h or y"),
    (dict(y=P + 8), "h or y")])
def test_norm_refusals(lib, change, word):
    _refused(lib, lib.ep_rms_norm_fp8(*{**NORM, **change}.values()), "ep_rms_norm_fp8", word)


COMMON = [(dict(W=0), "W="), (dict(W=33), "W="), (dict(k=0), "topk"), (dict(k=65), "topk"), (dict(R=-1), "rows_per_rank"),
          (dict(R=1 << 30), "rows_per_rank"), (dict(max_rows=-1), "max_rows"), (dict(max_rows=1 << 31), "max_rows"),
          (dict(counts=P + 2), "counts"), (dict(status=None), "device_status"), (dict(pos=None), "pos"),
          (dict(pos=P + 1), "pos")]


@pytest.mark.parametrize("change,word", COMMON + [
    (dict(E=0), "experts_per_rank"), (dict(E=4097), "experts_per_rank"), (dict(W=2, E=2049), "experts_per_rank"),
    (dict(offsets=None), "offsets"), (dict(idx=None), "indices"), (dict(src=None), "src"),
    (dict(R=100000), "workspace"), (dict(R=100000, ws=P, wsb=100), "workspace")])
def test_sort_refusals(lib, change, word):
    _refused(lib, lib.ep_sort_by_expert(*{**SORT, **change}.values()), "ep_sort_by_expert", word)


def test_sort_workspace_sizes(lib):
    assert lib.ep_sort_workspace_bytes(1, 256, 8, 256) == 0             # one CTA sorts 2048 pairs
    assert lib.ep_sort_workspace_bytes(1, 257, 8, 256) == 2 * 256 * 4   # tiles of 2048 pairs
    assert lib.ep_sort_workspace_bytes(1, 16384, 8, 64) == 64 * 64 * 4  # 131072 pairs: the last such size
    assert lib.ep_sort_workspace_bytes(1, 16385, 8, 64) == 17 * 64 * 4  # tiles of 8192 pairs
    assert lib.ep_sort_workspace_bytes(8, 32768, 8, 32) == 256 * 256 * 4
    assert lib.ep_sort_workspace_bytes(1, 10, 8, 2049) == 2049 * 4      # many groups: the tiled form
    for bad in ((0, 8, 8, 8), (1, -1, 8, 8), (1, 8, 65, 8), (1, 8, 8, 4097), (1, 1 << 31, 1, 1), (32, 1 << 26, 1, 1)):
        assert lib.ep_sort_workspace_bytes(*bad) == 0


def test_sort_of_no_rows_with_many_groups_takes_one_tile(lib):
    assert lib.ep_sort_workspace_bytes(1, 0, 8, 2048) == 0
    assert lib.ep_sort_workspace_bytes(1, 0, 8, 2049) == 2049 * 4
    assert lib.ep_sort_workspace_bytes(2, 0, 4, 1500) == 3000 * 4


@pytest.mark.parametrize("change,word", COMMON + [
    (dict(row_bytes=0), "row of"), (dict(row_bytes=24), "row of"), (dict(row_bytes=1 << 31), "row of"),
    (dict(sd=-1), "scale_dim"), (dict(sd=65537), "scale_dim"), (dict(sd=3), "scales"), (dict(x=P + 8), "x, out"),
    (dict(out=None), "x, out"), (dict(R=1 << 28, k=1, row_bytes=1 << 20), "CTAs")])
def test_sorted_rows_refusals(lib, change, word):
    _refused(lib, lib.ep_sorted_rows(*{**ROWS, **change}.values()), "ep_sorted_rows", word)


@pytest.mark.parametrize("change,word", COMMON + [
    (dict(hidden=0), "hidden"), (dict(hidden=12), "hidden"), (dict(dtype=2), "dtype"), (dict(y=None), "y, out"),
    (dict(out=P + 4), "y, out"), (dict(w=P + 2), "weights")])
def test_return_rows_refusals(lib, change, word):
    _refused(lib, lib.ep_return_rows(*{**RET, **change}.values()), "ep_return_rows", word)


@pytest.mark.parametrize("change,word", COMMON + [
    (dict(hidden=20), "hidden"), (dict(dtype=3), "dtype"), (dict(y=P + 8), "y, dout"), (dict(dout=None), "y, dout"),
    (dict(dy=None), "y, dout"), (dict(w=None), "weights"), (dict(dw=None), "weights or dweights")])
def test_return_rows_backward_refusals(lib, change, word):
    _refused(lib, lib.ep_return_rows_backward(*{**BACK, **change}.values()), "ep_return_rows_backward", word)


@pytest.mark.parametrize("change,word", [
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(groups=0), "groups"), (dict(groups=2), "groups"),
    (dict(groups=4097, offsets=P), "groups"), (dict(inner=0), "inner"), (dict(inner=120), "inner"),
    (dict(inner=(1 << 20) + 16), "inner"), (dict(columns=0), "columns"), (dict(columns=(1 << 20) + 1), "columns"),
    (dict(columns=48, swiglu=1, dtype=ep.EP_FP8_E4M3, os=P), "columns"), (dict(groups=4096, columns=1 << 20, offsets=P), "columns"),
    (dict(dtype=ep.EP_FP8_E4M3), "dtype"), (dict(swiglu=1), "dtype"), (dict(status=None), "device_status"),
    (dict(a=None), "a, b"), (dict(b=P + 8), "a, b"), (dict(sa=P + 2), "scale"), (dict(out=P + 8), "out"),
    (dict(swiglu=1, dtype=ep.EP_FP8_E4M3), "out_scales"), (dict(offsets=P + 2), "offsets")])
def test_product_refusals(lib, change, word):
    _refused(lib, lib.ep_matmul_fp8(*{**MUL, **change}.values()), "ep_matmul_fp8", word)


def test_product_rows_stay_in_32_bits_to_the_end_of_the_last_tile(lib):
    _refused(lib, lib.ep_matmul_fp8(*{**MUL, "rows": (1 << 31) - 128}.values()), "ep_matmul_fp8", "rows")


def test_empty_calls_succeed_without_a_gpu(lib):
    assert lib.ep_rms_norm_fp8(*{**NORM, "rows": 0, "x": None, "q": None}.values()) == ep.EP_OK
    assert lib.ep_sorted_rows(*{**ROWS, "R": 0, "x": None}.values()) == ep.EP_OK
    assert lib.ep_sorted_rows(*{**ROWS, "max_rows": 0, "out": None}.values()) == ep.EP_OK
    assert lib.ep_return_rows(*{**RET, "R": 0}.values()) == ep.EP_OK
    assert lib.ep_return_rows_backward(*{**BACK, "R": 0}.values()) == ep.EP_OK
    assert lib.ep_matmul_fp8(*{**MUL, "rows": 0, "a": None, "out": None}.values()) == ep.EP_OK


def test_live_check_refuses_a_null_plan(lib):
    assert lib.ep_check_live(None, 0) == ep.EP_ERR_ARG


def test_binding_takes_cuda_tensors_only(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    f8 = torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    order = ep.ExpertOrder(i, i, i[:, 0])
    for call in (lambda: ep.rms_norm_fp8(x, x[0]), lambda: ep.sort_by_expert(i, 4), lambda: ep.sorted_rows(order, x),
                 lambda: ep.return_rows(order, x), lambda: ep.return_rows_backward(order, x, x, x),
                 lambda: ep.matmul_fp8(f8, x, f8, x), lambda: ep.matmul_fp8_swiglu(f8, x, f8, x)):
        with pytest.raises(ep.EpError) as e:
            call()
        assert e.value.code == ep.EP_ERR_ARG and "not a CUDA device" in str(e.value)
    with pytest.raises(ep.EpError, match="x is a list, not a tensor"):
        ep.rms_norm_fp8([1.0], x[0])
    with pytest.raises(ep.EpError, match="out_dtype"):
        ep.matmul_fp8(f8, x, f8, x, out_dtype="fp32")


def test_take_status_refusals(lib):
    for args in ((None, P, None), (P, None, None), (P + 2, P, None), (P, P + 1, None)):
        _refused(lib, lib.ep_take_status(*args), "ep_take_status", "4-byte aligned")


def test_status_codes_have_messages(lib):
    assert ctypes.c_char_p(lib.ep_strerror(ep.EP_ERR_CAPACITY)).value


@pytest.mark.parametrize("name,kernels", [("ep_norm.cu", 1), ("ep_sort.cu", 8), ("ep_matmul.cu", 2)])
def test_kernels_read_no_memory_before_their_own_wait(name, kernels):
    """Launched as programmatic dependents, they may run before what they read is visible to them: before
    follow_predecessor() none names an array of its arguments or calls a function that reads one."""
    with open(os.path.join(epbuild.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    arrays = set()
    for struct in re.findall(r"struct \w+Args \{(.*?)\n\};", text, flags=re.S):
        for line in re.findall(r"[^;]*\*[^;]*;", struct):
            arrays |= set(re.findall(r"\*?\s*(\w+)\s*[,;]", line))
    arrays -= {"status"}                                      # handed on as an address
    assert {"x", "weight"} <= arrays or {"idx", "tile_counts", "pos"} <= arrays or {"a", "bs", "offsets"} <= arrays
    readers = set(re.findall(r"__device__ __forceinline__ \w+ (\w+)\(const \w+Args& ", text))
    bodies = re.findall(r"__global__ [^;{]*\{(.*?)\n\}", text, flags=re.S)
    assert len(bodies) == kernels
    for body in bodies:
        before, wait, _ = body.partition("follow_predecessor();")
        assert wait
        used = set(re.findall(r"\b[ap]\.(\w+)", before)) & arrays | set(re.findall(r"\b(\w+)(?:<[^;()]*>)?\(", before)) & readers
        assert not used, (name, used, before[-300:])


def test_binding_is_built_again_for_another_pytorch(lib, monkeypatch):
    """Its binary holds PyTorch's C++ layout, so its sources' times alone do not tell whether it still fits."""
    built = []
    monkeypatch.setattr(epbuild, "build_binding", lambda: built.append(1))
    monkeypatch.setattr(epbuild.subprocess, "run", lambda *a, **k: epbuild.subprocess.CompletedProcess(a, 0, "", ""))
    monkeypatch.setattr(epbuild.os, "replace", lambda *a: None)
    epbuild.build()
    assert not built
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    epbuild.build()
    assert built
