"""Bounded waits of the product kernels on the GPU, without a fault.

A test-only build (EP_TEST_WITHHOLD_LOAD, short EP_WAIT_CYCLES) never loads one block of K.  Every
wait that depends on it must run out, the kernel must free its tensor memory and return, the status word
must say EP_ERR_DEVICE_TIMEOUT, and the same process must then compute correctly with the regular
library.  Each role's loops and barriers keep their counts after a wait has given up, so every wait ends
whichever of them gives up first.
"""
import os

import pytest
import torch

import combine_ep_dispatch_02_gb300 as ep
from combine_ep_dispatch_02_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def withheld_lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    build.build()
    d = str(tmp_path_factory.mktemp("withheld_load"))
    return ep.load_library(build.build(force=True, defines=["EP_TEST_WITHHOLD_LOAD=1", "EP_WAIT_CYCLES=4000000"],
                                       lib_path=os.path.join(d, "libep.so"), build_dir=d))


# one row splits K over a cluster; 300 rows take tiles of 128
@pytest.mark.parametrize("rows,columns,swiglu", [(1, 512, False), (20, 256, True), (300, 512, False), (300, 512, True)])
def test_withheld_load_reports_timeout_and_context_survives(withheld_lib, monkeypatch, rows, columns, swiglu):
    dev = torch.device("cuda", 0)
    a = torch.full((rows, 4096), 0x38, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)      # 1.0
    b = torch.full((columns, 4096), 0x38, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    sa = torch.full((rows, 32), 2.0 ** -6, device=dev)
    sb = torch.full((columns // 128, 32), 2.0 ** -6, device=dev)

    def run():
        return ep.matmul_fp8_swiglu(a, sa, b, sb) if swiglu else ep.matmul_fp8(a, sa, b, sb)
    assert ep.op_status(dev) == 0
    with monkeypatch.context() as m:
        m.setattr(ep, "_lib", withheld_lib)
        run()
        torch.cuda.synchronize()
        assert ep.op_status(dev) == ep.EP_ERR_DEVICE_TIMEOUT
        assert ep.op_status(dev) == 0                 # reading clears the word
    out = run()
    torch.cuda.synchronize()
    assert ep.op_status(dev) == 0
    if swiglu:                                        # 4096 ones times 2^-12: gate = up = 1
        z = torch.tensor(1 / (1 + torch.exp(torch.tensor(-1.0, dtype=torch.float64)).item()))
        assert (out[0].float() == 448).all() and torch.allclose(out[1] * 448, z.to(dev).expand_as(out[1]), rtol=2.0 ** -20)
    else:
        assert (out == 1).all()


# several tiles to a CTA: the roles that go on after a wait has given up stay in step over all of them
@pytest.mark.parametrize("rows,columns,groups,swiglu", [
    (16384, 1024, 0, False), (16384, 1024, 0, True), (256, 4096, 32, False), (256, 4096, 32, True)])
def test_withheld_load_with_many_tiles_returns(withheld_lib, monkeypatch, rows, columns, groups, swiglu):
    dev = torch.device("cuda", 0)
    lead = (groups,) if groups else ()
    a = torch.full((rows, 1024), 0x38, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)      # 1.0
    b = torch.full((*lead, columns, 1024), 0x38, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    sa = torch.full((rows, 8), 2.0 ** -5, device=dev)
    sb = torch.full((*lead, columns // 128, 8), 2.0 ** -5, device=dev)
    offsets = torch.arange(groups + 1, dtype=torch.int32, device=dev) * (rows // groups) if groups else None

    def run():
        call = ep.matmul_fp8_swiglu if swiglu else ep.matmul_fp8
        return call(a, sa, b, sb, offsets=offsets)
    assert ep.op_status(dev) == 0
    with monkeypatch.context() as m:
        m.setattr(ep, "_lib", withheld_lib)
        for _ in range(3):
            run()
        assert ep.op_status(dev) == ep.EP_ERR_DEVICE_TIMEOUT
    out = run()
    assert ep.op_status(dev) == 0
    if swiglu:                                        # 1024 ones times 2^-10: gate = up = 1
        assert (out[0].float() == 448).all()
    else:
        assert (out == 1).all()
