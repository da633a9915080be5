"""Bounded waits of the weight gradient's kernel on the GPU, without a fault: as test_experts_failure_gpu.py, a test-only
build never loads one stage, every wait that depends on it runs out, and the process goes on."""
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
    d = str(tmp_path_factory.mktemp("withheld_stage"))
    return ep.load_library(build.build(force=True, defines=["EP_TEST_WITHHOLD_LOAD=1", "EP_WAIT_CYCLES=4000000"],
                                       lib_path=os.path.join(d, "libep.so"), build_dir=d))


# one tile; several to a pair of CTAs, by group
@pytest.mark.parametrize("rows,columns,inner,groups", [(300, 256, 256, 0), (4096, 2048, 4096, 8)])
def test_withheld_stage_reports_timeout_and_context_survives(withheld_lib, monkeypatch, rows, columns, inner, groups):
    dev = torch.device("cuda", 0)
    dy = torch.ones(rows, columns, dtype=torch.bfloat16, device=dev)
    a = torch.full((rows, inner), 0x38, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)      # 1.0
    s = torch.full((rows, inner // 128), 0.5, device=dev)
    offsets = torch.arange(groups + 1, dtype=torch.int32, device=dev) * (rows // groups) if groups else None

    def run():
        return ep.matmul_fp8_weight_gradient(dy, a, s, offsets=offsets, out_dtype="fp32")
    assert ep.op_status(dev) == 0
    with monkeypatch.context() as m:
        m.setattr(ep, "_lib", withheld_lib)
        for _ in range(3):
            run()
        assert ep.op_status(dev) == ep.EP_ERR_DEVICE_TIMEOUT
        assert ep.op_status(dev) == 0
    out = run()
    assert ep.op_status(dev) == 0
    assert (out == 0.5 * (rows // groups if groups else rows)).all()
