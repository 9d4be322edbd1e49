"""GPU: the step's operators at the limits their headers state."""

import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from memory_bound_w8a8_amd import step

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class _Absent:
    """_binding with every call left to Python."""

    @staticmethod
    def rmsnorm(*args):
        return None

    gemm_i8 = verify_drafts = rmsnorm


@pytest.fixture(params=["direct", "python"])
def way(request, monkeypatch):
    fp8bq.rmsnorm_quant(torch.ones(1, 128, dtype=BF16, device="cuda"), torch.ones(128, dtype=BF16, device="cuda"))
    if request.param == "python":
        monkeypatch.setattr(step, "_direct", _Absent())
    return request.param


def test_residual_output_is_ignored_without_a_residual():
    # at the C entry: an H that is given, and not even aligned, is neither read nor written
    x, w = torch.randn(5, 256, device="cuda").to(BF16), torch.ones(256, dtype=BF16, device="cuda")
    want = fp8bq.rmsnorm_quant(x, w)
    h = torch.full((5 * 256 + 1,), 3.0, dtype=BF16, device="cuda")
    codes, scales = torch.empty(5, 256, dtype=torch.uint8, device="cuda"), torch.empty(5, 2, device="cuda")
    st = step.step_lib().fp8bq_rmsnorm_quant(5, 256, x.data_ptr(), None, w.data_ptr(), 1e-6, h[1:].data_ptr(),
                                             codes.data_ptr(), scales.data_ptr(),
                                             torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and bool((h == 3).all())


def test_output_too_large_to_allocate(way):
    # 2^20 x 2^20 results: 2 TiB
    a, s = torch.ones(1 << 20, 128, dtype=torch.int8, device="cuda"), torch.ones(1 << 20, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        fp8bq.gemm_i8(a, s, a, s)
