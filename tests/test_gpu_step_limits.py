"""GPU: the step's operators at the limits their headers state."""

import sys

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


def test_more_weight_rows_than_one_grid():
    # 2^23 workgroups of 80 rows and some more, at the least depth: 86 GB of weights
    n, k = 80 * (1 << 23) + 1003, 128
    w = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    marks = torch.tensor([0, 79, 80 * (1 << 22), 80 * (1 << 23) - 81, 80 * (1 << 23) - 80, 80 * (1 << 23) - 1,
                          80 * (1 << 23), n - 1], device="cuda")
    w[marks] = torch.arange(1, len(marks) + 1, device="cuda", dtype=torch.int8)[:, None]
    w_s = torch.ones(n, device="cuda")
    w_s[marks] = 0.5
    a, a_s = torch.ones(2, k, dtype=torch.int8, device="cuda"), torch.tensor([1.0, 2.0], device="cuda")
    a[1, ::2] = 0
    c = fp8bq.gemm_i8(a, a_s, w, w_s)
    want = torch.arange(1, len(marks) + 1, device="cuda") * 64.0  # 128 x 0.5, and 64 x 0.5 x 2
    assert c.shape == (2, n)
    for row in range(2):
        assert torch.equal(c[row, marks].float(), want)
        assert int((c[row] != 0).sum()) == len(marks)


def test_largest_eps():
    x, w = torch.ones(3, 256, dtype=BF16, device="cuda"), torch.ones(256, dtype=BF16, device="cuda")
    codes, scales, _ = fp8bq.rmsnorm_quant(x, w, eps=1e300)  # 1 / sqrt(eps) is 0 in fp32
    assert not codes.any() and bool((scales == 1).all())


def test_depth_zero_gives_scales_of_one(way):
    # the scale of a row without values is that of a row of zeros
    x, w = torch.empty(300, 0, dtype=BF16, device="cuda"), torch.empty(0, dtype=BF16, device="cuda")
    for call in (lambda: fp8bq.rmsnorm_quant_i8(x, w), lambda: fp8bq.rmsnorm_quant_i8(x, w, x),
                 lambda: fp8bq.quant_act_i8(x), lambda: fp8bq.quant_weight_i8(x.float())):
        used = torch.full((300,), 7.0, device="cuda")  # memory that the next tensor of this size may get
        del used
        codes, scales = call()[:2]
        assert codes.shape == (300, 0) and scales.shape == (300,) and bool((scales == 1).all())


def test_without_the_native_binding(monkeypatch):
    x, w = torch.randn(5, 256, device="cuda").to(BF16), torch.ones(256, dtype=BF16, device="cuda")
    a, s = torch.ones(4, 128, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    p, d = torch.full((2, 2, 8), 0.125, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    u = torch.full((2, 1), 0.5, device="cuda")
    calls = (lambda: fp8bq.rmsnorm_quant(x, w, x), lambda: fp8bq.rmsnorm_quant_i8(x, w),
             lambda: (fp8bq.gemm_i8(a, s, a, s),), lambda: fp8bq.verify_drafts(p, d, u, u[:, 0].contiguous()))
    want = [call() for call in calls]
    monkeypatch.setattr(step, "_direct", None)
    monkeypatch.setitem(sys.modules, "memory_bound_w8a8_amd._binding", None)
    monkeypatch.delattr(fp8bq, "_binding", raising=False)
    with pytest.warns(RuntimeWarning, match="_binding.so is missing"):
        got = [call() for call in calls]
    assert all(torch.equal(a_, b_) for one, other in zip(got, want) for a_, b_ in zip(one, other))
