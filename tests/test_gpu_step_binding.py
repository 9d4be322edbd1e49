"""GPU: the two ways from Python to the step's operators, the direct one
(_binding.so) and the one that names what is wrong, take the same calls and
give the same bits."""

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from helpers import to_gpu
from memory_bound_w8a8_amd import step

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class _Absent:
    """_binding with every call left to Python."""

    @staticmethod
    def rmsnorm(*args):
        return None

    gemm_i8 = verify_drafts = rmsnorm


class _Only:
    """_binding, whose calls must all be taken."""

    def __getattr__(self, name):
        from memory_bound_w8a8_amd import _binding

        def call(*args):
            out = getattr(_binding, name)(*args)
            assert out is not None, f"{name}: left to Python"
            return out

        return call


def _calls():
    rng = np.random.default_rng(0)

    def bf16(*shape):
        return to_gpu(rng.standard_normal(shape).astype(np.float32), BF16)

    def codes(*shape):
        return to_gpu(rng.integers(-128, 128, shape, dtype=np.int8))

    def probs(*shape):
        return torch.softmax(2 * to_gpu(rng.standard_normal(shape).astype(np.float32)), -1)

    def rand(*shape):
        return to_gpu(rng.random(shape).astype(np.float32))

    x, r, w = bf16(7, 640), bf16(7, 640), bf16(640)
    a, b = (codes(70, 2048), rand(70), codes(130, 2048), rand(130)), (codes(9, 256), rand(9), codes(33, 256), rand(33))
    t, q = probs(5, 4, 700), probs(5, 3, 700)
    d = to_gpu(rng.integers(0, 700, (5, 3)).astype(np.int32))
    lens = to_gpu(np.array([0, 1, 2, 3, 3], np.int32))
    space = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    none = torch.empty(5, 0, device="cuda")
    return [
        lambda: fp8bq.rmsnorm_quant(x, w),
        lambda: fp8bq.rmsnorm_quant(x, w, r, 1e-5),
        lambda: fp8bq.rmsnorm_quant(x, w, r, 1, torch.empty_like(x)),
        lambda: fp8bq.rmsnorm_quant_i8(x, torch.nn.Parameter(w), r),
        lambda: fp8bq.rmsnorm_quant_i8(x[:0], w, r[:0]),
        lambda: (fp8bq.gemm_i8(*a),),
        lambda: (fp8bq.gemm_i8(*a, workspace=space),),
        lambda: (fp8bq.gemm_i8(*b, out=torch.empty(9, 33, dtype=BF16, device="cuda")),),
        lambda: fp8bq.verify_drafts(t, d, rand(5, 3) * 0 + 0.5, rand(5) * 0 + 0.3, q),
        lambda: fp8bq.verify_drafts(t, d, rand(5, 3) * 0 + 0.5, rand(5) * 0 + 0.3, q, lens, space),
        lambda: fp8bq.verify_drafts(t.to(BF16), d, rand(5, 3) * 0 + 0.5, rand(5) * 0 + 0.3),
        lambda: fp8bq.verify_drafts(t[:, :1].contiguous(), none.int(), none, rand(5) * 0 + 0.3),
    ]


def test_both_ways_give_the_same(monkeypatch):
    for i, call in enumerate(_calls()):
        monkeypatch.setattr(step, "_direct", _Only())
        direct = call()
        monkeypatch.setattr(step, "_direct", _Absent())
        python = call()
        assert len(direct) == len(python)
        for u, v in zip(direct, python):
            assert u.dtype == v.dtype and u.shape == v.shape, i
            assert torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)), i
            assert not u.requires_grad


def test_outputs_are_the_tensors_given():
    x, r = torch.ones(2, 128, dtype=BF16, device="cuda"), torch.ones(2, 128, dtype=BF16, device="cuda")
    w = torch.ones(128, dtype=BF16, device="cuda")
    assert fp8bq.rmsnorm_quant(x, w)[2] is x
    assert fp8bq.rmsnorm_quant(x, w, r, out_residual=r)[2] is r
    out = torch.empty(3, 4, dtype=BF16, device="cuda")
    a, s = torch.ones(4, 128, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    assert fp8bq.gemm_i8(a[:3], s[:3], a, s, out=out) is out


def test_what_is_left_to_python():
    from memory_bound_w8a8_amd import _binding

    at = torch.cuda.current_device()
    stream = torch.cuda.current_stream().cuda_stream
    x, w = torch.ones(2, 128, dtype=BF16, device="cuda"), torch.ones(128, dtype=BF16, device="cuda")
    ok = [x, w, x, 1e-6, None, False, at, stream]
    assert isinstance(_binding.rmsnorm(*ok), tuple)
    for i, bad in ((0, x.float()), (0, x.cpu()), (0, None), (0, x.t()), (0, x[0]), (1, w[:64]), (1, w[::2]), (2, x[:1]),
                   (2, "r"), (3, 1), (4, w), (6, at + 1)):
        args = list(ok)
        args[i] = bad
        assert _binding.rmsnorm(*args) is None, i
    args = list(ok)
    args[2], args[4] = None, x  # an output for a residual that is not there
    assert _binding.rmsnorm(*args) is None
    y = torch.ones(2, 100, dtype=BF16, device="cuda")
    assert _binding.rmsnorm(y, y[0], None, 1e-6, None, True, at, stream) == -2  # a status, as the library gives it
    with pytest.raises(TypeError):
        _binding.rmsnorm(*ok[:-1])


def test_other_stream():
    x, r = torch.randn(64, 5120, device="cuda").to(BF16), torch.randn(64, 5120, device="cuda").to(BF16)
    w = torch.ones(5120, dtype=BF16, device="cuda")
    want = fp8bq.rmsnorm_quant(x, w, r)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(10_000_000)
        late = (x * 1.0, r * 1.0)  # only there once the stream gets to them
        got = fp8bq.rmsnorm_quant(late[0], w, late[1])
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
