"""include/fp8bq_step.h: the library exports what it declares and its calls
refuse bad arguments on the host, before any device is touched (CPU only)."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8bq_step.h")
P = 1 << 20  # an aligned, never-dereferenced address
NULL, SHAPE, ALIGN, DEVICE, VALUE = -1, -2, -3, -4, -7


@pytest.fixture(scope="module")
def L():
    import memory_bound_w8a8_amd as m

    if not os.path.exists(m.LIB_PATH):
        from memory_bound_w8a8_amd import build

        build.build()
    from memory_bound_w8a8_amd import step

    return step.step_lib()


def test_exports(L):
    from memory_bound_w8a8_amd import LIB_PATH, STEP_EXPORTS

    text = open(HEADER).read()
    declared = set(re.findall(r"^\s*(?:int|int64_t)\s+(fp8bq_\w+)\s*\(", text, flags=re.M))
    assert declared == set(STEP_EXPORTS)
    raw = ctypes.CDLL(LIB_PATH)
    assert all(hasattr(raw, name) for name in declared)


def test_constants_match_the_header():
    from memory_bound_w8a8_amd import step

    text = open(HEADER).read()
    for name, value in (("FP8BQ_NORM_MAX_K", step.NORM_MAX_K), ("FP8BQ_GEMM_I8_MAX_K", step.GEMM_I8_MAX_K),
                        ("FP8BQ_MAX_DRAFTS", step.MAX_DRAFTS)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value
    assert 128 * 128 * step.GEMM_I8_MAX_K < 2 ** 31


def test_value_status_has_a_string(L):
    assert L.fp8bq_status_string(VALUE).decode() not in ("", "unknown status")


@pytest.mark.parametrize("name", ["fp8bq_rmsnorm_quant", "fp8bq_rmsnorm_quant_i8"])
def test_rmsnorm_refusals(L, name):
    f = getattr(L, name)

    def call(m=1, k=128, x=P, r=P, w=P, eps=1e-6, h=P, c=P, s=P):
        return f(m, k, x, r, w, eps, h, c, s, None)

    for bad in (dict(m=-1), dict(k=-128), dict(k=100), dict(k=65536 + 128), dict(m=1 << 31), dict(m=(1 << 30), k=65536)):
        assert call(**bad) == SHAPE, bad
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == VALUE
    assert call(m=0, x=None, w=None, h=None, c=None, s=None) == 0
    assert call(k=0, x=None, w=None, h=None, c=None, s=None) == 0
    for bad in (dict(x=None), dict(w=None), dict(c=None), dict(s=None), dict(h=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=P + 2), dict(r=P + 8), dict(w=P + 2), dict(h=P + 8), dict(c=P + 8), dict(s=P + 2)):
        assert call(**bad) == ALIGN, bad
    assert call(r=None, h=P + 2) in (DEVICE, 0, -5)  # h is ignored without a residual


@pytest.mark.parametrize("name", ["fp8bq_quant_act_i8", "fp8bq_quant_weight_i8"])
def test_quant_i8_refusals(L, name):
    f = getattr(L, name)
    assert f(-1, 128, P, P, P, None) == SHAPE
    assert f(1, 130, P, P, P, None) == SHAPE
    assert f(1, 65536 + 128, P, P, P, None) == SHAPE
    assert f(1 << 31, 128, P, P, P, None) == SHAPE
    assert f(0, 128, None, None, None, None) == 0
    assert f(1, 0, None, None, None, None) == 0
    for i in range(3):
        args = [P, P, P]
        args[i] = None
        assert f(1, 128, *args, None) == NULL
        args[i] = P + 2
        assert f(1, 128, *args, None) == ALIGN


def test_gemm_i8_refusals(L):
    def call(m=1, n=4, k=128, a=P, sa=P, w=P, sw=P, c=P, ws=None, nbytes=0):
        return L.fp8bq_gemm_i8(m, n, k, a, sa, w, sw, c, ws, nbytes, None)

    for bad in (dict(m=-1), dict(n=-1), dict(k=-128), dict(k=64), dict(k=130944 + 128), dict(m=1 << 31),
                dict(n=1 << 31), dict(m=1 << 21, n=1 << 21), dict(nbytes=-1)):
        assert call(**bad) == SHAPE, bad
    assert call(m=0, a=None, sa=None, w=None, sw=None, c=None) == 0
    assert call(n=0, a=None, sa=None, w=None, sw=None, c=None) == 0
    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(c=None), dict(nbytes=16)):
        assert call(**bad) == NULL, bad
    for bad in (dict(a=P + 8), dict(sa=P + 2), dict(w=P + 8), dict(sw=P + 1), dict(c=P + 2), dict(ws=P + 8)):
        assert call(**bad) == ALIGN, bad
    f = L.fp8bq_gemm_i8_workspace_bytes
    assert f(-1, 4, 128) == SHAPE and f(1, 4, 100) == SHAPE and f(0, 4, 128) == 0 and f(4, 4, 0) == 0
    for m in (1, 8, 16, 17, 33, 64, 65, 128, 257, 1024, 3465):
        for n, k in ((7168, 5120), (5120, 8704), (17408, 5120), (17, 128)):
            assert 0 <= f(m, n, k) <= 64 << 20


def test_verify_refusals(L):
    def call(b=1, k=2, v=10, dtype=0, t=P, q=P, d=P, ln=None, ua=P, us=P, ws=P, nbytes=1 << 20, tok=P, acc=P):
        return L.fp8bq_verify_drafts(b, k, v, dtype, t, q, d, ln, ua, us, ws, nbytes, tok, acc, None)

    for bad in (dict(b=-1), dict(b=65536), dict(k=-1), dict(k=65), dict(v=0), dict(v=1 << 31),
                dict(b=65535, k=64, v=1 << 20), dict(nbytes=0)):
        assert call(**bad) == SHAPE, bad
    assert call(dtype=2) == VALUE
    assert call(b=0, t=None, d=None, ua=None, us=None, ws=None, nbytes=0, tok=None, acc=None) == 0
    for bad in (dict(t=None), dict(d=None), dict(ua=None), dict(us=None), dict(ws=None), dict(tok=None), dict(acc=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(t=P + 2), dict(q=P + 2), dict(d=P + 1), dict(ln=P + 2), dict(ua=P + 2), dict(us=P + 2),
                dict(ws=P + 8), dict(tok=P + 2), dict(acc=P + 2), dict(t=P + 1, dtype=1)):
        assert call(**bad) == ALIGN, bad
    f = L.fp8bq_verify_workspace_bytes
    assert f(0, 2, 10) == 0 and f(-1, 2, 10) == SHAPE and f(1, 65, 10) == SHAPE and 0 < f(64, 7, 152064) <= 1 << 20


def test_binding_leaves_other_tensors_to_python(L):
    import torch

    from memory_bound_w8a8_amd import _binding

    x, w = torch.ones(2, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    assert _binding.rmsnorm(x, w, None, 1e-6, None, False, 0, 0) is None  # not on a GPU
    a, s = torch.ones(2, 128, dtype=torch.int8), torch.ones(2)
    assert _binding.gemm_i8(a, s, a, s, None, None, 0, 0) is None
    p, d, u = torch.ones(2, 2, 5), torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
    assert _binding.verify_drafts(p, d, u, s, None, None, None, 0, 0) is None
    for call in (_binding.rmsnorm, _binding.gemm_i8, _binding.verify_drafts):
        with pytest.raises(TypeError):
            call(x)


def test_tensors_off_the_gpu_are_refused(L):
    import torch

    import memory_bound_w8a8_amd as fp8bq

    x, w = torch.ones(2, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    a, s = torch.ones(2, 128, dtype=torch.int8), torch.ones(2)
    p, d, u = torch.ones(2, 2, 5), torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
    for call in (lambda: fp8bq.rmsnorm_quant(x, w), lambda: fp8bq.rmsnorm_quant_i8(x, w, x),
                 lambda: fp8bq.gemm_i8(a, s, a, s), lambda: fp8bq.verify_drafts(p, d, u, s),
                 lambda: fp8bq.quant_act_i8(x), lambda: fp8bq.quant_weight_i8(x.float())):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
    with pytest.raises(TypeError):
        fp8bq.rmsnorm_quant([1.0], w)
