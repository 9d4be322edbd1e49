"""GPU: the norm's codes, scales and residual against the elementary form in
torch, bit for bit at the sizes of a prompt, and the signs of zeros.

Both sides round at the same places (tests/test_oracle_norm_rounding.py), so
nothing may differ but where the 64-bit root's inverse lies within about 2^-50
of the border between two fp32 numbers: one row in 10^7."""

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from helpers import to_gpu
from oracle import quant_act_ref, rmsnorm_ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _inputs(m, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(m, k, device="cuda", generator=g)
    x = torch.where(torch.rand(m, k, device="cuda", generator=g) < 0.001, 20 * x, x)
    r = 3 * torch.randn(m, k, device="cuda", generator=g)
    w = 1 + 0.1 * torch.randn(k, device="cuda", generator=g)
    return x.to(BF16), r.to(BF16), w.to(BF16)


def _elementary(x, w, r, i8):
    h = x if r is None else (x.float() + r.float()).to(BF16)
    inv = (1.0 / (h.double().square().mean(1, keepdim=True) + 1e-6).sqrt()).float()
    y = ((h.float() * inv) * w.float()).to(BF16).float()
    m, k = y.shape
    top = torch.tensor(127.0 if i8 else 448.0, device="cuda")  # a tensor: a true division, no product with 1 / top
    groups = y.view(m, -1, k if i8 else 128)
    amax = groups.abs().amax(2, keepdim=True)
    scales = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    q = (groups / scales).clamp(-float(top), float(top)).view(m, k)
    codes = q.round().to(torch.int8) if i8 else q.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales.view(m, -1) if not i8 else scales.view(m), h


@pytest.mark.parametrize("m,k,residual", [(3465, 5120, True), (2049, 8704, False), (1731, 4352, True), (257, 8320, True),
                                          (9, 16384, False), (64, 640, True)])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("seed", [1, 2])
def test_equals_the_elementary_form(m, k, residual, i8, seed):
    x, r, w = _inputs(m, k, seed)
    r = r if residual else None
    got = (fp8bq.rmsnorm_quant_i8 if i8 else fp8bq.rmsnorm_quant)(x, w, r)
    for name, u, v in zip(("codes", "scales", "residual"), got, _elementary(x, w, r, i8)):
        assert u.shape == v.shape and u.dtype == v.dtype, name
        bad = (u != v).nonzero()
        assert bad.numel() == 0, f"{name}: {len(bad)} of {u.numel()} differ, first at {bad[0].tolist()}"


def test_zeros_keep_their_sign():
    rng = np.random.default_rng(3)
    x, _, w = (t.float().cpu().numpy() for t in _inputs(64, 640, 4))
    x[rng.random(x.shape) < 0.1] = 0.0
    x[rng.random(x.shape) < 0.1] = -0.0
    w[rng.random(w.shape) < 0.5] *= -1
    codes, scales, _ = fp8bq.rmsnorm_quant(to_gpu(x, BF16), to_gpu(w, BF16))
    y, _ = rmsnorm_ref(x, w)
    want_c, want_s = quant_act_ref(y)
    assert 0 < (want_c == 0x80).sum() < want_c.size
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s)


def test_inverse_past_the_largest_number():
    x = np.zeros((3, 256), np.float32)
    x[1, 3], x[1, 200] = 2.0 ** -133, -2.0 ** -130
    x[2] = 2.0 ** -127
    w = np.ones(256, np.float32)
    codes, scales, _ = fp8bq.rmsnorm_quant(to_gpu(x, BF16), to_gpu(w, BF16), eps=1e-300)
    y, _ = rmsnorm_ref(x, w, eps=1e-300)
    assert np.isfinite(y).all()
    want_c, want_s = quant_act_ref(y)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s)
