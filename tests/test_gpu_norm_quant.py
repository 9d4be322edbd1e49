"""GPU: norm with the residual's addition and 8-bit output, and the int8
quantisers, bitwise against the oracle.

Codes, scales and residual have to be equal bit for bit: the norm is computed
in 64 bits on both sides up to the rounding of y, so y can differ only where
its 64-bit value lies within about 2^-50 of a rounding border (one value in
10^8 or fewer, 2^-50 against the borders' distance of 2^-24 before the second
rounding), and every later operation is a single correctly rounded one on both
sides."""

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from helpers import to_gpu
from oracle import quant_act_ref, quant_rows_i8_ref, rmsnorm_ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(BF16)


def _inputs(m, k, seed, scale=1.0):
    rng = np.random.default_rng([seed, m, k])
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[rng.random((m, k)) < 0.002] *= 20
    r = 3 * rng.standard_normal((m, k))
    w = 1 + 0.1 * rng.standard_normal(k)
    return _bf16(scale * x), _bf16(scale * r), _bf16(w)


def _same(got, want):
    got = got.cpu().numpy()
    if got.dtype == np.float32:
        got, want = got.view(np.uint32), np.asarray(want, np.float32).view(np.uint32)
    assert np.array_equal(got, want)


def _check(x, r, w, eps=1e-6, i8=None):
    y, h = rmsnorm_ref(x, w, r, eps)
    xg, wg, rg = to_gpu(x), to_gpu(w), None if r is None else to_gpu(r)
    for want_i8 in ((False, True) if i8 is None else (i8,)):
        call = fp8bq.rmsnorm_quant_i8 if want_i8 else fp8bq.rmsnorm_quant
        codes, scales, h_out = call(xg, wg, rg, eps)
        want_c, want_s = (quant_rows_i8_ref if want_i8 else quant_act_ref)(y)
        _same(h_out.float(), h)
        _same(scales, want_s)
        _same(codes, want_c)
        if r is None:
            assert h_out is xg
        # the fused call is the quantiser on the norm's bf16 output
        two = (fp8bq.quant_act_i8 if want_i8 else fp8bq.quant_act)(to_gpu(_bf16(y)))
        assert torch.equal(codes, two[0]) and torch.equal(scales, two[1])


@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (1, 5120), (8, 5120), (17, 8704), (5, 8192), (4, 8320), (2, 16384),
                                 (3, 16512), (1, 32768), (2, 32896), (1, 65536), (301, 640)])
@pytest.mark.parametrize("residual", [True, False])
def test_codes_are_the_definitions(m, k, residual):
    x, r, w = _inputs(m, k, 1)
    _check(x, r if residual else None, w)


def test_more_rows_than_workgroups_take_at_once():
    x, r, w = _inputs(3465, 1024, 2)
    _check(x, r, w)


def test_rows_of_zeros_and_opposites():
    x, r, w = _inputs(6, 256, 3)
    x[1] = 0.0
    r[1] = 0.0
    r[2] = -x[2]  # the sum cancels: norm of zeros
    x[3] = -0.0
    r[3] = -0.0
    w[128:] = 0.0  # a group of zeros beside a group that is none
    _check(x, r, w)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e18, 1e36])
def test_far_magnitudes(scale):
    x, r, w = _inputs(5, 384, 4, scale)
    _check(x, r, w)
    # a mean far below eps gives tiny norms, whose scales come near the smallest fp32 numbers
    _check(x, None, _bf16(np.full(384, min(1.0, scale * 1e3))), eps=1.0)


def _group_scales(x, exponents):
    """x with group g of each row times 2^exponents[g % len]."""
    k = x.shape[1]
    e = np.repeat(np.resize(exponents, k // 128), 128)
    return _bf16(x.float().numpy() * np.exp2(e.astype(np.float64)).astype(np.float32))


@pytest.mark.parametrize("x_exp,w_exp", [((0, -40, -80, -110), (0,)), ((0,), (0, -60, -120, 60)),
                                         ((60, 0, -60), (60, -60, 100)), ((100, 64, 30), (0, 27)),
                                         ((-100, -126), (90, 120)), ((0, -100), (-100, -30))])
def test_groups_far_apart(x_exp, w_exp):
    # products of a value and its weight that leave fp32's range, or come near its smallest numbers, in some groups
    x, r, w = _inputs(5, 1536, 8)
    x, r = _group_scales(x, x_exp), _group_scales(r, x_exp)
    w = _group_scales(w[None], w_exp)[0]
    _check(x, r, w)
    _check(x, None, w)


def test_product_past_fp32_with_a_norm_inside_it():
    # h w overflows fp32, h inv w does not
    x, r, w = _inputs(4, 512, 9, 2.0 ** 70)
    w = _bf16(w.float().numpy() * 2.0 ** 80)
    _check(x, r, w)
    _check(x, None, w)


@pytest.mark.parametrize("eps", [1e-300, 1e-30, 1e30])
def test_ends_of_eps(eps):
    x, r, w = _inputs(4, 384, 10, 1e-3)
    x[2] = 0.0
    r[2] = 0.0
    _check(x, r, w, eps)


def test_weight_rows_of_the_smallest_numbers():
    rng = np.random.default_rng(11)
    w = np.zeros((200, 128), np.float32)
    for i in range(200):  # amax = i units of 2^-149: the scale is 0, 1 or 2 of them
        w[i] = (rng.integers(-i, i + 1, 128).astype(np.int64)).astype(np.float32) * np.float32(2.0 ** -149)
        w[i, 5] = np.float32(i) * np.float32(2.0 ** -149)
    codes, scales = fp8bq.quant_weight_i8(to_gpu(w))
    want_c, want_s = quant_rows_i8_ref(w)
    _same(codes, want_c)
    _same(scales, want_s)


def test_residual_in_place_and_out_tensor():
    x, r, w = _inputs(9, 640, 5)
    y, h = rmsnorm_ref(x, w, r)
    rg = to_gpu(r)
    codes, scales, out = fp8bq.rmsnorm_quant(to_gpu(x), to_gpu(w), rg, out_residual=rg)
    assert out is rg
    _same(rg.float(), h)
    _same(codes, quant_act_ref(y)[0])


@pytest.mark.parametrize("m,k", [(1, 128), (7, 5120), (33, 8704), (2, 65536), (3, 16512)])
def test_quantisers_by_rows(m, k):
    rng = np.random.default_rng([6, m, k])
    a = _bf16(rng.standard_normal((m, k)))
    a[m // 2] = 0.0
    codes, scales = fp8bq.quant_act_i8(to_gpu(a))
    want_c, want_s = quant_rows_i8_ref(a)
    _same(codes, want_c)
    _same(scales, want_s)
    w = (0.02 * rng.standard_normal((m, k))).astype(np.float32)
    codes, scales = fp8bq.quant_weight_i8(to_gpu(w))
    want_c, want_s = quant_rows_i8_ref(w)
    _same(codes, want_c)
    _same(scales, want_s)


def test_int8_ties_over_every_mantissa():
    # row a: amax = (1 + a / 128) 2^e; values: every bf16 in the eight binades below it
    for e in (-120, -100, -96, -20, 0, 90):
        mant = (1 + np.arange(128) / 128.0).astype(np.float32)
        below = np.concatenate([mant * 2.0 ** -j for j in range(9)])
        rows = np.zeros((128, 1280), np.float32)
        rows[:, :1152] = np.where(below[None] <= mant[:, None], below[None], 0)
        rows[:, 1152] = mant
        rows[:, 1] = -rows[:, 1]
        a = _bf16(rows * np.float32(2.0) ** e)
        codes, scales = fp8bq.quant_act_i8(to_gpu(a))
        want_c, want_s = quant_rows_i8_ref(a)
        _same(scales, want_s)
        _same(codes, want_c)


def test_empty_calls():
    w = torch.ones(128, dtype=BF16, device="cuda")
    codes, scales, h = fp8bq.rmsnorm_quant(torch.empty(0, 128, dtype=BF16, device="cuda"), w)
    assert codes.shape == (0, 128) and scales.shape == (0, 1) and h.shape == (0, 128)
    assert fp8bq.quant_act_i8(torch.empty(0, 128, dtype=BF16, device="cuda"))[1].shape == (0,)


def test_other_stream_and_graph_replay():
    x, r, w = (to_gpu(t) for t in _inputs(4, 5120, 7))
    want = fp8bq.rmsnorm_quant_i8(x, w, r)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = fp8bq.rmsnorm_quant_i8(x, w, r)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fp8bq.rmsnorm_quant_i8(x, w, r)
    for step in range(3):
        x.copy_(to_gpu(_inputs(4, 5120, 8 + step)[0]))
        graph.replay()
        want = fp8bq.rmsnorm_quant_i8(x, w, r)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    x, r, w = (to_gpu(t) for t in _inputs(4, 256, 9))
    with pytest.raises(TypeError):
        fp8bq.rmsnorm_quant(x.float(), w)
    with pytest.raises(ValueError):
        fp8bq.rmsnorm_quant(x.t(), w)
    with pytest.raises(ValueError):
        fp8bq.rmsnorm_quant(x, w[:128])
    with pytest.raises(ValueError):
        fp8bq.rmsnorm_quant(x, w, r[:2])
    with pytest.raises(ValueError):
        fp8bq.rmsnorm_quant(x, w, out_residual=r)
    with pytest.raises(fp8bq.Fp8bqError):
        fp8bq.rmsnorm_quant(x, w, eps=0.0)
    with pytest.raises(fp8bq.Fp8bqError):
        fp8bq.rmsnorm_quant(x[:, :100].contiguous(), w[:100].contiguous())
    with pytest.raises(ValueError):
        fp8bq.rmsnorm_quant(x.cpu(), w)
