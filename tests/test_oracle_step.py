"""Pins of the oracle's functions for the operators around the linear layer:
closed forms, torch's own conversions and exact rational brute force (CPU)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draw_ref, gemm_i8_ref, quant_rows_i8_ref, rmsnorm_ref, verify_ref, weight_units
from oracle.step import bf16_round

F32 = np.float32


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=F32)).to(torch.bfloat16).float().numpy()


def test_bf16_round_equals_torch():
    rng = np.random.default_rng(0)
    x = rng.integers(0, 2 ** 32, 1 << 16, dtype=np.uint64).astype(np.uint32).view(F32)
    x = np.concatenate([x[np.isfinite(x)], np.array([0.0, -0.0, 1.00390625, 1.01171875], F32)])
    assert np.array_equal(bf16_round(x).view(np.uint32), _bf16(x).view(np.uint32))


def test_norm_closed_forms():
    # constant rows: y = sign(h) w / sqrt(1 + eps / h^2), exact for eps << h^2
    w = _bf16(np.linspace(0.5, 2.0, 128))
    x = np.array([[3.0], [-0.25], [0.0]], F32) * np.ones((1, 128), F32)
    y, h = rmsnorm_ref(x, w, eps=1e-30)
    assert np.array_equal(h, x)
    assert np.array_equal(y, np.stack([w, -w, 0 * w]))
    # the residual's addition is rounded to bf16 before the norm sees it
    r = np.full((1, 128), 1.0, F32)
    y, h = rmsnorm_ref(np.full((1, 128), 2.0 ** -9, F32), w, r)
    assert np.all(h == 1.0)


def test_norm_against_fractions():
    rng = np.random.default_rng(1)
    x, r = _bf16(rng.standard_normal((4, 128))), _bf16(3 * rng.standard_normal((4, 128)))
    w = _bf16(1 + 0.1 * rng.standard_normal(128))
    eps = 1e-6
    y, h = rmsnorm_ref(x, w, r, eps)
    assert np.array_equal(h, _bf16(x.astype(np.float64) + r))
    for i in range(4):
        mean = sum(Fraction(float(v)) ** 2 for v in h[i]) / 128 + Fraction(eps)
        for j in range(128):
            # |y| = |h w| / sqrt(mean): half a bf16 step (eps / 2 = 2^-8) and three fp32 roundings
            square = Fraction(float(h[i, j])) ** 2 * Fraction(float(w[j])) ** 2 / mean
            true = float(square) ** 0.5 * np.sign(h[i, j] * w[j])
            assert abs(float(y[i, j]) - true) <= abs(true) * (torch.finfo(torch.bfloat16).eps / 2 + 4 * 2.0 ** -24)


def test_quant_rows():
    x = np.array([[0.0] * 8, [127, -127, 63.5, -63.5, 0.5, 1.5, -2.5, 0], [1e-3, 0, 0, 0, -5e-4, 2.5e-4, 0, 0]], F32)
    q, s = quant_rows_i8_ref(x)
    assert s[0] == 1.0 and not q[0].any()
    assert s[1] == 1.0 and q[1].tolist() == [127, -127, 64, -64, 0, 2, -2, 0]
    assert q[2, 0] == 127
    rng = np.random.default_rng(2)
    x = _bf16(rng.standard_normal((5, 256)))
    q, s = quant_rows_i8_ref(x)
    for i in range(5):
        assert s[i] == F32(F32(np.abs(x[i]).max()) / F32(127))
        # nearest whole number of the exact quotient, but for ties moved by the fp32 division (2^-24 relative)
        exact = [Fraction(float(v)) / Fraction(float(s[i])) for v in x[i]]
        assert all(abs(e - int(c)) <= Fraction(1, 2) + abs(e) * Fraction(1, 2 ** 24) for e, c in zip(exact, q[i]))


def test_gemm_i8_against_whole_numbers():
    rng = np.random.default_rng(3)
    a, w = rng.integers(-128, 128, (3, 256)).astype(np.int8), rng.integers(-128, 128, (5, 256)).astype(np.int8)
    a_s, w_s = rng.random(3).astype(F32), rng.random(5).astype(F32)
    c = gemm_i8_ref(a, a_s, w, w_s)
    for m in range(3):
        for n in range(5):
            s = sum(int(x) * int(y) for x, y in zip(a[m], w[n]))
            assert c[m, n] == _bf16([F32(s) * F32(a_s[m] * w_s[n])])[0]


def test_weight_units():
    w = np.array([0.0, -1.0, np.nan, 1.0, 2.0, np.inf, 2.0 ** -32, 2.0 ** -33, 1.5 * 2.0 ** -32, 2.5 * 2.0 ** -32], F32)
    assert weight_units(w).tolist() == [0, 0, 0, 2 ** 32 - 1, 2 ** 32 - 1, 2 ** 32 - 1, 1, 0, 2, 2]


def test_draw_covers_every_point_once():
    units = np.array([0, 3, 0, 1, 4, 0], np.int64)  # S = 8: the points z / 2^32 of eighths
    got = [draw_ref(units, j / 8) for j in range(8)]
    assert got == [1, 1, 1, 3, 4, 4, 4, 4]
    assert draw_ref(np.zeros(4, np.int64), 0.5) == -1
    assert draw_ref(units, 0.9999999) == 4


@pytest.mark.parametrize("certain", [False, True])
def test_verification_keeps_the_target_distribution(certain):
    # one draft: over a grid of the random numbers, the first token's distribution is the target's
    v, g = 4, 64
    p = np.array([0.5, 0.25, 0.125, 0.125], F32)
    q = np.array([0.25, 0.25, 0.0, 0.5], F32)
    target = np.stack([p, p])[None]
    counts = np.zeros(v)
    for d in range(v):
        weight = float(q[d]) if not certain else 0.25  # a certain drafter's choice does not matter
        if weight == 0:
            continue
        for ua in range(g):
            for us in range(g):
                t, n = verify_ref(target, np.array([[d]]), np.array([[ua / g]], F32), np.array([us / g], F32),
                                  None if certain else q[None, None])
                assert n[0] in (0, 1) and (t[0, 1] >= 0) == (n[0] == 1)
                counts[t[0, 0]] += weight
    # grid points are multiples of 1/64; the residual's shares are met within one grid step each
    assert np.abs(counts / counts.sum() - p).max() <= 1.0 / g


def test_verification_rules():
    v = 5
    p = np.full((1, 4, v), 0.2, F32)
    half = np.array([0.5], F32)
    drafts = np.array([[1, 7, 2]])
    u = np.zeros((1, 3), F32)
    t, n = verify_ref(p, drafts, u, half)  # the token outside the vocabulary ends the drafts
    assert n[0] == 1 and t[0, 0] == 1 and t[0, 2] == -1
    t, n = verify_ref(p, np.array([[1, 3, 2]]), u, half, draft_len=np.array([0]))
    assert n[0] == 0 and t[0].tolist() == [2, -1, -1, -1]
    q = p[:, :3].copy()
    t, n = verify_ref(p, np.array([[1, 3, 2]]), np.array([[0.0, 1.0, 0.0]], F32), half, q)
    assert n[0] == 1 and t[0, 1] == 2  # u q < p fails at u = 1; no residual: drawn from the target
    nothing = np.zeros((1, 4, v), F32)
    t, n = verify_ref(nothing, drafts, u, half)
    assert n[0] == 0 and t[0].tolist() == [-1] * 4


def test_int8_rows_of_the_smallest_numbers():
    x = (np.array([[63, -20], [64, -64], [190, -190], [0, 0]]) * 2.0 ** -149).astype(F32)
    codes, scales = quant_rows_i8_ref(x)
    assert scales.tolist() == [1.0, 2.0 ** -149, 2.0 ** -149, 1.0]  # 63 / 127 units round to 0, 190 / 127 to 1
    assert codes.tolist() == [[0, 0], [64, -64], [127, -127], [0, 0]]


def test_two_float_inverse_is_the_64_bit_product():
    # y = fma(h w, hi, (h w) lo) with hi + lo the inverse: the bf16 of the 64-bit product, as the kernels form it
    rng = np.random.default_rng(12)
    h = _bf16(3 * rng.standard_normal(1 << 18))
    w = _bf16(1 + 0.1 * rng.standard_normal(1 << 18))
    inv = 1.0 / np.sqrt(rng.random(1 << 18) * 10 + 1e-6)
    hi = inv.astype(F32)
    lo = (inv - hi).astype(F32)
    p = h * w
    assert np.array_equal(p.astype(np.float64), h.astype(np.float64) * w)
    # the fma's one rounding: its exact sum is below 2^53 units of the smaller term's last place, but for that sum's own
    y = (p.astype(np.float64) * hi + (p * lo).astype(np.float64)).astype(F32)
    assert np.array_equal(bf16_round(y), bf16_round(((h.astype(np.float64) * inv) * w).astype(F32)))
