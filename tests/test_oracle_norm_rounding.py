"""Where the norm rounds (CPU): the inverse root once to fp32, then each of the
two products to fp32. Products kept in 64 bits put a few values in 10^6 on the
other side of a bf16 border, which shows in the codes."""

import numpy as np
import torch

from oracle import rmsnorm_ref

F32 = np.float32


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=F32)).to(torch.bfloat16).float().numpy()


def test_products_are_rounded_to_fp32_one_after_the_other():
    rng = np.random.default_rng(0)
    h, w = _bf16(3 * rng.standard_normal((400, 5120))), _bf16(1 + 0.1 * rng.standard_normal(5120))
    wide = 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-6)
    # a product of two fp32 numbers has 48 bits: exact in 64, then one rounding
    inv = wide.astype(F32).astype(np.float64)
    first = (h.astype(np.float64) * inv).astype(F32)
    want = _bf16((first.astype(np.float64) * w).astype(F32))
    y, _ = rmsnorm_ref(h, w)
    assert np.array_equal(y, want)
    other = _bf16(((h.astype(np.float64) * wide) * w).astype(F32))
    assert 0 < (want != other).sum() < 1e-4 * want.size  # the inputs tell the two forms apart


def test_inverse_is_held_to_the_largest_number():
    x = np.zeros((2, 128), F32)
    x[1, 3] = -0.0
    x[1, 4] = 2.0 ** -133  # the smallest bf16 number: the mean square is far below eps
    y, _ = rmsnorm_ref(x, np.ones(128, F32), eps=1e-300)
    assert not y[0].any() and np.isfinite(y).all()
    assert np.signbit(y[1, 3]) and y[1, 4] == _bf16([F32(2.0 ** -133) * np.finfo(F32).max])[0]


def test_zeros_keep_their_sign():
    x = np.ones((1, 128), F32)
    x[0, :4] = [0.0, -0.0, 0.0, -0.0]
    w = np.ones(128, F32)
    w[2:4] = -1.0
    y, _ = rmsnorm_ref(x, w)
    assert np.signbit(y[0, :4]).tolist() == [False, True, True, False]
