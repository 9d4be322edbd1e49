"""GPU: int8 codes of every bf16 row maximum in the upper binades, both signs,
bitwise against the oracle: the quotient there is near the end of fp32's range
(tests/quotient_i8_check.c checks every pair on the host)."""

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from helpers import to_gpu
from oracle import quant_rows_i8_ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _values(patterns):
    return (np.asarray(patterns, np.uint32) << 16).view(np.float32)


def _rows(e):
    """Row a: every bf16 in the nine binades below the maximum (1 + a / 128) 2^e, both signs."""
    rows = np.zeros((128, 2560), np.float32)
    for a in range(128):
        amax = ((e + 127) << 7) + a
        x = _values(np.arange(amax - 1151, amax + 1))
        rows[a, :1152], rows[a, 1152:2304] = x, -x
    return rows


@pytest.mark.parametrize("e", [-96, -95, 1, *range(99, 128)])
def test_codes_up_to_the_largest_rows(e):
    rows = _rows(e)
    codes, scales = fp8bq.quant_act_i8(to_gpu(rows, BF16))
    want_c, want_s = quant_rows_i8_ref(rows)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    bad = np.argwhere(codes.cpu().numpy() != want_c)
    assert bad.size == 0, f"{len(bad)} differ, first at {bad[0]}"


@pytest.mark.parametrize("pattern", [0x7E51, 0x7EB3, 0x7ED1, 0x7F33, 0x7F51, 0x7F7F])
def test_norm_of_large_weights(pattern):
    # rows of ones: y is the weight itself
    w = np.resize(_rows((pattern >> 7) - 127)[pattern & 127], 2560)
    x = np.ones((3, 2560), np.float32)
    codes, scales, _ = fp8bq.rmsnorm_quant_i8(to_gpu(x, BF16), to_gpu(w, BF16), eps=1e-30)
    want_c, want_s = quant_rows_i8_ref(np.stack([w] * 3))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
