"""The limits that include/fp8bq_step.h states are the ones its calls keep
(host checks only, CPU)."""

import os

import pytest

P = 1 << 20  # an aligned, never-dereferenced address
SHAPE, ALIGN, VALUE = -2, -3, -7


@pytest.fixture(scope="module")
def L():
    import memory_bound_w8a8_amd as m

    if not os.path.exists(m.LIB_PATH):
        from memory_bound_w8a8_amd import build

        build.build()
    from memory_bound_w8a8_amd import step

    return step.step_lib()


def test_product_with_more_tiles_than_one_grid_is_a_shape(L):
    # 2^23 tiles of 256 x 256; the bad alignment of C keeps a call that passes from any device
    def call(m, n):
        return L.fp8bq_gemm_i8(m, n, 128, P, P, P, P, P + 2, None, 0, None)

    for m, n in ((2 ** 31 - 1, 1), (256 * 2 ** 11, 256 * 2 ** 12), (256 * (2 ** 23 - 1) + 1, 100)):
        assert call(m, n) == SHAPE, (m, n)
        assert L.fp8bq_gemm_i8_workspace_bytes(m, n, 128) == SHAPE, (m, n)
    for m, n in ((256 * (2 ** 23 - 1), 100), (256 * 2 ** 11, 256 * (2 ** 12 - 1)), (64, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        assert call(m, n) == ALIGN, (m, n)
        assert L.fp8bq_gemm_i8_workspace_bytes(m, n, 128) >= 0, (m, n)


@pytest.mark.parametrize("name", ["fp8bq_rmsnorm_quant", "fp8bq_rmsnorm_quant_i8"])
def test_every_finite_eps_serves(L, name):
    # the bad alignment of the codes is looked at after eps
    for eps, status in ((5e-324, ALIGN), (1e30, ALIGN), (2e30, ALIGN), (1.7e308, ALIGN), (float("inf"), VALUE),
                        (float("nan"), VALUE), (0.0, VALUE), (-1e300, VALUE)):
        assert getattr(L, name)(1, 128, P, None, P, eps, None, P + 2, P, None) == status, eps
