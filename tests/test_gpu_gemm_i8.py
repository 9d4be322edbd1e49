"""GPU: the int8 product, bitwise against the oracle.

The sums are exact on both sides, their conversion to fp32, the product of
the two scales, the product with it and the rounding to bf16 are one correctly
rounded operation each: C has to be equal bit for bit, whatever the tile, the
order or the split."""

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from helpers import to_gpu
from oracle import gemm_i8_ref

pytestmark = pytest.mark.gpu


def _problem(m, n, k, seed=0):
    rng = np.random.default_rng([seed, m, n, k])
    a = rng.integers(-128, 128, (m, k), dtype=np.int8)
    w = rng.integers(-128, 128, (n, k), dtype=np.int8)
    a_s = (rng.random(m) * 0.1 + 1e-3).astype(np.float32)
    w_s = (rng.random(n) * 1e-3 + 1e-5).astype(np.float32)
    return a, a_s, w, w_s


def _check(a, a_s, w, w_s):
    m, n, k = a.shape[0], w.shape[0], a.shape[1]
    want = gemm_i8_ref(a, a_s, w, w_s)
    args = [to_gpu(t) for t in (a, a_s, w, w_s)]
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    need = fp8bq.gemm_i8_workspace_bytes(m, n, k)
    dirty = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    for workspace in (none, dirty, None):
        out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
        got = fp8bq.gemm_i8(*args, out=out, workspace=workspace).float().cpu().numpy()
        bad = np.argwhere(got.view(np.uint32) != want.view(np.uint32))
        assert bad.size == 0, f"M={m} N={n} K={k}: {len(bad)} of {got.size} differ, first at {bad[0]}"


TOKENS = [1, 2, 3, 5, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 80, 96, 127, 128, 129, 200, 256, 257, 300]


@pytest.mark.parametrize("m", TOKENS)
@pytest.mark.parametrize("n,k", [(640, 1024), (701, 384), (130, 1152), (17, 128), (1, 256)])
def test_whole_output(m, n, k):
    _check(*_problem(m, n, k))


@pytest.mark.parametrize("m", [1, 8, 16, 17, 33, 64, 65, 130])
@pytest.mark.parametrize("n,k", [(5120, 8704), (7168, 5120), (8192, 5120), (4099, 2304)])
def test_layer_sizes(m, n, k):
    _check(*_problem(m, n, k, 1))


@pytest.mark.parametrize("m,n,k", [(1, 17408, 5120), (7, 17408, 5120), (40, 17408, 5120), (513, 1031, 640),
                                   (700, 2048, 512), (1025, 4096, 896), (2049, 770, 256)])
def test_larger(m, n, k):
    _check(*_problem(m, n, k, 2))


def _check_on_gpu(m, n, k, seed, workspace=None):
    """The whole output against the exact product in 64 bits, computed on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, w = (torch.randint(-128, 128, (rows, k), dtype=torch.int8, device="cuda", generator=g) for rows in (m, n))
    a_s, w_s = (torch.rand(rows, device="cuda", generator=g) * 0.01 + 1e-4 for rows in (m, n))
    got = fp8bq.gemm_i8(a, a_s, w, w_s, workspace=workspace)
    sums = torch.matmul(a.double(), w.double().t().contiguous())
    want = (sums.float() * (a_s[:, None] * w_s)).to(torch.bfloat16)
    bad = (got.view(torch.int16) != want.view(torch.int16)).nonzero()
    assert bad.numel() == 0, f"M={m} N={n} K={k}: {len(bad)} of {got.numel()} differ, first at {bad[0].tolist()}"


# each tile shape and its edges, one K step and many, one round of tiles and several
@pytest.mark.parametrize("m,n,k", [(129, 1000, 2560), (129, 8024, 4736), (90, 10001, 640), (302, 15014, 512),
                                   (346, 12445, 4480), (774, 9616, 1024), (2541, 4565, 1792), (1187, 1576, 1024),
                                   (300, 3001, 1280), (129, 15581, 2048), (129, 8192, 5120), (257, 8191, 5120),
                                   (1499, 5119, 1280), (2047, 7170, 1280), (1025, 17408, 640), (3465, 600, 512),
                                   (438, 7051, 3712), (2500, 9001, 5120), (3465, 8195, 5120), (5000, 17409, 128),
                                   (4097, 16385, 4096)])
def test_every_tile_shape(m, n, k):
    _check_on_gpu(m, n, k, 1)


# K split over workgroups: parts of unequal length, odd N, few and many parts
@pytest.mark.parametrize("m,n,k", [(33, 64, 16384), (63, 5120, 8704), (64, 5117, 8704), (65, 512, 5120),
                                   (128, 513, 8704), (300, 602, 8704), (65, 3, 130944), (1000, 130, 16512)])
def test_split_of_the_depth(m, n, k):
    need = fp8bq.gemm_i8_workspace_bytes(m, n, k)
    assert need >= 8 * m * n and need % (4 * m * n) == 0
    _check_on_gpu(m, n, k, 2)
    _check_on_gpu(m, n, k, 3, torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    _check_on_gpu(m, n, k, 4, torch.full((need - 1,), 255, dtype=torch.uint8, device="cuda"))  # too small: no split


@pytest.mark.parametrize("m,n,k", [(1, 400_000, 5632), (300, 400_000, 5632), (70_000, 31_000, 128)])
def test_offsets_past_31_bits(m, n, k):
    # weights or outputs of more than 2^31 entries, the last rows against the exact product
    assert max(n * k, m * n) > 2 ** 31
    a = torch.randint(-128, 128, (m, k), dtype=torch.int8, device="cuda")
    w = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda")
    a_s, w_s = torch.rand(m, device="cuda") + 0.1, torch.rand(n, device="cuda") + 0.1
    got = fp8bq.gemm_i8(a, a_s, w, w_s)
    rows, cols = slice(max(0, m - 300), m), slice(n - 300, n)
    sums = torch.matmul(a[rows].double(), w[cols].double().t().contiguous())
    want = (sums.float() * (a_s[rows, None] * w_s[cols])).to(torch.bfloat16)
    assert torch.equal(got[rows, cols], want)


@pytest.mark.parametrize("m,n", [(3, 20), (40, 64), (300, 300)])
def test_deepest_sum_stays_in_32_bits(m, n):
    k = 130944
    a, w = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    _check(a, np.full(m, 1e-6, np.float32), w, np.ones(n, np.float32))
    w[:, ::2] = 127
    _check(a, np.full(m, 1e-6, np.float32), w, np.ones(n, np.float32))


def test_zero_depth_and_empty():
    z = fp8bq.gemm_i8(torch.empty(3, 0, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"),
                      torch.empty(5, 0, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"))
    assert z.shape == (3, 5) and bool((z == 0).all())
    e = fp8bq.gemm_i8(torch.empty(0, 128, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"),
                      torch.empty(5, 128, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"))
    assert e.shape == (0, 5)


def test_extreme_scales():
    a, a_s, w, w_s = _problem(20, 70, 256, 3)
    a_s[:4] = [0.0, 1e-38, 1e30, 3e-39]
    w_s[:4] = [0.0, 1e-38, 1e8, 1e30]
    _check(a, a_s, w, w_s)


@pytest.mark.parametrize("m", [4, 40, 70])
def test_other_stream_and_graph_replay(m):
    a, a_s, w, w_s = (to_gpu(t) for t in _problem(m, 5120, 2048, 4))
    want = fp8bq.gemm_i8(a, a_s, w, w_s)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = fp8bq.gemm_i8(a, a_s, w, w_s)
    stream.synchronize()
    assert torch.equal(got, want)
    workspace = torch.empty(max(16, fp8bq.gemm_i8_workspace_bytes(m, 5120, 2048)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fp8bq.gemm_i8(a, a_s, w, w_s, workspace=workspace)
    for step in range(3):
        a.copy_(to_gpu(_problem(m, 1, 2048, 5 + step)[0]))
        graph.replay()
        want = fp8bq.gemm_i8(a, a_s, w, w_s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals():
    a, a_s, w, w_s = (to_gpu(t) for t in _problem(4, 8, 256, 6))
    with pytest.raises(TypeError):
        fp8bq.gemm_i8(a.view(torch.uint8), a_s, w, w_s)
    with pytest.raises(ValueError):
        fp8bq.gemm_i8(a, a_s, w[:, :128].contiguous(), w_s)
    with pytest.raises(ValueError):
        fp8bq.gemm_i8(a, a_s[:2], w, w_s)
    with pytest.raises(ValueError):
        fp8bq.gemm_i8(a, a_s, w.t(), w_s)
    with pytest.raises(ValueError):
        fp8bq.gemm_i8(a, a_s, w, w_s, out=torch.empty(4, 9, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fp8bq.Fp8bqError):
        fp8bq.gemm_i8(a[:, :100].contiguous(), a_s, w[:, :100].contiguous(), w_s)
