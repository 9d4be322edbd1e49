"""GPU: verification of drafted tokens, equal to the oracle's whole numbers
(the definition leaves no rounding to the order of a sum)."""

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from helpers import to_gpu
from oracle import verify_ref

pytestmark = pytest.mark.gpu

F32 = np.float32


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(F32)


def _problem(b, k, v, seed, bf16=False, spread=2.5):
    rng = np.random.default_rng([seed, b, k, v])
    z = spread * rng.standard_normal((b, k + 1, v))
    p = _softmax(z)
    q = _softmax(z[:, :k] + 0.6 * rng.standard_normal((b, k, v)))
    drafts = np.argmax(np.log(q + 1e-30) + rng.gumbel(size=q.shape), axis=-1) if k else np.zeros((b, 0))
    if bf16:
        p, q = (torch.from_numpy(t).to(torch.bfloat16).float().numpy() for t in (p, q))
    return p, q, drafts.astype(np.int32), rng.random((b, k)).astype(F32), rng.random(b).astype(F32)


def _check(p, q, drafts, ua, us, draft_len=None, bf16=False):
    want_t, want_n = verify_ref(p, drafts, ua, us, q, draft_len)
    kind = torch.bfloat16 if bf16 else torch.float32
    got_t, got_n = fp8bq.verify_drafts(
        to_gpu(p, kind), to_gpu(drafts.astype(np.int32)), to_gpu(ua), to_gpu(us), None if q is None else to_gpu(q, kind),
        None if draft_len is None else to_gpu(np.asarray(draft_len, np.int32)))
    assert got_n.cpu().tolist() == want_n.tolist()
    assert got_t.cpu().tolist() == want_t.tolist()


@pytest.mark.parametrize("b,k,v", [(1, 1, 1), (1, 3, 2), (2, 0, 5), (3, 2, 255), (5, 7, 256), (4, 4, 257), (33, 3, 1023),
                                   (64, 7, 1031), (2, 64, 4097), (17, 5, 20011), (1, 3, 152064), (3, 4, 151937)])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
def test_equals_the_definition(b, k, v, with_q, bf16):
    p, q, drafts, ua, us = _problem(b, k, v, 1, bf16)
    _check(p, q if with_q else None, drafts, ua, us, bf16=bf16)


def test_ragged_drafts_and_tokens_outside():
    b, k, v = 40, 5, 700
    p, q, drafts, ua, us = _problem(b, k, v, 2)
    rng = np.random.default_rng(3)
    lens = rng.integers(-1, k + 2, b)
    drafts[rng.random((b, k)) < 0.1] = -1
    drafts[rng.random((b, k)) < 0.05] = v
    drafts[0, 0] = np.iinfo(np.int32).max
    drafts[1, 0] = np.iinfo(np.int32).min
    ua *= 0.3
    _check(p, q, drafts, ua, us, lens)
    _check(p, None, drafts, ua, us, lens)


def test_all_accepted_and_none():
    p, q, drafts, ua, us = _problem(6, 4, 3000, 4)
    _check(p, q, drafts, np.zeros_like(ua), us)
    _check(p, q, drafts, np.full_like(ua, 1.0), us)
    _check(p, p[:, :4], drafts, ua, us)  # the drafter is the target: u < 1 accepts all
    _check(p, p[:, :4], drafts, np.full_like(ua, 1.0), us)  # rejected without a residual: the target's row


def test_ends_of_the_random_numbers():
    p, q, drafts, ua, us = _problem(8, 2, 5000, 5)
    p[:, :, :7] = 0.0  # words without weight at both ends are never drawn
    p[:, :, -9:] = 0.0
    ua[:] = 1.0
    for u in (0.0, 2.0 ** -40, 0.5, 1 - 2.0 ** -24):
        _check(p, q, drafts, ua, np.full(8, u, F32))
        _check(p, q, drafts, np.zeros_like(ua), np.full(8, u, F32))


def test_single_words_and_empty_rows():
    b, k, v = 6, 2, 2500
    p = np.zeros((b, k + 1, v), F32)
    for i in range(b - 1):
        p[i, :, (411 * i) % v] = 1.0  # one-hot; the last sequence has no weight at all
    drafts = np.array([[(411 * i) % v, 5] for i in range(b)], np.int32)
    u = np.full((b, k), 0.5, F32)
    us = np.linspace(0, 0.99, b).astype(F32)
    _check(p, None, drafts, u, us)
    _check(p, np.full((b, k, v), 1.0 / v, F32), drafts, u, us)


def test_values_that_are_no_probabilities():
    p, q, drafts, ua, us = _problem(6, 3, 1500, 6)
    p[0, :, 10] = np.nan
    p[1, :, 20] = np.inf
    p[2, :, 30] = -5.0
    p[3] = 2.0
    q[4, :, 40] = np.nan
    q[5, :, 50] = np.inf
    drafts[0, 0], drafts[1, 0], drafts[4, 0], drafts[5, 0] = 10, 20, 40, 50
    ua[:] = 0.999
    # acceptance of a NaN or an infinity is left out of the oracle: those drafts are compared by rule below
    pt, qt = to_gpu(p), to_gpu(q)
    tokens, n = fp8bq.verify_drafts(pt, to_gpu(drafts), to_gpu(ua), to_gpu(us), qt)
    n = n.cpu().numpy()
    assert n[0] == 0 and n[4] == 0  # NaN accepts nothing
    assert n[1] >= 1 and n[5] == 0  # u q < inf; u inf < p never
    drafts[1, 0], drafts[5, 0] = 21, 51
    _check(p, q, drafts, ua, us)
    _check(p, None, drafts, ua, us)


def test_smallest_weights():
    b, v = 4, 3000
    p = np.zeros((b, 1, v), F32)
    p[0, 0, 5::7] = 2.0 ** -32
    p[1, 0, :] = 2.0 ** -33  # half a unit: ties to even, nothing
    p[2, 0, :] = 1.5 * 2.0 ** -33
    p[3, 0, 2999] = 2.0 ** -32
    empty = np.zeros((b, 0))
    for u in (0.0, 0.37, 0.999):
        _check(p, None, empty.astype(np.int32), empty.astype(F32), np.full(b, u, F32))


def test_wide_vocabulary_past_32_bit_offsets():
    # 3 x 2 rows of 400,000,000 bf16: the rows start past 2^31 values
    b, k, v = 3, 1, 400_000_000
    p = torch.zeros(b, k + 1, v, dtype=torch.bfloat16, device="cuda")
    marks = [(0, 1, v - 1), (1, 0, 7), (2, 0, v // 2), (2, 1, 399_999_990)]
    for i, r, at in marks:
        p[i, r, at] = 0.5
    drafts = torch.tensor([[0], [0], [v // 2]], dtype=torch.int32, device="cuda")
    p[0, 0, 0] = 1.0
    tokens, n = fp8bq.verify_drafts(p, drafts, torch.full((b, k), 0.4, device="cuda"),
                                    torch.full((b,), 0.9, device="cuda"))
    assert n.cpu().tolist() == [1, 0, 1]
    assert tokens.cpu().tolist() == [[0, v - 1], [7, -1], [v // 2, 399_999_990]]


def test_workspace_contents_and_graph_replay():
    p, q, drafts, ua, us = _problem(9, 4, 30011, 7)
    args = [to_gpu(t) for t in (p, drafts, ua, us)]
    qg = to_gpu(q)
    want = fp8bq.verify_drafts(*args, qg)
    need = fp8bq.verify_workspace_bytes(9, 4, 30011)
    workspace = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = fp8bq.verify_drafts(*args, qg, workspace=workspace)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(fp8bq.Fp8bqError):
        fp8bq.verify_drafts(*args, qg, workspace=workspace[: need - 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fp8bq.verify_drafts(*args, qg, workspace=workspace)
    for step in range(3):
        fresh = _problem(9, 4, 30011, 8 + step)
        for t, f in zip(args, (fresh[0], fresh[2], fresh[3], fresh[4])):
            t.copy_(to_gpu(f))
        qg.copy_(to_gpu(fresh[1]))
        graph.replay()
        want = fp8bq.verify_drafts(*args, qg)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    p, q, drafts, ua, us = (to_gpu(t) for t in _problem(2, 3, 50, 9))
    with pytest.raises(TypeError):
        fp8bq.verify_drafts(p.half(), drafts, ua, us)
    with pytest.raises(TypeError):
        fp8bq.verify_drafts(p, drafts.long(), ua, us)
    with pytest.raises(TypeError):
        fp8bq.verify_drafts(p, drafts, ua, us, q.to(torch.bfloat16))
    with pytest.raises(ValueError):
        fp8bq.verify_drafts(p[:, :3].contiguous(), drafts, ua, us)
    with pytest.raises(ValueError):
        fp8bq.verify_drafts(p, drafts, ua, us, q[:, :2].contiguous())
    with pytest.raises(ValueError):
        fp8bq.verify_drafts(p, drafts, ua, us[:1])
    with pytest.raises(ValueError):
        fp8bq.verify_drafts(p, drafts, ua, us, draft_len=torch.zeros(3, dtype=torch.int32, device="cuda"))
