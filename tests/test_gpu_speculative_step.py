"""GPU: the example's decoding step against the oracle, layer by layer."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import memory_bound_w8a8_amd as fp8bq
from oracle import gemm_i8_ref, quant_rows_i8_ref, rmsnorm_ref, verify_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _f32(t):
    return t.float().cpu().numpy()


def test_layers_are_the_oracles(example, monkeypatch):
    model = example.Model(dim=256, layers=3, vocab=640, seed=3)
    tokens = torch.tensor([5, 9, 639, 0, 5], device="cuda")
    seen = []
    product = fp8bq.gemm
    monkeypatch.setattr(example.fp8bq, "gemm", lambda *args: seen.append(args) or product(*args))
    p = model.probabilities(tokens)
    assert p.shape == (5, 640) and torch.equal(p[0], p[4])
    x, r = _f32(model.embedding[tokens]), None
    for norm, (w_q, w_s) in zip(model.norms, model.layers):
        y, r = rmsnorm_ref(x, _f32(norm), r)
        codes, scales = quant_rows_i8_ref(y)
        x = gemm_i8_ref(codes, scales, w_q.cpu().numpy(), w_s.cpu().numpy())
    y, _ = rmsnorm_ref(x, _f32(model.norms[-1]), r)
    want = fp8bq.quant_act(torch.from_numpy(y).to(torch.bfloat16).cuda())
    assert torch.equal(seen[0][0], want[0]) and torch.equal(seen[0][1], want[1])


def test_steps_append_the_verified_tokens(example, monkeypatch):
    model = example.Model(dim=256, layers=1, vocab=640, seed=4)
    texts = [[1, 2, 3, 1, 2, 3, 1], [7], [9, 9, 9, 9], [4, 5, 4]]
    assert [example.lookup(t, 3) for t in texts] == [[2, 3, 1], [], [9], [5, 4]]
    checked = []
    verify = fp8bq.verify_drafts

    def watched(p, drafts, u_accept, u_sample, draft_len=None):
        out = verify(p, drafts, u_accept, u_sample, draft_len=draft_len)
        want = verify_ref(_f32(p), drafts.cpu().numpy(), _f32(u_accept), _f32(u_sample), None, draft_len.cpu().numpy())
        assert out[0].cpu().tolist() == want[0].tolist() and out[1].cpu().tolist() == want[1].tolist()
        checked.append(want)
        return out

    monkeypatch.setattr(example.fp8bq, "verify_drafts", watched)
    generator = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(4):
        before = [len(t) for t in texts]
        accepted = example.step(model, texts, 3, generator)
        assert [len(t) - b for t, b in zip(texts, before)] == [n + 1 for n in accepted]
        rows = checked[-1][0].tolist()
        assert [t[-n - 1:] for t, n in zip(texts, accepted)] == [row[:n + 1] for row, n in zip(rows, accepted)]
        assert all(0 <= token < 640 for t in texts for token in t)
    assert len(checked) == 4
