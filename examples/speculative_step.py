"""Speculative decoding steps of a small random model, on one GPU.

    python examples/speculative_step.py [--steps 30] [--drafts 4] [--streams 8]

Each step verifies the drafts of every stream with one pass over their last
tokens, as a serving program would:

    rmsnorm_quant_i8 -> gemm_i8      in every layer (int8 codes, a scale per token and channel)
    rmsnorm_quant    -> gemm         at the vocabulary projection (e4m3 codes, block scales)
    softmax          -> verify_drafts

The drafts are looked up in the stream's own text (the tokens that followed
the last occurrence of its last token), so they are certain (no draft_p). The
model looks at single tokens only: there is no cache to keep.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import memory_bound_w8a8_amd as fp8bq  # noqa: E402


class Model:
    """`layers` residual layers of width `dim` over a vocabulary of `vocab`."""

    def __init__(self, dim=1024, layers=4, vocab=256, seed=0):
        g = torch.Generator().manual_seed(seed)

        def matrix(rows, gain=1.0):
            return (torch.randn(rows, dim, generator=g) * gain / dim ** 0.5).cuda()

        self.vocab = vocab
        self.embedding = torch.randn(vocab, dim, generator=g).to(torch.bfloat16).cuda()
        self.norms = [torch.ones(dim, dtype=torch.bfloat16, device="cuda") for _ in range(layers + 1)]
        self.layers = [fp8bq.quant_weight_i8(matrix(dim)) for _ in range(layers)]
        self.head = fp8bq.quant_weight(matrix(vocab, gain=20.0))  # peaked: the text repeats itself soon

    def probabilities(self, tokens):
        """int64 tokens [M] -> fp32 probabilities of the next one [M, vocab]."""
        x, residual = self.embedding[tokens], None
        for norm, (w_q, w_s) in zip(self.norms, self.layers):
            a_q, a_s, residual = fp8bq.rmsnorm_quant_i8(x, norm, residual)
            x = fp8bq.gemm_i8(a_q, a_s, w_q, w_s)
        a_q, a_s, _ = fp8bq.rmsnorm_quant(x, self.norms[-1], residual)
        return torch.softmax(fp8bq.gemm(a_q, a_s, *self.head).float(), -1)


def lookup(text, count):
    """Up to `count` tokens that followed the last earlier occurrence of text's last token."""
    for at in range(len(text) - 2, -1, -1):
        if text[at] == text[-1]:
            return text[at + 1:at + 1 + count]
    return []


def step(model, texts, count, generator):
    """One step of every stream: drafts, their verification, and the new
    tokens appended to `texts`. Returns the drafts accepted in each."""
    drafts = [lookup(text, count) for text in texts]
    padded = torch.tensor([d + [0] * (count - len(d)) for d in drafts], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([len(d) for d in drafts], dtype=torch.int32, device="cuda")
    last = torch.tensor([[t[-1]] for t in texts], device="cuda")
    inputs = torch.cat([last, padded.long()], 1)
    p = model.probabilities(inputs.reshape(-1)).view(len(texts), count + 1, model.vocab)
    tokens, accepted = fp8bq.verify_drafts(
        p, padded, torch.rand(padded.shape, device="cuda", generator=generator),
        torch.rand(len(texts), device="cuda", generator=generator), draft_len=lengths)
    accepted = accepted.tolist()
    for text, row, n in zip(texts, tokens.tolist(), accepted):
        text.extend(row[:n + 1])
    return accepted


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=30)
    parser.add_argument("--drafts", type=int, default=4)
    parser.add_argument("--streams", type=int, default=8)
    args = parser.parse_args()
    model = Model()
    generator = torch.Generator(device="cuda").manual_seed(1)
    # texts that repeat, so that there is something to look up
    texts = [[(17 * s + i % 5) % model.vocab for i in range(12)] for s in range(args.streams)]
    for i in range(args.steps):
        accepted = step(model, texts, args.drafts, generator)
        print(f"step {i}: accepted {accepted}, {sum(accepted) + len(texts)} tokens", flush=True)
    print("first text:", texts[0])


if __name__ == "__main__":
    main()
