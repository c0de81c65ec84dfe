"""A drafter's training on packed sequences, and the same layer serving them from a
paged cache: one attention layer and the LM head, random weights and tokens.

  training   norm_rotate -> packed_attention -> linear_cross_entropy, with the
             gradients of every weight (autograd)
  serving    kv_append with norms -> paged_attention, the prompt in two chunks

python examples/train_drafter.py [--steps 5]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import speculative_decoding_verification_83_gb300 as dv


class Drafter:
    """Embedding, one attention layer with norms of queries and keys, LM head."""

    def __init__(self, vocab=4000, q_heads=8, kv_heads=2, head_dim=64, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        hidden = q_heads * head_dim
        self.shape = q_heads, kv_heads, head_dim

        def weight(*shape, scale=1.0):
            w = torch.randn(shape, generator=g, device=device) * (scale / shape[-1] ** 0.5)
            return w.to(torch.bfloat16).requires_grad_(True)

        self.weights = {
            "emb": weight(vocab, hidden, scale=hidden ** 0.5), "qkv": weight((q_heads + 2 * kv_heads) * head_dim, hidden),
            "out": weight(hidden, hidden), "head": weight(vocab, hidden, scale=2.0),
            "q_norm": torch.ones(head_dim, device=device, requires_grad=True),
            "k_norm": torch.ones(head_dim, device=device, requires_grad=True)}
        self.phases = dv.rope_phases(1e5 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim), device)

    def project(self, tokens):
        hq, hk, d = self.shape
        x = self.weights["emb"][tokens]
        qkv = (x @ self.weights["qkv"].t()).view(len(tokens), hq + 2 * hk, d)
        return x, qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]

    def hidden(self, tokens, starts, positions, status=None):
        """The packed sequences' last hidden states (sequence b: tokens starts[b] .. starts[b + 1] - 1)."""
        x, q, k, v = self.project(tokens)
        q, k = dv.norm_rotate(q, k, self.weights["q_norm"], self.weights["k_norm"], positions, self.phases)
        y = dv.packed_attention(q, k, v, starts, status=status)
        return x + y.flatten(1) @ self.weights["out"].t()

    def losses(self, tokens, starts, positions, labels, row_weight=None, status=None):
        """Per token; label -1 takes no part."""
        return dv.linear_cross_entropy(self.hidden(tokens, starts, positions, status), self.weights["head"], labels,
                                       row_weight=row_weight, status=status)

    @torch.no_grad()
    def serve(self, cache, tokens, lens, starts, status=None):
        """New tokens of requests whose first `lens` are in the cache; the cache keeps the new ones."""
        x, q, k, v = self.project(tokens)
        q = dv.kv_append(cache, k, v, lens, q_start=starts, q=q, phases=self.phases, eps=1e-6, status=status,
                         q_weight=self.weights["q_norm"], k_weight=self.weights["k_norm"])
        y = dv.paged_attention(cache, q, lens + starts.diff(), q_start=starts, status=status)
        return x + y.flatten(1) @ self.weights["out"].t()


def batch(counts, vocab, seed=1, device="cuda"):
    """Packed sequences of random tokens: tokens, first tokens, positions, and each token's next one as its label."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    n = torch.tensor(counts, device=device)
    starts = torch.zeros(len(counts) + 1, device=device, dtype=torch.int32)
    starts[1:] = n.cumsum(0)
    tokens = torch.randint(0, vocab, (sum(counts),), generator=g, device=device)
    positions = torch.cat([torch.arange(c, device=device, dtype=torch.int32) for c in counts])
    labels = tokens.roll(-1).to(torch.int32)
    labels[(starts[1:] - 1).long()] = -1  # a sequence's last token has no next one
    return tokens, starts, positions, labels


def run(counts=(300, 17, 150), steps=5, lr=0.5, seed=1):
    vocab = 4000
    drafter = Drafter(vocab, seed=seed)
    tokens, starts, positions, labels = batch(counts, vocab, seed)
    used = int((labels >= 0).sum())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    report = []
    for _ in range(steps):
        loss = drafter.losses(tokens, starts, positions, labels, status=status).sum() / used
        grads = torch.autograd.grad(loss, list(drafter.weights.values()))
        with torch.no_grad():
            for w, dw in zip(drafter.weights.values(), grads):
                w -= lr * dw
        report.append(float(loss.detach()))
    if int(status):
        raise RuntimeError(f"status {int(status)}")
    return report


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    dv.build()
    for i, loss in enumerate(run(steps=a.steps)):
        print(f"step {i}: loss {loss:.4f}")
