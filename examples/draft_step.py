"""One step of block-drafted speculative decoding around a paged cache, and one
training step of its drafter, with the package's calls in the order a serving
loop makes them. Random weights, one attention layer, one LM head:

  1. the block's keys and values go into the paged cache, keys and queries
     rotated to their positions                             (kv_append)
  2. the block's queries attend over everything before them (paged_attention)
  3. the LM head projects the target's and the drafter's hidden states
                                                            (lmhead_logits)
  4. the drafts are verified; the cache keeps what was accepted (verify)
  5. the target's top logits of the verified positions move the drafter's
     hidden states towards it                               (distill_loss)

python examples/draft_step.py [--requests 8] [--steps 3]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import speculative_decoding_verification_83_gb300 as dv


class Layer:
    """A target layer's attention over its own pages: B requests, page tables
    filled as positions come up."""

    def __init__(self, B, q_heads, kv_heads, head_dim, max_len, page=64, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        hidden = q_heads * head_dim
        width = -(-max_len // page)
        self.shape = q_heads, kv_heads, head_dim
        self.wqkv = (torch.randn((hidden, (q_heads + 2 * kv_heads) * head_dim), generator=g, device=device)
                     / hidden ** 0.5).to(dtype)
        self.wo = (torch.randn((hidden, hidden), generator=g, device=device) / hidden ** 0.5).to(dtype)
        pages = torch.randperm(B * width, generator=g, device=device).view(B, width).to(torch.int32)
        kv = torch.zeros((2, B * width, kv_heads, page, head_dim), dtype=dtype, device=device)
        self.cache = dv.PagedCache(kv[0], kv[1], pages)
        self.phases = dv.rope_phases(1e6 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim), device)
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)

    def forward(self, x, status):
        """x [B, n, hidden]: the block's hidden states, at the positions behind
        self.lens (which the caller moves on once the block is verified)."""
        B, n, hidden = x.shape
        hq, hk, d = self.shape
        qkv = (x.reshape(B * n, hidden) @ self.wqkv).view(B * n, hq + 2 * hk, d)
        q = dv.kv_append(self.cache, qkv[:, hq:hq + hk], qkv[:, hq + hk:], self.lens, q=qkv[:, :hq],
                         phases=self.phases, status=status)
        y = dv.paged_attention(self.cache, q, self.lens + n, causal=True, status=status)
        return x + (y.view(B * n, hidden) @ self.wo).view(B, n, hidden)


def run(requests=8, gamma=7, vocab=4096, q_heads=16, kv_heads=2, head_dim=128, prompt=100, steps=3, top_k=20, seed=1):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hidden, B = q_heads * head_dim, requests
    layer = Layer(B, q_heads, kv_heads, head_dim, prompt + (steps + 1) * (gamma + 1), seed=seed)
    emb = torch.randn((vocab, hidden), generator=g, device=dev).to(torch.bfloat16)
    head = (torch.randn((vocab, hidden), generator=g, device=dev) * (2.0 / hidden ** 0.5)).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    temperature = torch.ones(B, device=dev)
    # the prompts, of one length here
    tokens = torch.randint(0, vocab, (B, prompt), generator=g, device=dev)
    layer.forward(emb[tokens], status)
    layer.lens += prompt
    last = tokens[:, -1:].to(torch.int32)
    # the drafter: a state per position (random here), trained by the step's loss
    drafter = torch.randn((B, gamma, hidden), generator=g, device=dev).to(torch.bfloat16).requires_grad_(True)
    report = []
    for step in range(steps):
        with torch.no_grad():
            q_logits = dv.lmhead_logits(drafter.view(B * gamma, hidden), head)
            drafts = dv.sample_rows(q_logits, temperature.repeat_interleave(gamma), top_k, 0.95, seed * 1000 + step)
            drafts = drafts.view(B, gamma)
            block = torch.cat([last, drafts], 1)
            h = layer.forward(emb[block.long()], status)
            p_logits = dv.lmhead_logits(h.reshape(B * (gamma + 1), hidden), head).view(B, gamma + 1, vocab)
            out, length = dv.verify(p_logits, q_logits.view(B, gamma, vocab), drafts, temperature, top_k, 0.95,
                                    seed * 7919 + step, status=status)
            layer.lens += length  # the block's first slot and the accepted drafts stay; the rest is written over
            last = out.gather(1, (length - 1).long()[:, None])
            teacher, ids = p_logits[:, :gamma].reshape(B * gamma, vocab).float().topk(32, dim=1)
            # positions after the first rejection were conditioned on a token that is not there
            weight = (torch.arange(gamma, device=dev)[None] < length[:, None]).float().view(-1)
        logits = drafter.view(B * gamma, hidden) @ head.t()
        loss = dv.distill_loss(logits, ids.to(torch.int32), teacher, row_weight=weight, status=status).sum() / weight.sum()
        drafter.grad = None
        loss.backward()
        with torch.no_grad():
            drafter -= 20.0 * drafter.grad
            after = dv.distill_loss(drafter.view(B * gamma, hidden) @ head.t(), ids.to(torch.int32), teacher,
                                    row_weight=weight, status=status).sum() / weight.sum()
        report.append((float(loss.detach()), float(after), float(length.float().mean())))
    if int(status):
        raise RuntimeError(f"status {int(status)}")
    return report


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args()
    dv.build()
    for i, (loss, after, accepted) in enumerate(run(a.requests, steps=a.steps)):
        print(f"step {i}: loss {loss:.4f}, after its update {after:.4f}, tokens per verification {accepted:.2f}")
