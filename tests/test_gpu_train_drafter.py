"""The training operators in a run, as the example makes it: every weight's gradient
against the same network in 64 bits, and the same layer serving from a paged cache."""
import os
import sys
import weakref

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as dv

    dv.build()
    dv.load()
    import train_drafter

    return train_drafter


def network64(d, weights, tokens, counts, positions, labels):
    """Losses of the example's network, from the definitions."""
    hq, hk, D = d.shape
    w = weights
    x = w["emb"][tokens]
    qkv = (x @ w["qkv"].t()).view(len(tokens), hq + 2 * hk, D)
    freq = 1e5 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=x.device) / D)
    ang = positions.double()[:, None, None] * freq

    def normed(t, g):
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * g
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    q, k, v = normed(qkv[:, :hq], w["q_norm"]), normed(qkv[:, hq:hq + hk], w["k_norm"]), qkv[:, hq + hk:]
    outs, i = [], 0
    for n in counts:
        s = torch.einsum("nhd,mhd->hnm", q[i:i + n], k[i:i + n].repeat_interleave(hq // hk, 1)) * D ** -0.5
        s = s.masked_fill(torch.ones((n, n), dtype=torch.bool, device=x.device).triu(1), -torch.inf)
        outs.append(torch.einsum("hnm,mhd->nhd", torch.softmax(s, -1), v[i:i + n].repeat_interleave(hq // hk, 1)))
        i += n
    h = x + torch.cat(outs).flatten(1) @ w["out"].t()
    used = labels >= 0
    logp = torch.log_softmax(h @ w["head"].t(), 1)
    return torch.where(used, -logp.gather(1, labels.long().clamp(0)[:, None])[:, 0], 0.0)


@pytest.mark.parametrize("counts", [[1, 2], [130, 7, 64], [300]])
def test_gradients_of_every_weight(ex, counts):
    d = ex.Drafter(vocab=1000)
    tokens, starts, positions, labels = ex.batch(counts, 1000)
    if not bool((labels >= 0).any()):
        labels[0] = 3
    loss = d.losses(tokens, starts, positions, labels).sum()
    grads = torch.autograd.grad(loss, list(d.weights.values()))
    wide = {n: w.detach().double().requires_grad_(True) for n, w in d.weights.items()}
    want_loss = network64(d, wide, tokens, counts, positions, labels).sum()
    want = torch.autograd.grad(want_loss, list(wide.values()))
    # Between a weight and the loss lie at most 10 tensors rounded to bf16 on the way there and 10 on the way back, each
    # by at most 2^-8 of its values; a change of a tensor is passed on without growing (norms, residual, softmax).
    bound = 20 * 2.0 ** -8
    assert abs(float(loss.detach()) - float(want_loss.detach())) <= bound * abs(float(want_loss.detach()))
    # Where a query sees one key, dS = P (dP - delta) is 0, and what is left of it a rounding: dP and delta are sums of D =
    # 64 products in fp32, so |dS| <= 2^-16 |dout| |v|, dq <= |dS| |k| / sqrt(D) and dw <= |dq| |x r| with |v|, |k|, |x r| about
    # sqrt(D) = 8: 2^-10 |dout|. The gradient of the values' projection is |x| |dout| with |x| about sqrt(512) = 22: that
    # times 2^-14 is as much, for the weights that reach the loss through dS.
    least = 2.0 ** -14 * float(want[list(d.weights).index("qkv")].norm())
    for n, g, r in zip(d.weights, grads, want):
        assert float((g.double() - r).norm()) <= bound * float(r.norm()) + (least if n in ("q_norm", "k_norm") else 0.0), n


def test_serving_agrees_with_packed_sequences(ex):
    """The prompts in two chunks through the paged cache, against the packed sequences: bf16 roundings in other
    places (the cached keys, two kernels' weights and outputs)."""
    import speculative_decoding_verification_83_gb300 as dv

    counts, first = [150, 33, 70], [100, 1, 70]
    d = ex.Drafter(vocab=1000)
    tokens, starts, positions, _ = ex.batch(counts, 1000)
    with torch.no_grad():
        want = d.hidden(tokens, starts, positions)
    B, width, (_, hk, D) = len(counts), 10, d.shape
    table = torch.randperm(B * width, device="cuda").view(B, width).to(torch.int32)
    kv = torch.zeros((2, B * width, hk, 16, D), dtype=torch.bfloat16, device="cuda")
    cache = dv.PagedCache(kv[0], kv[1], table)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = torch.zeros_like(want)
    s = starts.tolist()
    for chunk in range(2):
        rows = [torch.arange(s[b], s[b] + first[b]) if chunk == 0 else torch.arange(s[b] + first[b], s[b + 1]) for b in range(B)]
        at = torch.cat(rows).cuda()
        part = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        part[1:] = torch.tensor([len(r) for r in rows]).cumsum(0)
        got[at] = d.serve(cache, tokens[at], lens, part, status)
        lens += part.diff()
    assert int(status) == 0
    assert float((got.double() - want.double()).norm()) <= 8 * 2.0 ** -8 * float(want.double().norm())


def test_example_runs(ex):
    report = ex.run(counts=(40, 9), steps=2)
    assert len(report) == 2 and all(0 < x < 100 for x in report)


def test_a_status_word_may_be_reset_between_the_passes(ex):
    """The word is its owner's: read and reset after the forward passes, it still takes the backward passes' reports."""
    dv, g = ex.dv, torch.Generator(device="cuda")
    g.manual_seed(4)
    q, k, v = (torch.randn((40, 2, 64), generator=g, device="cuda").bfloat16().requires_grad_(True) for _ in range(3))
    w = torch.randn((50, 128), generator=g, device="cuda").bfloat16().requires_grad_(True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 30, 45], dtype=torch.int32, device="cuda")  # past the end: reported by either pass
    out = dv.packed_attention(q, k, v, starts, status=status)
    assert int(status) == dv.STATUS_BAD_LENGTH
    status.zero_()
    loss = dv.linear_cross_entropy(out.flatten(1), w, torch.arange(40, dtype=torch.int32, device="cuda"), status=status)
    assert int(status) == 0
    status.zero_()
    loss.sum().backward()
    assert int(status) == dv.STATUS_BAD_LENGTH and all(t.grad.isfinite().all() for t in (q, k, v, w))


def test_inputs_are_freed_after_the_backward_pass(ex):
    """A result that is kept keeps no inputs, once the backward pass is done; retained graphs go back twice."""
    dv, g = ex.dv, torch.Generator(device="cuda")
    g.manual_seed(5)
    leaf = torch.randn((40, 4, 64), generator=g, device="cuda").bfloat16().requires_grad_(True)
    starts = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    calls = {"norm": lambda x: dv.norm_rotate(x)[0], "attention": lambda x: dv.packed_attention(x, x, x, starts),
             "attention of strided heads": lambda x: dv.packed_attention(x[:, :2], x[:, 2:].expand(40, 2, 64), x[:, 2:], starts),
             "entropy": lambda x: dv.linear_cross_entropy(x.flatten(1), x.flatten(1), starts[:1].expand(40).contiguous())}
    for name, call in calls.items():
        x = leaf * 2
        out = call(x)
        gone = weakref.ref(x)
        a, = torch.autograd.grad(out.float().sum(), leaf, retain_graph=True)
        b, = torch.autograd.grad(out.float().sum(), leaf)
        del x
        assert gone() is None and torch.equal(a, b) and a.any(), name


@pytest.mark.parametrize("way", ["checkpoint", "offload"])
def test_tensors_that_autograd_keeps_elsewhere(ex, way):
    """Checkpointing computes the saved tensors again, offloading brings copies back: the gradients follow them, not the
    places of the forward pass."""
    from torch.utils.checkpoint import checkpoint

    dv, g = ex.dv, torch.Generator(device="cuda")
    g.manual_seed(6)
    leaf = torch.randn((40, 6, 64), generator=g, device="cuda").bfloat16().requires_grad_(True)
    base = torch.rand(64, generator=g, device="cuda") + 0.5
    phases = dv.rope_phases(1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64), "cuda")

    def net(x):
        x = x * 2  # what follows is the checkpoint's own
        pos = torch.arange(40, dtype=torch.int32, device="cuda") * 3
        q, k = dv.norm_rotate(x[:, :2], x[:, 2:4], base * 1.5, base * 0.5, pos, phases=phases)
        out = dv.packed_attention(q, k, x[:, 4:] * 1, torch.tensor([0, 25, 40], device="cuda", dtype=torch.int32))
        labels = torch.arange(40, device="cuda", dtype=torch.int32) % 30
        return dv.linear_cross_entropy(out.flatten(1), x.flatten(1)[:30, :128], labels, row_weight=base[:40] * 2)

    want, = torch.autograd.grad(net(leaf).sum(), leaf)
    if way == "checkpoint":
        loss = checkpoint(net, leaf, use_reentrant=False)
    else:
        with torch.autograd.graph.save_on_cpu():
            loss = net(leaf)
    junk = [torch.full((40, 6, 64), 1e4, device="cuda", dtype=torch.bfloat16) for _ in range(20)]  # where they lay
    got, = torch.autograd.grad(loss.sum(), leaf)
    assert torch.equal(got, want) and want.any() and len(junk) == 20
