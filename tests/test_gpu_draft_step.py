"""The operators together, as a serving loop uses them (examples/draft_step.py)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    import draft_step

    return draft_step


def test_the_loop_runs_and_updates_lower_the_loss(step):
    report = step.run(requests=4, steps=5)
    assert all(0 <= after < loss < 100 and 1 <= n <= 8 for loss, after, n in report)
    assert report == step.run(requests=4, steps=5)


def test_a_block_attends_like_plain_softmax_attention(step):
    """The layer's output for a block behind a prompt against the same layer in
    plain torch (fp32 attention over bf16 projections)."""
    B, n, prompt, hq, hk, d = 3, 8, 37, 8, 2, 64
    layer = step.Layer(B, hq, hk, d, 64, page=16, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((B, prompt + n, hq * d), generator=g, device="cuda").to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.forward(x[:, :prompt], st)
    layer.lens += prompt
    got = layer.forward(x[:, prompt:], st)
    assert int(st) == 0
    qkv = (x.view(-1, hq * d) @ layer.wqkv).view(B, prompt + n, hq + 2 * hk, d)
    ang = torch.arange(prompt + n, device="cuda", dtype=torch.float64)[:, None] \
        * 1e6 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    c, s = ang.cos().float()[None, :, None], ang.sin().float()[None, :, None]

    def turn(v):
        a, b = v.float().chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16).float()

    q, k, v = turn(qkv[:, :, :hq]), turn(qkv[:, :, hq:hq + hk]), qkv[:, :, hq + hk:].float()
    k, v = (t.repeat_interleave(hq // hk, 2) for t in (k, v))
    w = torch.einsum("bqhd,bkhd->bhqk", q[:, prompt:], k) * d ** -0.5
    i = torch.arange(n, device="cuda")[:, None] + prompt
    w = w.masked_fill(torch.arange(prompt + n, device="cuda")[None] > i, -torch.inf).softmax(-1)
    y = torch.einsum("bhqk,bkhd->bqhd", w, v).reshape(B * n, hq * d).to(torch.bfloat16)
    want = x[:, prompt:] + (y @ layer.wo).view(B, n, -1)
    # the attention's output is rounded twice (weights, result), then projected:
    # each a bf16 half step of values of size about 1
    assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -8 * 8 * float(want.float().abs().max())
