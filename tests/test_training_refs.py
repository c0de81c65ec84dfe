"""The definitions that the training operators are held to: their gradients
against differences of the values they belong to (64 bits, CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

STEP = 1e-5  # central differences: an error of about STEP^2 times the third derivative, and 1e-16 / STEP


def differences(f, x, d):
    return (f(x + STEP * d) - f(x - STEP * d)) / (2 * STEP)


def direction(g, shape):
    return torch.randn(shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm(interleaved):
    g = torch.Generator().manual_seed(3)
    x, w, dy = direction(g, (4, 3, 64)), 1 + 0.2 * direction(g, (64,)), direction(g, (4, 3, 64))
    pos, freq = torch.tensor([0, 1, -5, 1000]), 1e4 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    dx, _, dw, _ = refs.norm_grad64(x, w, 1e-6, pos, freq, interleaved, dy)
    for grad, at, f in ((dx, x, lambda t: refs.norm64(t, w, 1e-6, pos, freq, interleaved)[0]),
                        (dw, w, lambda t: refs.norm64(x, t, 1e-6, pos, freq, interleaved)[0])):
        d = direction(g, at.shape)
        assert math.isclose((differences(f, at, d) * dy).sum(), (grad * d).sum(), rel_tol=1e-7, abs_tol=1e-7)


@pytest.mark.parametrize("n,m,causal", [(5, 5, True), (7, 3, True), (3, 9, True), (4, 6, False), (1, 1, True)])
def test_attention(n, m, causal):
    g = torch.Generator().manual_seed(4)
    q, k, v, do = (direction(g, s) for s in ((n, 4, 8), (m, 2, 8), (m, 2, 8), (n, 4, 8)))
    mask = refs.sees(n, m, causal)
    grads, _ = refs.attention_grad64(q, k, v, 0.3, mask, do, 0.0)
    for i, grad in enumerate(grads):
        def f(t):
            a = [q, k, v]
            a[i] = t
            return refs.attention64(*a, 0.3, mask, 0.0)[0]

        at = (q, k, v)[i]
        d = direction(g, at.shape)
        assert math.isclose((differences(f, at, d) * do).sum(), (grad * d).sum(), rel_tol=1e-7, abs_tol=1e-8)


def test_entropy():
    g = torch.Generator().manual_seed(5)
    h, w = direction(g, (6, 8)), direction(g, (11, 8))
    labels, weight, up = torch.tensor([0, 10, -1, 3, 3, 99]), torch.rand(6, generator=g).double(), direction(g, (6,))
    weight[4] = 0.0
    _, _, dh, _, dw, _ = refs.entropy64(h, w, labels, weight, up, 0.0)
    assert not dh[2].any() and not dh[4].any() and not dh[5].any()
    for grad, at, f in ((dh, h, lambda t: refs.entropy64(t, w, labels, weight, up, 0.0)[0]),
                        (dw, w, lambda t: refs.entropy64(h, t, labels, weight, up, 0.0)[0])):
        d = direction(g, at.shape)
        assert math.isclose((differences(f, at, d) * up).sum(), (grad * d).sum(), rel_tol=1e-7, abs_tol=1e-8)
