"""linear_cross_entropy's weight gradients where rows of one label repeat: what is left of
the roundings of the label's entry, against the 64-bit definition."""
import math

import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
KEPT = 4  # rows of a label whose entries are not rounded


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


def between(got, want, err):
    """got is some value within `err` of want, rounded to its type (rounding keeps order)."""
    return ((got >= (want - err).to(got.dtype)) & (got <= (want + err).to(got.dtype))).all()


@pytest.mark.parametrize("n", [1, 2, 4, 5, 8, 100, 600])
@pytest.mark.parametrize("spread", [False, True])
def test_rows_that_repeat(dv, n, spread):
    """n equal rows of one label, side by side or among other rows: the label's entry of each beyond the first four is
    rounded, the same way, by half a step at most."""
    V, K, label, others = 700, 64, 389, 60
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    w = (torch.randn((V, K), generator=g, device=DEV) * 2.0 ** -8).to(BF)
    w[label] *= 2.0 ** 6
    h = (torch.randn((others + n, K), generator=g, device=DEV) * 2.0 ** -4).to(BF)
    labels = torch.arange(others + n, device=DEV, dtype=torch.int32) % label  # (never the label itself)
    up = torch.rand(others + n, generator=g, device=DEV) / (others + n) + 1e-3
    rows = torch.arange(n, device=DEV) * (others // n if spread and n <= others else 1)
    h[rows], labels[rows], up[rows] = h[rows[0]].clone(), label, up[rows[0]].clone()
    x, y = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    dw, = torch.autograd.grad(dv.linear_cross_entropy(x, y, labels), [y], up)
    u, N = refs.U[BF], others + n
    r = refs.entropy64(h.double(), w.double(), labels, torch.ones(N, device=DEV).double(), up.double(), u)
    entry = (torch.softmax(h[rows[0]].double() @ w.double().t(), 0)[label] - 1.0) * up[rows[0]].double()
    err = r[5].clone()
    err[label] -= u * min(n, KEPT) * entry.abs() * h[rows[0]].double().abs()
    assert (err > 0).all() and between(dw[label], r[4][label], err[label])
    assert ((dw.double() - r[4]).abs() <= refs.rounded(r[4], r[5], BF)).all()
    if n == 1 or n > KEPT:
        return
    # the bound has its worth: with every entry rounded it would not hold
    step = math.ulp(float(entry)) * 2.0 ** 45 / 2  # half a step of bf16 at the entry (its 8 bits of 53)
    assert float(err[label].max() / h[rows[0]].double().abs().max() / n) < step
