"""linear_cross_entropy's gradients where the logits' gradients take several pieces of
the vocabulary, with bounds that zeros, a wrong piece or a wrong sign do not meet."""
import math

import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


def inputs(seed, N, V, K, borders, device):
    """Rows that share a direction, so that sums over rows grow with their number; labels at the pieces' borders, for
    one row and for several; rows that take no part."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    common = torch.where(torch.rand(K, generator=g, device=device) < 0.5, -2.0, 2.0)
    h = (torch.randn((N, K), generator=g, device=device) * 0.5 + common).to(BF)
    w = (torch.randn((V, K), generator=g, device=device) * (0.5 / math.sqrt(K))).to(BF)
    labels = torch.randint(0, V // 37, (N,), generator=g, device=device, dtype=torch.int32) * 37  # (few of them)
    at = torch.tensor([v + d for v in borders for d in (-1, 0, 31)] + [0, V - 1], device=device, dtype=torch.int32)
    at = at.clamp(max=V - 1)
    labels[:len(at)] = at
    labels[N - 7 * len(at):] = at.repeat(7)
    labels[100::997] = -1
    weight = torch.rand(N, generator=g, device=device) + 0.5
    weight[200::991] = 0.0
    up = (torch.rand(N, generator=g, device=device) + 0.5) / N
    return h, w, labels, weight, up


def definition(h, w, labels, weight, up, at_once):
    """refs.entropy64 over runs of rows: its losses and dh with their bounds, dW and its bound over all rows."""
    N = h.shape[0]
    w64 = w.double()
    parts, dw, edw = [], 0.0, 0.0
    for r0 in range(0, N, at_once):
        s = slice(r0, min(N, r0 + at_once))
        a = h[s].double(), w64, labels[s], weight[s].double(), up[s].double()
        r = refs.entropy64(*a, refs.U[BF])
        n = a[0].shape[0]
        # the rest of the sum's length: entropy64 counts this run's n rows
        used = (labels[s] >= 0) & (weight[s] != 0)
        g = torch.softmax(a[0] @ w64.t(), 1)
        g[torch.arange(n), labels[s].long().clamp(min=0)] -= 1.0
        g *= torch.where(used, a[3] * a[4], 0.0)[:, None]
        dw = dw + r[4]
        edw = edw + r[5] + (g.abs().t() @ a[0].abs()) * (N - n) * 2.0 ** -23
        parts.append(r[:4])
    return [torch.cat(t) for t in zip(*parts)] + [dw, edw]


@pytest.mark.parametrize("N,V,K,piece", [(17000, 15616 + 4001, 64, 15616), (70001, 2 * 4096 + 33, 72, 4096)])
def test_pieces_of_distinct_rows(dv, N, V, K, piece):
    """A narrow last piece, labels on both sides of the borders, and (70001 rows) several runs of the statistics."""
    borders = list(range(piece, V, piece))
    h, w, labels, weight, up = inputs(N, N, V, K, borders, DEV)
    word = torch.zeros(1, device=DEV, dtype=torch.int32)
    x, y = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = dv.linear_cross_entropy(x, y, labels, row_weight=weight, status=word)
    dh, dw = torch.autograd.grad(loss, (x, y), up)
    want, e, wdh, edh, wdw, edw = definition(h, w, labels, weight, up, 4000)
    assert ((loss.double() - want).abs() <= e).all() and int(word) == 0
    assert ((dh.double() - wdh).abs() <= refs.rounded(wdh, edh, BF)).all()
    bound = refs.rounded(wdw, edw, BF)
    # what the bound is worth: nearly all entries, of every piece, lie far outside it
    for lo in [0] + borders:
        assert (8 * bound < wdw.abs())[lo:lo + piece].float().mean() > 0.97
    assert ((dw.double() - wdw).abs() <= bound).all()
