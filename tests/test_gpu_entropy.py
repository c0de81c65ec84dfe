"""linear_cross_entropy against the definition in 64 bits: odd sizes, labels that
take no part, strides, pieces of the vocabulary, values that are not finite,
gradients, captured calls."""
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


def inputs(seed, N, V, K, spread=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    w = (torch.randn((V, K), generator=g, device=DEV) * (spread / math.sqrt(K))).to(BF)
    labels = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    pull = torch.rand((N, 1), generator=g, device=DEV) * 2
    h = (torch.randn((N, K), generator=g, device=DEV) + pull * w[labels.long()].float()).to(BF)
    weight = torch.rand(N, generator=g, device=DEV) + 0.1
    up = torch.randn(N, generator=g, device=DEV) / N
    return h, w, labels, weight, up


def check(dv, h, w, labels, weight=None, up=None, status=0):
    N = h.shape[0]
    word = torch.zeros(1, device=DEV, dtype=torch.int32)
    h, w = (t.detach().requires_grad_(True) for t in (h, w))
    loss = dv.linear_cross_entropy(h, w, labels, row_weight=weight, status=word)
    up = torch.ones(N, device=DEV) if up is None else up
    dh, dw = torch.autograd.grad(loss, (h, w), up)
    one = torch.ones(N, device=DEV) if weight is None else weight
    r = refs.entropy64(h.detach().double(), w.detach().double(), labels, one.double(), up.double(), refs.U[BF])
    assert ((loss.double() - r[0]).abs() <= r[1]).all()
    assert ((dh.double() - r[2]).abs() <= refs.rounded(r[2], r[3], BF)).all()
    assert ((dw.double() - r[4]).abs() <= refs.rounded(r[4], r[5], BF)).all()
    assert int(word) == status
    with torch.no_grad():
        assert torch.equal(dv.linear_cross_entropy(h, w, labels, row_weight=weight), loss)
    return loss, dh, dw


@pytest.mark.parametrize("N,V,K", [(1, 1, 8), (1, 2, 64), (3, 255, 72), (128, 256, 64), (129, 257, 128), (255, 1000, 200),
                                   (257, 513, 64), (300, 4099, 328), (7, 20000, 512), (513, 777, 1024), (1, 5000, 2056),
                                   (600, 300, 5120)])
@pytest.mark.parametrize("weighted", [False, True])
def test_sizes(dv, N, V, K, weighted):
    h, w, labels, weight, up = inputs(N + V + K, N, V, K)
    check(dv, h, w, labels, weight if weighted else None, up if weighted else None)


def test_labels_that_take_no_part(dv):
    h, w, labels, weight, up = inputs(1, 300, 1000, 128)
    labels[::3] = -1
    weight[1::7] = 0.0
    up[2::11] = 0.0
    _, dh, _ = check(dv, h, w, labels, weight, up)
    assert not dh[::3].any() and not dh[1::7].any() and not dh[2::11].any()
    labels[5], labels[100], labels[299] = 1000, -2, 2 ** 31 - 1
    loss, dh, _ = check(dv, h, w, labels, weight, up, status=1)
    assert not loss[[5, 100, 299]].any() and not dh[[5, 100, 299]].any()
    labels[:] = -1
    loss, dh, dw = check(dv, h, w, labels, weight, up)
    assert not loss.any() and not dh.any() and not dw.any()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_that_take_no_part_hold_anything(dv, bad):
    h, w, labels, weight, up = inputs(2, 200, 600, 64)
    rows = torch.arange(5, 200, 9, device=DEV)
    labels[rows] = -1
    a = check(dv, h, w, labels, weight, up)
    h[rows] = bad
    word = torch.zeros(1, device=DEV, dtype=torch.int32)
    x, y = (t.detach().requires_grad_(True) for t in (h, w))
    loss = dv.linear_cross_entropy(x, y, labels, row_weight=weight, status=word)
    b = (loss, *torch.autograd.grad(loss, (x, y), up))
    assert all(torch.equal(s, t) for s, t in zip(a, b)) and int(word) == 0


def test_rows_that_are_not_sound(dv):
    h, w, labels, _, up = inputs(3, 140, 500, 64)
    clean = dv.linear_cross_entropy(h, w, labels)
    h[7, 3], h[130, 0] = math.nan, math.inf
    word = torch.zeros(1, device=DEV, dtype=torch.int32)
    loss = dv.linear_cross_entropy(h, w, labels, status=word)
    keep = torch.ones(140, device=DEV, dtype=torch.bool)
    keep[[7, 130]] = False
    assert torch.equal(loss[keep], clean[keep]) and loss[~keep].isnan().all() and int(word) == 2


def test_logits_of_any_size(dv):
    """Large logits of both signs: the loss and its gradient follow their differences."""
    h, w, labels, weight, up = inputs(4, 64, 300, 64)
    big = torch.zeros((64, 8), device=DEV, dtype=BF)
    big[:, 0] = 2.0 ** torch.arange(-20, 44, device=DEV).float()
    wb = torch.zeros((300, 8), device=DEV, dtype=BF)
    wb[:, 0] = (torch.arange(300, device=DEV) % 16 - 8).to(BF)
    check(dv, big, wb, labels, weight, up)


def test_strides(dv):
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    h = torch.randn((90, 200), generator=g, device=DEV).to(BF)[:, 64:128]
    w = torch.randn((333, 128), generator=g, device=DEV).to(BF)[:, 8:72]
    labels = torch.randint(0, 333, (90,), generator=g, device=DEV, dtype=torch.int32)
    a = check(dv, h, w, labels)
    b = check(dv, h.contiguous(), w.contiguous(), labels)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # an upstream gradient that all rows share
    x, y = (t.detach().requires_grad_(True) for t in (h, w))
    c = torch.autograd.grad(dv.linear_cross_entropy(x, y, labels).sum(), (x, y))
    assert torch.equal(c[0], a[1]) and torch.equal(c[1], a[2])


@pytest.mark.parametrize("N", [1, 5, 64, 65, 600])
def test_the_label_s_entry_is_not_rounded(dv, N):
    """A label's entry of the logits' gradients rules its row of both gradients: there the bound is that of the
    definition without the half step of bf16 of this entry."""
    V, K = 600, 64
    h, w, _, weight, up = inputs(9, N, V, K)
    labels = torch.arange(N, device=DEV, dtype=torch.int32) * 389 % V  # (no label twice)
    w *= 2.0 ** -6
    w[labels.long()] *= 2.0 ** 6
    h *= 2.0 ** -4
    x, y = (t.detach().requires_grad_(True) for t in (h, w))
    loss = dv.linear_cross_entropy(x, y, labels, row_weight=weight)
    dh, dw = torch.autograd.grad(loss, (x, y), up)
    u, ids = refs.U[BF], labels.long()
    r = refs.entropy64(h.double(), w.double(), labels, weight.double(), up.double(), u)
    entry = (torch.softmax(h.double() @ w.double().t(), 1)[torch.arange(N), ids] - 1.0) * weight * up
    edh = r[3] - u * entry.abs()[:, None] * w[ids].double().abs()
    edw = r[5].clone()
    edw[ids] -= u * entry.abs()[:, None] * h.double().abs()
    assert ((dh.double() - r[2]).abs() <= refs.rounded(r[2], edh, BF)).all()
    assert ((dw.double() - r[4]).abs() <= refs.rounded(r[4], edw, BF)).all()


def test_many_rows_of_few_labels(dv):
    """One label, and two beside each other, for hundreds of rows."""
    h, w, labels, weight, up = inputs(10, 700, 300, 72)
    for ids in (torch.full((700,), 299, device=DEV, dtype=torch.int32), 31 + labels % 2):
        check(dv, h, w, ids.to(torch.int32), weight, up)


@pytest.mark.parametrize("N,V,K", [(1, 40000, 72), (31, 4095, 2056), (32, 40001, 1024), (32, 1, 8), (33, 40001, 1032)])
def test_few_rows(dv, N, V, K):
    """Few rows, vocabularies of more tiles than there are pairs of processors, several chunks of the inner index."""
    h, w, labels, weight, up = inputs(N + V + K, N, V, K)
    labels[0], labels[-1] = 0, V - 1
    check(dv, h, w, labels, weight, up)


def test_one_gradient_alone(dv):
    h, w, labels, weight, up = inputs(6, 300, 3000, 256)
    _, dh, dw = check(dv, h, w, labels, weight, up)
    for i, want in ((0, dh), (1, dw)):
        a = [h.detach(), w.detach()]
        a[i] = a[i].requires_grad_(True)
        got, = torch.autograd.grad(dv.linear_cross_entropy(*a, labels, row_weight=weight), [a[i]], up)
        assert torch.equal(got, want)


def test_no_rows(dv):
    h = torch.zeros((0, 64), device=DEV, dtype=BF, requires_grad=True)
    w = torch.ones((10, 64), device=DEV, dtype=BF, requires_grad=True)
    loss = dv.linear_cross_entropy(h, w, torch.zeros(0, device=DEV, dtype=torch.int32))
    dh, dw = torch.autograd.grad(loss, (h, w), torch.zeros(0, device=DEV))
    assert loss.shape == (0,) and dh.shape == (0, 64) and not dw.any()


def test_many_rows_and_pieces(dv):
    """More rows than the statistics are held for at a time (rows repeat, so one definition serves), and more
    of the logits' gradients than one piece holds."""
    N, V, K = 17000, 20000, 64
    h, w, labels, _, _ = inputs(7, 100, V, K)
    many, ids = h.repeat(N // 100, 1), labels.repeat(N // 100)
    up = torch.full((N,), 1.0 / N, device=DEV)
    x, y = many.requires_grad_(True), w.detach().requires_grad_(True)
    loss = dv.linear_cross_entropy(x, y, ids)
    dh, dw = torch.autograd.grad(loss, (x, y), up)
    r = refs.entropy64(h.double(), w.double(), labels, torch.ones(100, device=DEV).double(), up[:100].double(), refs.U[BF])
    assert ((loss.view(-1, 100).double() - r[0]).abs() <= r[1]).all()
    assert ((dh.view(-1, 100, K).double() - r[2]).abs() <= refs.rounded(r[2], r[3], BF)).all()
    n = N // 100
    assert ((dw.double() - n * r[4]).abs() <= refs.rounded(n * r[4], n * n * r[5], BF)).all()


def test_repeats_and_captured(dv):
    h, w, labels, weight, up = inputs(8, 500, 9000, 512)
    x, y = h.detach().clone().requires_grad_(True), w.detach().clone().requires_grad_(True)

    def step():
        loss = dv.linear_cross_entropy(x, y, labels, row_weight=weight)
        return [loss.detach(), *torch.autograd.grad(loss, (x, y), up)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = step(), step()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        x.mul_(0.5)
        labels.add_(1).remainder_(9000)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(got, step()))
