"""The training operators at their limits: arrays whose places pass 32 bits, the largest
batch and count of heads, calls at once on several streams."""
import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402
from test_gpu_packed import BF, DEV, check, dv, inputs, starts  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def filled(shape, block):
    """A large array that repeats a small one along its first dimension."""
    x = torch.empty(shape, device=DEV, dtype=block.dtype)
    x.view(-1, *block.shape).copy_(block.expand(shape[0] // block.shape[0], *block.shape))
    return x


def test_attention_of_many_rows(dv):  # noqa: F811
    """2^19 tokens of 40 heads of 128, 2.7e9 values: sequences that repeat give results that repeat, the first's and the
    last's by the definition."""
    n, S, Hq, Hk, D = 1024, 512, 40, 2, 128
    q, k, v, do = inputs(1, n, n, Hq, Hk, D, BF)
    big = [filled((n * S, *t.shape[1:]), t) for t in (q, k, v)]
    up = filled((n * S, Hq, D), do)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    leaves = [t.requires_grad_(True) for t in big]
    out, lse = dv.packed_attention(*leaves, starts([n] * S), return_lse=True, status=status)
    grads = torch.autograd.grad(out, leaves, up)
    assert int(status) == 0 and out.numel() > 1 << 31
    first = [t.detach()[:n] for t in (out, lse, *grads)]
    check(first[0], first[1], first[2:], q, k, v, do, [n], [n], D ** -0.5, True)
    for t, f in zip((out.detach(), lse, *grads), first):
        for s in range(0, S, 64):
            part = t[s * n:(s + 64) * n].view(64, *f.shape)
            assert torch.equal(part, f.expand(part.shape))


def test_norms_of_many_rows(dv):  # noqa: F811
    n, S, Hq, Hk, D = 1024, 512, 40, 8, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    q, k, uq, uk = (torch.randn((n, h, D), generator=g, device=DEV).to(BF) for h in (Hq, Hk, Hq, Hk))
    w = [torch.rand(D, generator=g, device=DEV) + 0.5 for _ in range(2)]
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    phases = dv.rope_phases(1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D), DEV)

    def run(q, k, uq, uk, pos):
        leaves = [t.detach().requires_grad_(True) for t in (q, k)]
        out = dv.norm_rotate(*leaves, *w, positions=pos, phases=phases)
        return [t.detach() for t in out] + list(torch.autograd.grad(out, leaves, [uq, uk]))

    want = run(q, k, uq, uk, pos)
    got = run(*(filled((n * S, *t.shape[1:]), t) for t in (q, k, uq, uk)), pos.repeat(S))
    assert got[0].numel() > 1 << 31
    for t, f in zip(got, want):
        for s in range(0, S, 64):
            part = t[s * n:(s + 64) * n].view(64, *f.shape)
            assert torch.equal(part, f.expand(part.shape))


def test_a_projection_of_many_values(dv):  # noqa: F811
    """600001 entries of 4096, 2.5e9 values: losses and dh by the definition, dW at both ends and at the labels."""
    N, V, K, run = 40, 600001, 4096, 50000
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    w = torch.empty((V, K), device=DEV, dtype=BF)
    for v in range(0, V, run):
        w[v:v + run] = torch.randn((min(run, V - v), K), generator=g, device=DEV) * (K ** -0.5)
    h = torch.randn((N, K), generator=g, device=DEV).to(BF)
    labels = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    labels[:4] = torch.tensor([0, V - 1, V - 2, 1 << 19], device=DEV)
    x, y = h.clone().requires_grad_(True), w.requires_grad_(True)
    up = torch.rand(N, generator=g, device=DEV) + 0.5
    loss = dv.linear_cross_entropy(x, y, labels)
    dh, dw = torch.autograd.grad(loss, (x, y), up)
    with torch.no_grad():
        few = dv.linear_cross_entropy(h[:20], w, labels[:20])
    w = w.detach()
    assert w.numel() > 1 << 31
    h64, u, ids = h.double(), refs.U[BF], labels.long()
    z = torch.cat([h64 @ w[v:v + run].double().t() for v in range(0, V, run)], 1)
    far = 2 * K * 2.0 ** -23 * (h64.abs() @ w.abs().amax(0).double())[:, None]  # (no row of W is larger anywhere)
    lse = torch.logsumexp(z, 1)
    want = lse - z.gather(1, ids[:, None])[:, 0]
    bound = far[:, 0] + 2.0 ** -18 + 8 * refs.F32 * want.abs()
    assert ((loss.double() - want).abs() <= bound).all() and ((few.double() - want[:20]).abs() <= bound[:20]).all()
    p = torch.exp(z - lse[:, None])
    gr = p.clone()
    gr[torch.arange(N), ids] -= 1.0
    eg = (p * (far + 2.0 ** -18) + gr.abs() * (u + 4 * refs.F32)) * up.double()[:, None]
    gr *= up.double()[:, None]
    wdh, edh = 0.0, 0.0
    for v in range(0, V, run):
        part = w[v:v + run].double()
        wdh = wdh + gr[:, v:v + run] @ part
        edh = edh + (eg[:, v:v + run] + gr[:, v:v + run].abs() * V * 2.0 ** -23) @ part.abs()
    assert ((dh.double() - wdh).abs() <= refs.rounded(wdh, edh, BF)).all()
    for rows in (torch.arange(300, device=DEV), torch.arange(V - 300, V, device=DEV), ids, ids.clamp(1) - 1):
        wdw = gr[:, rows].t() @ h64
        edw = (eg[:, rows] + gr[:, rows].abs() * N * 2.0 ** -23).t() @ h64.abs()
        assert ((dw[rows].double() - wdw).abs() <= refs.rounded(wdw, edw, BF)).all()


@pytest.mark.parametrize("S,most,Hq,Hk,D", [(2048, 3, 4, 2, 64), (2048, 40, 2, 1, 128), (5, 60, 1024, 8, 64),
                                            (3, 50, 1024, 1024, 128)])
def test_the_largest_batch_and_the_most_heads(dv, S, most, Hq, Hk, D):  # noqa: F811
    g = torch.Generator().manual_seed(S + D)
    cq = torch.randint(0, most + 1, (S,), generator=g).tolist()
    q, k, v, do = inputs(S, sum(cq), sum(cq), Hq, Hk, D, BF)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    leaves = [t.requires_grad_(True) for t in (q, k, v)]
    out, lse = dv.packed_attention(*leaves, starts(cq), return_lse=True, status=status)
    grads = torch.autograd.grad(out, leaves, do)
    check(out.detach(), lse, grads, q, k, v, do, cq, cq, D ** -0.5, True)
    assert int(status) == 0


def test_at_once_on_several_streams(dv):  # noqa: F811
    """Steps of all three operators side by side: the bits of each alone."""
    cq = [700, 33, 1200]
    q, k, v, do = inputs(4, sum(cq), sum(cq), 8, 2, 128, BF)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    h, w = torch.randn((700, 512), generator=g, device=DEV).to(BF), torch.randn((9001, 512), generator=g, device=DEV).to(BF)
    labels = torch.arange(700, device=DEV, dtype=torch.int32) * 11
    s, one = starts(cq), torch.rand(128, generator=g, device=DEV)

    def attend():
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v)]
        out = dv.packed_attention(*leaves, s)
        return [out.detach(), *torch.autograd.grad(out, leaves, do)]

    def norm():
        leaves = [t.detach().requires_grad_(True) for t in (q, one)]
        out, _ = dv.norm_rotate(leaves[0], None, leaves[1])
        return [out.detach(), *torch.autograd.grad(out, leaves, do)]

    def entropy():
        leaves = [t.detach().requires_grad_(True) for t in (h, w)]
        loss = dv.linear_cross_entropy(*leaves, labels)
        return [loss.detach(), *torch.autograd.grad(loss.sum(), leaves)]

    calls = [attend, entropy, norm, attend]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in calls], [[] for _ in calls]
    for _ in range(4):
        for stream, call, into in zip(streams, calls, got):
            with torch.cuda.stream(stream):
                into.append(call())
    torch.cuda.synchronize()
    for a, runs in zip(want, got):
        for b in runs:
            assert all(torch.equal(x, y) for x, y in zip(a, b))
