"""packed_attention where every processor takes several units of work in turn, in the
forward kernel and in both gradients' kernels."""
import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402
from test_gpu_packed import BF, DEV, HF, check, dv, inputs, starts  # noqa: E402,F401

pytestmark = pytest.mark.gpu
SMS = 152


def counts(seed, n, most, empty):
    """Lengths between 1 and `most`, some of them 0."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(1, most + 1, (n,), generator=g)
    c[torch.randperm(n, generator=g)[:empty]] = 0
    return c.tolist()


def units(cs, rows, heads):
    return sum(-(-c // rows) for c in cs) * heads


CASES = [
    # sequences, most queries, most keys (None: the same), without queries, without keys, q heads, kv heads, head_dim, causal
    (64, 300, None, 5, 0, 8, 8, 128, True), (64, 300, None, 5, 0, 16, 8, 64, True), (48, 200, 330, 6, 6, 16, 8, 128, True),
    (60, 330, 200, 6, 6, 16, 8, 64, True), (40, 260, 390, 4, 4, 12, 12, 128, False), (60, 140, 400, 3, 7, 24, 8, 64, False),
]


@pytest.mark.parametrize("S,mq,mk,eq,ek,Hq,Hk,D,causal", CASES)
def test_gradients(dv, S, mq, mk, eq, ek, Hq, Hk, D, causal):  # noqa: F811
    """Three rounds and more of units for each processor, among them units that see nothing."""
    cq = counts(S + D, S, mq, eq)
    ck = cq if mk is None else counts(S + D + 1, S, mk, ek)
    assert units(ck, 128, Hk) > 3 * SMS and units(cq, 128, Hq) > 3 * SMS and units(cq, 256, Hq) > 2 * SMS
    q, k, v, do = inputs(S + mq, sum(cq), sum(ck), Hq, Hk, D, BF)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    for t in (q, k, v):
        t.requires_grad_(True)
    args = dict(kv_start=None if mk is None else starts(ck), causal=causal, status=status)
    out, lse = dv.packed_attention(q, k, v, starts(cq), return_lse=True, **args)
    grads = torch.autograd.grad(out, (q, k, v), do)
    check(out.detach(), lse, grads, q, k, v, do, cq, ck, D ** -0.5, causal)
    again, lse2 = dv.packed_attention(q, k, v, starts(cq), return_lse=True, **args)
    both = torch.autograd.grad(again, (q, k, v), do)
    assert torch.equal(again, out) and torch.equal(lse2, lse) and all(torch.equal(a, b) for a, b in zip(grads, both))
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
def test_values(dv, D, dtype):  # noqa: F811
    """The forward kernel without what it keeps for gradients, units of several tiles of keys."""
    cq = counts(D, 24, 900, 2)
    assert units(cq, 256, 12) > 3 * SMS
    q, k, v, do = inputs(D, sum(cq), sum(cq), 12, 4, D, dtype)
    out, lse = dv.packed_attention(q, k, v, starts(cq), return_lse=True)
    check(out, lse, None, q, k, v, do, cq, cq, D ** -0.5, True)


def test_one_sequence_of_many_units(dv):  # noqa: F811
    """Units of one long sequence, of very different work."""
    n, Hq, Hk, D = 8200, 8, 8, 64
    q, k, v, do = inputs(1, n, n, Hq, Hk, D, BF)
    assert units([n], 128, Hk) > 3 * SMS
    for t in (q, k, v):
        t.requires_grad_(True)
    out, lse = dv.packed_attention(q, k, v, starts([n]), return_lse=True)
    grads = torch.autograd.grad(out, (q, k, v), do)
    for h in range(0, Hq, 3):  # (some of the heads: each is a definition of 8200 x 8200 in 64 bits)
        s = slice(h, h + 1)
        check(out.detach()[:, s], lse[:, s], [g[:, s] for g in grads], q[:, s], k[:, s], v[:, s], do[:, s], [n], [n],
              D ** -0.5, True)
