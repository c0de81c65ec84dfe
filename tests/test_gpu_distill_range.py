"""The distillation's logits at the ends of their types' range, and infinite ones
wherever they stand in a row."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


def make(seed, N, V, K, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = (torch.randn((N, V), generator=g, device=DEV) * 2).to(dtype)
    ids = torch.rand((N, V), generator=g, device=DEV).topk(K, dim=1).indices.to(torch.int32)
    return z, ids, torch.randn((N, K), generator=g, device=DEV) * 2


def both(dv, z, ids, t, T=1.0):
    """(loss, gradient, status) of the one call and of autograd's two."""
    out = []
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, grad = dv.distill_loss_grad(z, ids, t, T, status=st)
    out.append((loss, grad, int(st)))
    st.zero_()
    a = z.clone().requires_grad_(True)
    loss = dv.distill_loss(a, ids, t, T, status=st)
    loss.backward(torch.ones_like(loss))
    out.append((loss.detach(), a.grad, int(st)))
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [5, 999, 5003, 100003])
def test_infinite_logits_anywhere_in_a_row(dv, dtype, V):
    """The row's unaligned ends, its body and the borders of its slices: a
    largest logit of +inf gives NaN and the status bit."""
    for at in sorted({0, 1, 2, 3, 4, V // 2, V // 2 + 1, V - 3, V - 2, V - 1} & set(range(V))):
        z, ids, t = make(V, 3, V, 3, dtype)
        want = dv.distill_loss_grad(z, ids, t)
        z[1, at] = math.inf
        for loss, grad, st in both(dv, z, ids, t):
            assert st == dv.STATUS_BAD_ROW, (at, st)
            assert bool(loss[1].isnan()) and bool(grad[1].isnan().any()), (at, loss)
            assert torch.equal(loss[0], want[0][0]) and torch.equal(loss[2], want[0][2])
            assert bool(grad[::2].isfinite().all())
