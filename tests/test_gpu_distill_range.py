"""The distillation's logits at the ends of their types' range, and infinite ones
wherever they stand in a row."""
import math

import pytest

torch = pytest.importorskip("torch")
from operator_refs import F32, U, distill64  # noqa: E402

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


LOWEST = {BF: torch.finfo(BF).min, FP: torch.finfo(FP).min}


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [7, 1000, 5003, 100003])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_rows_at_the_range_s_ends(dv, dtype, V, T):
    """Finite logits have a distribution: rows that are nothing but their type's
    lowest (or highest) value, or whose largest one is, and ordinary rows whose
    masked places hold the lowest."""
    z, ids, t = make(V, 5, V, 4, dtype)
    z[0] = LOWEST[dtype]
    z[1] = -LOWEST[dtype]
    z[2, V // 2:] = LOWEST[dtype]
    z[3] = LOWEST[dtype]
    z[3, 1] = -LOWEST[dtype]
    z[3, ids[3, 0].long()] = -LOWEST[dtype]
    ids[2] = torch.arange(4, device=DEV) % (V // 2)  # no teacher token where the student rules it out
    ids[3] = ids[3, 0]
    z[4, 0] = -LOWEST[dtype] / 2
    ids[4] = 0
    want, wg = distill64(z, ids, t, T)
    p = torch.softmax(t.double() / T, 1)
    for loss, grad, st in both(dv, z, ids, t, T):
        assert st == 0
        # differences of logits of a row's size are exact here; the rest as for ordinary logits
        tol = (math.log(V) + 40) * 8 * F32 + (V / 512 + 300) * F32 + 2.0 ** -20
        assert bool(((loss.double() - want).abs() <= tol).all()), (loss, want)
        gt = U[dtype] * wg.abs() + tol / T * (wg.abs() + torch.zeros_like(wg).scatter_add_(1, ids.long(), p) + 2e-6)
        assert bool(((grad.double() - wg).abs() <= gt).all())


def test_row_statistics_of_ordinary_rows(dv):
    """The C call's statistics: log sum e^(z / T) = (R + log2 s) ln 2."""
    import ctypes

    lib = dv.load()
    T = 0.8
    z, ids, t = make(3, 4, 5003, 4, FP)
    z[2] *= 400
    loss, stats = torch.empty(4, device=DEV), torch.empty((4, 2), device=DEV)
    rc = lib.dflash_distill_loss(z.data_ptr(), 5003, 4, 5003, dv.DFLASH_F32,
                                 ids.data_ptr(), t.data_ptr(), 4, ctypes.c_float(T), None, loss.data_ptr(),
                                 stats.data_ptr(), None, None)
    assert rc == 0
    torch.cuda.synchronize()
    got = (stats[:, 0].double() + stats[:, 1].double().log2()) * math.log(2.0)
    want = torch.logsumexp(z.double() / T, 1)
    # the scale 1 / (T ln 2) and the reference are rounded
    assert bool(((got - want).abs() <= want.abs() * 4 * F32 + (5003 / 512 + 300) * F32 + 2.0 ** -20).all())
