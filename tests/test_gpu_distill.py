"""dflash_distill_loss, _grad and _loss_grad against the definition in 64 bits
and against differences of the loss."""
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


def make(seed, N, V, K, dtype, repeat=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = torch.randn((N, V), generator=g, device=DEV) * 2
    if repeat:
        ids = torch.randint(0, max(1, min(V, K // 2)), (N, K), generator=g, device=DEV, dtype=torch.int32)
    else:
        ids = torch.rand((N, V), generator=g, device=DEV).topk(K, dim=1).indices.to(torch.int32)
    t = torch.randn((N, K), generator=g, device=DEV) * 2 + 5
    z.scatter_add_(1, ids.long(), t * 0.7)
    return g, z.to(dtype), ids, t


def check(z, ids, t, T, loss, grad, w=None, up=None, grad_dtype=None):
    want, wg = distill64(z, ids, t, T, w, up)
    V = z.shape[1]
    ww = torch.ones(z.shape[0], device=DEV, dtype=torch.float64) if w is None else w.double().abs()
    # scores and their differences up to `span` in units of 1 / T; sums of V terms by threads
    zf = z.double()
    top = torch.where(zf.isfinite(), zf, torch.zeros_like(zf)).abs().amax(1) / T
    span = 2 * top + t.abs().amax(1).double() / T + math.log(V) + 1
    acc = (V / 512 + 300) * F32 + 2.0 ** -21
    tol = ww * (span * 8 * F32 + acc)
    err = (loss.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float(tol.max()))
    if grad is not None:
        c = (ww if up is None else ww * up.double().abs())[:, None] / T
        tol = U[z.dtype] * wg.abs() + c * (span[:, None] * 8 * F32 + acc) * (wg.abs() / c.clamp_min(1e-300) + 2e-6) \
            + c * torch.zeros_like(wg).scatter_add_(1, ids.long().clamp_min(0), torch.ones_like(t.double())) \
            * (span[:, None] * 8 * F32 + acc) + 1e-37
        err = (grad.double() - wg).abs()
        assert bool((err <= tol).all()), float((err - tol).max())


SHAPES = [(1, 1, 1), (3, 5, 5), (2, 7, 1), (4, 1000, 20), (5, 4097, 32), (2, 8191, 256), (40, 1031, 64),
          (1, 100003, 20), (3, 248320, 32), (400, 257, 3)]


@pytest.mark.parametrize("N,V,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_loss_and_gradient(dv, N, V, K, dtype):
    for T, weighted in ((1.0, False), (0.7, True)):
        g, z, ids, t = make(N * 31 + V + K, N, V, K, dtype)
        w = torch.rand(N, generator=g, device=DEV) * 2 - 0.5 if weighted else None
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        loss, grad = dv.distill_loss_grad(z, ids, t, T, row_weight=w, status=st)
        assert int(st) == 0 and grad.dtype == dtype
        check(z, ids, t, T, loss, grad, w)
        zz = z.clone().requires_grad_(True)
        loss2 = dv.distill_loss(zz, ids, t, T, row_weight=w, status=st)
        up = torch.rand(N, generator=g, device=DEV) * 3 - 1
        loss2.backward(up)
        assert int(st) == 0 and loss2.dtype == FP
        check(z, ids, t, T, loss2.detach(), zz.grad, w, up)


def test_sum_and_mean_backward(dv):
    """A broadcast upstream gradient (stride 0)."""
    g, z, ids, t = make(2, 6, 500, 8, FP)
    for reduce in (torch.sum, torch.mean):
        a = z.clone().requires_grad_(True)
        reduce(dv.distill_loss(a, ids, t)).backward()
        up = torch.full((6,), 1.0 if reduce is torch.sum else 1 / 6, device=DEV)
        check(z, ids, t, 1.0, dv.distill_loss(z, ids, t), a.grad, None, up)


def test_broadcast_student(dv):
    """One row of logits against several teachers: the rows' gradients add up."""
    g, z, ids, t = make(3, 4, 300, 8, FP)
    a = z[:1].clone().requires_grad_(True)
    dv.distill_loss(a.expand(4, 300), ids, t).sum().backward()
    zz = z[:1].expand(4, 300).contiguous()
    _, parts = dv.distill_loss_grad(zz, ids, t)
    want = parts.double().sum(0, keepdim=True)
    assert bool(((a.grad.double() - want).abs() <= 8 * F32 * parts.double().abs().sum(0) + 1e-12).all())


def test_gradient_against_differences(dv):
    """Central differences of the kernel's own loss: truncation h^2 / 6 times
    the third derivative (below 1 / T^3 for a log-sum-exp), and twice the loss's
    rounding over 2 h."""
    N, V, K, T, h = 1, 40, 6, 1.3, 2.0 ** -5
    g, z, ids, t = make(5, N, V, K, FP)
    _, grad = dv.distill_loss_grad(z, ids, t, T)
    zz = z.expand(V, V)
    eye = torch.eye(V, device=DEV) * h
    many = ids.expand(V, K).contiguous(), t.expand(V, K).contiguous()
    d = (dv.distill_loss(zz + eye, *many, T).double() - dv.distill_loss(zz - eye, *many, T).double()) / (2 * h)
    tol = h * h / 6 / T ** 3 + 2 * (40 * 8 * F32 + 2.0 ** -20) / (2 * h)
    assert bool(((grad[0].double() - d).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_repeated_and_empty_entries(dv, dtype):
    g, z, ids, t = make(7, 6, 777, 16, dtype, repeat=True)
    ids[1, ::2] = -1
    ids[2, :] = -1
    ids[3, 1:] = -1
    t[4, 3:9] = -math.inf
    t[5, :] = -math.inf  # no teacher mass at all: like a row without entries
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, grad = dv.distill_loss_grad(z, ids, t, status=st)
    assert int(st) == 0
    tt = torch.where(t == -math.inf, torch.full_like(t, -1e30), t)
    ids2 = ids.clone()
    ids2[5] = -1
    want, wg = distill64(z, ids2, tt, 1.0)
    assert float(loss[2]) == 0 and float(loss[5]) == 0
    assert bool((grad[2] == 0).all()) and bool((grad[5] == 0).all())
    assert bool(((loss.double() - want).abs() <= 60 * 8 * F32 + 2.0 ** -19).all())
    assert bool(((grad.double() - wg).abs() <= U[dtype] * wg.abs() + 2.0 ** -17).all())


def test_rows_without_weight_are_not_read(dv):
    """Weight 0, or no entries: loss and gradient 0 over NaN logits."""
    g, z, ids, t = make(8, 4, 1003, 8, FP)
    z[1] = float("nan")
    z[2] = float("nan")
    ids[2] = -1
    w = torch.tensor([1.0, 0.0, 1.0, 2.0], device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, grad = dv.distill_loss_grad(z, ids, t, row_weight=w, status=st)
    zz = z.clone().requires_grad_(True)
    l2 = dv.distill_loss(zz, ids, t, row_weight=w, status=st)
    up = torch.tensor([1.0, 1.0, 1.0, 0.0], device=DEV)
    l2.backward(up)
    assert int(st) == 0
    assert torch.equal(loss[1:3], torch.zeros(2, device=DEV)) and torch.equal(l2.detach(), loss)
    assert bool((grad[1:3] == 0).all()) and bool((zz.grad[1:] == 0).all())
    ok = torch.tensor([0, 3], device=DEV)
    check(z[ok], ids[ok], t[ok], 1.0, loss[ok], grad[ok], w[ok])


def test_infinite_and_nan_logits(dv):
    g, z, ids, t = make(9, 8, 3001, 8, FP)
    out = torch.arange(3001, device=DEV)
    out = out[~torch.isin(out, ids[0].long())]
    z[0, out[:1500]] = -math.inf          # masked vocabulary: no mass, no gradient
    loss, grad = dv.distill_loss_grad(z[:1], ids[:1], t[:1])
    check(z[:1], ids[:1], t[:1], 1.0, loss, grad)
    assert bool((grad[0, out[:1500]] == 0).all())
    z[1, 5] = math.inf
    z[2, 7] = math.nan
    z[3] = -math.inf
    t[4, 0] = math.nan
    t[5, 0] = math.inf
    z[6, int(ids[6, 0])] = -math.inf      # the student rules out a teacher's token
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for r in range(1, 6):
        st.zero_()
        a = z[r:r + 1].clone().requires_grad_(True)
        loss, grad = dv.distill_loss_grad(z[r:r + 1], ids[r:r + 1], t[r:r + 1], status=st)
        assert bool(loss.isnan().all()) and bool(grad.isnan().any()) and int(st) == dv.STATUS_BAD_ROW
        l2 = dv.distill_loss(a, ids[r:r + 1], t[r:r + 1])
        l2.sum().backward()
        assert bool(l2.isnan().all()) and bool(a.grad.isnan().any())
    st.zero_()
    loss, grad = dv.distill_loss_grad(z[6:7], ids[6:7], t[6:7], status=st)
    assert float(loss) == math.inf and int(st) == 0 and bool(grad.isfinite().all())


def test_ids_outside_the_vocabulary(dv):
    g, z, ids, t = make(10, 2, 64, 4, FP)
    ids[0, 1], ids[1, 2] = 64, -2
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, grad = dv.distill_loss_grad(z, ids, t, status=st)
    assert int(st) == dv.STATUS_BAD_TOKEN
    ids[0, 1] = ids[1, 2] = -1
    check(z, ids, t, 1.0, loss, grad)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [999, 5003, 248319])
def test_strided_misaligned_and_in_place(dv, dtype, V):
    """Rows at any alignment; the gradient over the logits themselves."""
    g, z, ids, t = make(11 + V, 3, V, 12, dtype)
    wide = torch.zeros((3, V + 13), dtype=dtype, device=DEV)
    wide[:, 5:5 + V] = z
    want, wg = dv.distill_loss_grad(z, ids, t)
    view = wide[:, 5:5 + V]
    loss, grad = dv.distill_loss_grad(view, ids, t)
    check(z, ids, t, 1.0, loss, grad)
    other = torch.full((3, V + 6), 7.0, dtype=dtype, device=DEV)
    l2, g2 = dv.distill_loss_grad(view, ids, t, grad=other[:, 3:3 + V])
    check(z, ids, t, 1.0, l2, g2)
    assert bool((other[:, :3] == 7).all()) and bool((other[:, 3 + V:] == 7).all())
    l3, g3 = dv.distill_loss_grad(view, ids, t, grad=view)
    assert g3.data_ptr() == view.data_ptr()
    assert torch.equal(l3, loss) and torch.equal(g3, grad)
    assert bool((wide[:, :5] == 0).all()) and bool((wide[:, 5 + V:] == 0).all())


def test_results_repeat(dv):
    g, z, ids, t = make(13, 64, 30000, 32, BF)
    a = dv.distill_loss_grad(z, ids, t)
    b = dv.distill_loss_grad(z, ids, t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_side_stream_and_graph(dv):
    g, z, ids, t = make(14, 5, 5000, 16, BF)
    want = dv.distill_loss_grad(z, ids, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = z.clone().requires_grad_(True)
        loss = dv.distill_loss(a, ids, t)
        loss.sum().backward()
    s.synchronize()
    assert torch.equal(loss.detach(), want[0])
    grad = torch.empty_like(z)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        l3, _ = dv.distill_loss_grad(z, ids, t, grad=grad)
    z.copy_(torch.randn_like(z.float()).to(BF))
    want = dv.distill_loss_grad(z, ids, t)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(l3, want[0]) and torch.equal(grad, want[1])


def test_refusals(dv):
    g, z, ids, t = make(15, 2, 50, 4, FP)
    with pytest.raises(TypeError):
        dv.distill_loss(z, ids.long(), t)
    with pytest.raises(TypeError):
        dv.distill_loss(z, ids, t.half())
    with pytest.raises(ValueError):
        dv.distill_loss(z, ids[:1], t)
    with pytest.raises(ValueError):
        dv.distill_loss(z, ids, t[:, :3])
    with pytest.raises(ValueError):
        dv.distill_loss(z.t().contiguous().t(), ids, t)
    with pytest.raises(ValueError):
        dv.distill_loss(z, ids, t, row_weight=torch.ones(3, device=DEV))
    with pytest.raises(dv.DFlashError):
        dv.distill_loss(z, ids, t, temperature=0.0)
    with pytest.raises(ValueError):
        dv.distill_loss_grad(z, ids, t, grad=torch.empty((2, 49), device=DEV))
    with pytest.raises(ValueError):
        dv.distill_loss_grad(z, ids, t, grad=torch.empty((2, 50), device=DEV, dtype=BF))
    a = z.clone().requires_grad_(True)
    loss = dv.distill_loss(a, ids, t).sum()
    gr, = torch.autograd.grad(loss, a, create_graph=True)
    with pytest.raises(RuntimeError):
        gr.sum().backward()


def test_no_rows(dv):
    z = torch.zeros((0, 50), device=DEV, requires_grad=True)
    ids, t = torch.zeros((0, 4), dtype=torch.int32, device=DEV), torch.zeros((0, 4), device=DEV)
    loss = dv.distill_loss(z, ids, t)
    loss.sum().backward()
    assert loss.shape == (0,) and z.grad.shape == (0, 50)
    loss, grad = dv.distill_loss_grad(z.detach(), ids, t)
    assert loss.shape == (0,) and grad.shape == (0, 50)


def test_outputs_belong_to_the_call_s_stream(dv):
    """Tensors made by a call on another stream are not handed out again to the
    current one while that stream still writes them."""
    g, z, ids, t = make(16, 64, 50000, 8, BF)
    want = dv.distill_loss_grad(z, ids, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        loss, grad = dv.distill_loss_grad(z, ids, t, stream=s)
        del grad
        torch.full_like(z, 3.0)  # would take the freed memory at once, were it this stream's
    loss, grad = dv.distill_loss_grad(z, ids, t, stream=s)
    s.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


def test_backward_in_a_graph(dv):
    """Loss and backward captured together: replays read the tensors' contents."""
    g, z, ids, t = make(17, 6, 3000, 8, BF)
    a = z.clone().requires_grad_(True)
    up = torch.rand(6, generator=g, device=DEV)

    def both():
        loss = dv.distill_loss(a, ids, t)
        return loss.detach(), torch.autograd.grad(loss, a, up)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        loss, grad = both()
    with torch.no_grad():
        a.copy_(torch.randn(a.shape, generator=g, device=DEV).to(BF))
    up.mul_(-2.0)
    gr.replay()
    torch.cuda.synchronize()
    want = both()
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])
