"""What the operators' binding does with torch's own bookkeeping: gradients it
does not carry, tensors it writes in place, and streams."""
import pytest

torch = pytest.importorskip("torch")

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


def setup(dv, B=2, H=2, Hq=4, D=64, page=16, pages=4):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    c = [torch.randn((B * pages, H, page, D), generator=g, device=DEV).to(BF) for _ in range(2)]
    t = torch.arange(B * pages, device=DEV, dtype=torch.int32).view(B, pages)
    q = torch.randn((B, Hq, D), generator=g, device=DEV).to(BF)
    kv = [torch.randn((B, H, D), generator=g, device=DEV).to(BF) for _ in range(2)]
    return dv.PagedCache(c[0], c[1], t), q, kv, torch.full((B,), 40, dtype=torch.int32, device=DEV)


def test_gradients_are_not_dropped_in_silence(dv):
    pc, q, (k, v), ln = setup(dv)
    leaf = [t.clone().requires_grad_(True) for t in (q, k, v)]
    with pytest.raises(ValueError, match="q has no gradient"):
        dv.paged_attention(pc, leaf[0], ln)
    with pytest.raises(ValueError, match="k has no gradient"):
        dv.kv_append(pc, leaf[1], v, ln)
    with pytest.raises(ValueError, match="v has no gradient"):
        dv.kv_append(pc, k, leaf[2], ln)
    with pytest.raises(ValueError, match="q has no gradient"):
        dv.kv_append(pc, k, v, ln, q=leaf[0] * 1)
    with pytest.raises(ValueError, match="cache has no gradient"):
        grown = dv.PagedCache(pc.k.clone().requires_grad_(True), pc.v, pc.page_table)
        dv.paged_attention(grown, q, ln)
    with pytest.raises(ValueError, match="out has no gradient"):
        dv.paged_attention(pc, q, ln, out=q.clone().requires_grad_(True))
    want = dv.paged_attention(pc, q, ln)
    with torch.no_grad():
        assert torch.equal(dv.paged_attention(pc, leaf[0], ln), want)
        dv.kv_append(pc, leaf[1], leaf[2], ln, q=leaf[0])
    assert torch.equal(dv.paged_attention(pc, leaf[0].detach(), ln + 1), dv.paged_attention(pc, q, ln + 1))
    z = torch.randn((2, 50), device=DEV, requires_grad=True)
    ids, t = torch.zeros((2, 3), dtype=torch.int32, device=DEV), torch.zeros((2, 3), device=DEV)
    with pytest.raises(ValueError, match="grad has no gradient"):
        dv.distill_loss_grad(z, ids, t, grad=z)
    with torch.no_grad():
        dv.distill_loss_grad(z, ids, t, grad=z)
    dv.distill_loss_grad(z, ids, t)


def test_tensors_written_in_place_are_known_to_autograd(dv):
    """A tensor that autograd keeps for a backward pass and a call then writes
    over is an error of the backward pass, as it is for torch's own operations."""
    pc, q, (k, v), ln = setup(dv)
    w = torch.ones((), device=DEV, requires_grad=True)

    def refused(t, write):
        y = (t * w).float().sum()
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()

    refused(pc.k, lambda: dv.kv_append(pc, k, v, ln))
    refused(pc.v, lambda: dv.kv_append(pc, k, v, ln))
    refused(q, lambda: dv.kv_append(pc, k, v, ln, q=q, q_out=q))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    refused(out, lambda: dv.paged_attention(pc, q, ln, out=out, lse=lse))
    refused(lse, lambda: dv.paged_attention(pc, q, ln, out=out, lse=lse))
    z = torch.randn((2, 50), device=DEV)
    ids, t = torch.zeros((2, 3), dtype=torch.int32, device=DEV), torch.zeros((2, 3), device=DEV)
    refused(z, lambda: dv.distill_loss_grad(z, ids, t, grad=z))
    # the loss's own saved logits
    a = torch.randn((2, 50), device=DEV, requires_grad=True)
    b = a * 1
    loss = dv.distill_loss(b, ids, t).sum()
    with torch.no_grad():
        dv.distill_loss_grad(b, ids, t, grad=b)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # tensors without a version are written as ever
        pi, qi, (ki, vi), li = setup(dv)
        dv.kv_append(pi, ki, vi, li)
        dv.paged_attention(pi, qi, li + 1)


def test_inputs_outlive_a_call_on_another_stream(dv):
    """A call on another stream still reads its inputs when Python has let go of
    them: their memory is not handed out before."""
    pc, q, (k, v), ln = setup(dv, B=64, Hq=64, H=8, D=128)
    want = dv.paged_attention(pc, q, ln)
    s = torch.cuda.Stream()
    z = torch.randn((64, 20000), device=DEV)
    ids = torch.randint(0, 20000, (64, 8), device=DEV, dtype=torch.int32)
    t = torch.randn((64, 8), device=DEV)
    wl, wg = dv.distill_loss_grad(z, ids, t)
    torch.cuda.synchronize()
    for _ in range(3):
        q1, z1 = q.clone(), z.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # the calls wait in the stream for about 10 ms
        got = dv.paged_attention(pc, q1, ln, stream=s)
        loss, grad = dv.distill_loss_grad(z1, ids, t, stream=s)
        del q1, z1
        over = [torch.full_like(q, 3.0), torch.full_like(z, 3.0)]  # at once in the freed memory, were it free
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(loss, wl) and torch.equal(grad, wg)
        del over


def test_tables_of_one_column(dv):
    """Extents of one in a page table are never stepped over."""
    pc, q, (k, v), ln = setup(dv, pages=1)
    ln = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    want = dv.paged_attention(pc, q, ln)
    column = torch.stack([pc.page_table[:, 0]] * 3).t()[:, :1]
    assert column.stride(1) != 1 and column.shape == (2, 1)
    assert torch.equal(dv.paged_attention(dv.PagedCache(pc.k, pc.v, column), q, ln), want)


def test_outputs_whose_rows_share_memory_are_refused(dv):
    """As torch's own operations refuse them: which row's result stays would be
    left to chance."""
    pc, q, (k, v), ln = setup(dv)
    for shared in (torch.zeros((1, 4, 64), dtype=BF, device=DEV).expand(2, 4, 64),
                   torch.zeros((2, 1, 64), dtype=BF, device=DEV).expand(2, 4, 64),
                   torch.zeros(1000, dtype=BF, device=DEV).as_strided((2, 4, 64), (256, 32, 1))):
        with pytest.raises(ValueError, match="share memory"):
            dv.paged_attention(pc, q, ln, out=shared)
        with pytest.raises(ValueError, match="share memory"):
            dv.kv_append(pc, k, v, ln, q=q, q_out=shared)


def test_a_cache_without_requests_is_refused(dv):
    pc, q, (k, v), ln = setup(dv)
    none = dv.PagedCache(pc.k, pc.v, pc.page_table[:0])
    for call in (lambda: dv.paged_attention(none, q, ln[:0]), lambda: dv.kv_append(none, k, v, ln[:0])):
        with pytest.raises(dv.DFlashError, match="batch=0"):
            call()
