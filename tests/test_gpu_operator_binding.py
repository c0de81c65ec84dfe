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
