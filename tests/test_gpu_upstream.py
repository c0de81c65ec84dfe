"""Gradients of the training operators from upstream gradients that begin anywhere in
memory, as slices of a joined gradient do."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


def joined(lead, parts, ups):
    """The parts one behind the other after `lead` values, and upstream gradients of the whole."""
    front = torch.zeros(lead, device=DEV, dtype=parts[0].dtype)
    return torch.cat([front, *(p.reshape(-1) for p in parts)]), torch.cat([front, *(u.reshape(-1) for u in ups)])


@pytest.mark.parametrize("lead", [1, 4, 7, 8])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_norms(dv, dtype, lead):
    leaves = [torch.randn((9, h, 64), device=DEV).to(dtype).requires_grad_(True) for h in (3, 2)]
    ups = [torch.randn_like(t) for t in leaves]
    want = torch.autograd.grad(dv.norm_rotate(*leaves), leaves, ups)
    whole, up = joined(lead, dv.norm_rotate(*leaves), ups)
    got = torch.autograd.grad(whole, leaves, up)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lead", [1, 4, 7, 8])
def test_attention(dv, lead):
    leaves = [torch.randn((70, h, 64), device=DEV).to(BF).requires_grad_(True) for h in (4, 2, 2)]
    start = torch.tensor([0, 30, 70], dtype=torch.int32, device=DEV)
    do = torch.randn((70, 4, 64), device=DEV).to(BF)
    want = torch.autograd.grad(dv.packed_attention(*leaves, start), leaves, do)
    whole, up = joined(lead, [dv.packed_attention(*leaves, start)], [do])
    got = torch.autograd.grad(whole, leaves, up)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_row_weights_that_are_learned(dv):
    h, w = torch.randn((40, 64), device=DEV).to(BF), torch.randn((300, 64), device=DEV).to(BF)
    labels = torch.arange(40, device=DEV, dtype=torch.int32)
    weight = torch.rand(40, device=DEV)
    want = dv.linear_cross_entropy(h, w, labels, row_weight=weight)
    with torch.no_grad():
        assert torch.equal(dv.linear_cross_entropy(h, w, labels, row_weight=weight.clone().requires_grad_(True)), want)
