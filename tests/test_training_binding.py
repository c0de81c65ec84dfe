"""What the training operators' binding makes of tensors as autograd and callers hand
them over, on CPU tensors."""
import pytest

import speculative_decoding_verification_83_gb300 as dv
from speculative_decoding_verification_83_gb300 import training as tr

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    dv.build()
    tr._setup()


@pytest.mark.parametrize("first", [0, 1, 3, 8])
@pytest.mark.parametrize("shape", [(5, 2, 64), (1, 3, 64), (4, 1, 128), (1, 1, 64)])
def test_upstream_gradients_anywhere_in_memory(shape, first):
    """A slice of a joined gradient is contiguous and may begin anywhere: the kernels read 16 bytes at a time."""
    like = torch.zeros(shape, dtype=torch.bfloat16)
    n = like.numel()
    g = torch.randn(n + 8).to(torch.bfloat16)[first:first + n].view(shape)
    got, pointer, ts, hs = tr._usable(g, like)
    assert torch.equal(got, g) and pointer == got.data_ptr() and pointer % 16 == 0
    assert (ts, hs) == got.stride()[:2] and got.stride(2) == 1
    if g.data_ptr() % 16 == 0:
        assert pointer == g.data_ptr()  # no copy


def test_row_weights_that_are_learned():
    """A gradient that would be dropped is refused; under no_grad none is, and the call goes on to its other checks."""
    args = (torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((10, 64), dtype=torch.bfloat16),
            torch.zeros(2, dtype=torch.int32))
    weight = torch.ones(2, requires_grad=True)
    with pytest.raises(ValueError, match="row_weight"):
        dv.linear_cross_entropy(*args, row_weight=weight)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        dv.linear_cross_entropy(*args, row_weight=weight)
