"""dflash_kv_append: values over their scale."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_values_are_divided_by_their_scale(dv, dtype):
    """A quotient that stands halfway between two e4m3 values goes to the even
    one, and scales down to 2^-149 and up to 3e38 are divided by: a product with
    a rounded reciprocal does neither."""
    vals = torch.arange(1, 0x7F, dtype=torch.uint8).view(F8).float().unique()
    ties = (vals[1:] + vals[:-1]) / 2
    ties = ties[(ties > 2.0 ** -5) & (ties < 400)]
    scales = [float(2 * i + 1) for i in range(1, 32)] + [2.0 ** -149, 2.0 ** -140, 1.7 * 2.0 ** 127, 1.0]
    D, H = 64, len(scales)
    z = torch.tensor(scales, device=DEV)
    x = torch.zeros((-(-ties.numel() // D) * D, H))
    x[:ties.numel()] = ties[:, None] * torch.tensor(scales)
    x = x.view(-1, D, H).transpose(1, 2).to(dtype).to(DEV).contiguous()  # [tokens, heads, D]
    n = x.shape[0]
    caches = [torch.zeros((1, H, 32, D), device=DEV).to(F8) for _ in range(2)]
    pc = dv.PagedCache(caches[0], caches[1], torch.zeros((1, 1), dtype=torch.int32, device=DEV), z, z)
    dv.kv_append(pc, x, x, torch.zeros(1, dtype=torch.int32, device=DEV))
    want = (x.float() / z[:, None]).clamp(-448, 448).to(F8)
    for c in caches:
        got = c[0, :, :n].transpose(0, 1)
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), \
            (z[:, None].expand_as(got)[got.float() != want.float()], got[got.float() != want.float()])


@pytest.mark.parametrize("unit", [2.0 ** -130, 2.0 ** -100, 2.0 ** -9, 1.0, 2.0 ** 9])
def test_quotients_of_any_size(dv, unit):
    """Random values and scales (negative ones and powers of 2 among them), into
    e4m3's normal and subnormal range and beyond both ends."""
    D, H, n = 256, 64, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    z = (torch.rand(H, generator=g, device=DEV) + 0.5) * unit
    z[1::5] *= -1.0
    z[::7] = unit * 2.0 ** torch.arange(-4, 6, device=DEV, dtype=torch.float32)[:10].tile(2)[:len(z[::7])]
    x = torch.randn((n, H, D), generator=g, device=DEV) * 2.0 ** torch.randint(-14, 12, (n, 1, 1), generator=g, device=DEV)
    x = (x * unit).to(torch.bfloat16)
    caches = [torch.zeros((1, H, n, D), device=DEV).to(F8) for _ in range(2)]
    pc = dv.PagedCache(caches[0], caches[1], torch.zeros((1, 1), dtype=torch.int32, device=DEV), z, z)
    dv.kv_append(pc, x, x, torch.zeros(1, dtype=torch.int32, device=DEV))
    want = (x.float() / z[:, None]).clamp(-448, 448).to(F8)
    for c in caches:
        assert torch.equal(c[0].transpose(0, 1).view(torch.uint8), want.view(torch.uint8))
