"""dflash_kv_append: values over their scale, and what its status word says of
offsets and lengths."""
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


def cache_of(dv, batch, pages=4, page=16, D=64, H=2):
    c = [torch.zeros((batch * pages, H, page, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    t = torch.arange(batch * pages, device=DEV, dtype=torch.int32).view(batch, pages)
    return c, dv.PagedCache(c[0], c[1], t)


@pytest.mark.parametrize("starts,cached,bad", [
    ([0, 4, 8], [0, 3], False), ([0, 0, 8], [0, 3], False), ([2, 4, 6], [0, 3], False), ([0, 8, 8], [0, 64], False),
    ([0, 8, 100], [0, 3], True), ([0, 6, 4, 8], [0, 3, 1], True), ([-3, 4, 8], [0, 3], True), ([0, 9, 9], [0, 3], True),
    ([0, 8, 8], [0, 65], True), ([0, 8, 8], [0, -1], True), ([0, 4, 8], [0, 61], True),
])
@pytest.mark.parametrize("spare", [0, 600])
def test_status_names_bad_offsets_and_lengths(dv, starts, cached, bad, spare):
    """Offsets that do not ascend inside the packed tokens, and lengths outside
    the page table, are reported whether or not a token meets them."""
    B = len(cached)
    starts, cached = starts + [starts[-1]] * spare, cached + [0] * spare
    c, pc = cache_of(dv, B + spare)
    x = torch.randn((8, 2, 64), device=DEV).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dv.kv_append(pc, x, x, torch.tensor(cached, dtype=torch.int32, device=DEV), status=st,
                 q_start=torch.tensor(starts, dtype=torch.int32, device=DEV))
    assert int(st) == (dv.STATUS_BAD_LENGTH if bad else 0)


def test_nothing_outside_is_touched(dv):
    """Negative lengths write nothing; clamped offsets write the tokens that are
    there and nothing else."""
    x = torch.randn((12, 2, 64), device=DEV).to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c, pc = cache_of(dv, 3)
    dv.kv_append(pc, x, x, torch.tensor([-1, -5, -2 ** 31], dtype=torch.int32, device=DEV), status=st)
    assert int(st) == dv.STATUS_BAD_LENGTH and all(bool((t == 0).all()) for t in c)
    st.zero_()
    dv.kv_append(pc, x, x, torch.tensor([0, 14, 3], dtype=torch.int32, device=DEV), status=st,
                 q_start=torch.tensor([0, 4, 100, 200], dtype=torch.int32, device=DEV))
    assert int(st) == dv.STATUS_BAD_LENGTH
    for t in c:
        want = torch.zeros_like(t)
        want[0, :, :4] = x[:4].transpose(0, 1)
        want[4, :, 14:16] = x[4:6].transpose(0, 1)
        want[5, :, :6] = x[6:12].transpose(0, 1)
        assert torch.equal(t, want)
