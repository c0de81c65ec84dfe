"""dflash_kv_append against the rotation's definition in 64 bits: pages of any
size and order, both cache layouts, strided inputs, ragged requests, 8-bit
caches, far positions, bad pages and lengths."""
import pytest

torch = pytest.importorskip("torch")
from operator_refs import F32, U, rotate64, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


def setup(seed, counts, cached, Hq, Hkv, D, page, dtype, cache_dtype, heads_inner, spare=3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, n = len(counts), sum(counts)
    width = max(-(-(c + m) // page) for c, m in zip(cached, counts)) + 1
    pages = B * width + spare
    table = torch.randperm(pages, generator=g, device=DEV)[:B * width].view(B, width).to(torch.int32)
    shape = (pages, page, Hkv, D) if heads_inner else (pages, Hkv, page, D)
    caches = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV).to(cache_dtype)
        caches.append(x.transpose(1, 2) if heads_inner else x)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)
    return g, table, caches, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


def expected(caches, table, k, v, counts, cached, page, freq, interleaved, scales):
    """The caches in fp64 with bounds on the errors (0 where nothing is written)."""
    out, tol = [c.double().clone() for c in caches], [torch.zeros(c.shape, dtype=torch.float64, device=DEV) for c in caches]
    u = U[caches[0].dtype]
    f8 = caches[0].dtype == torch.float8_e4m3fn
    for b, s in enumerate(starts_of(counts)[:-1]):
        for i in range(counts[b]):
            pos = cached[b] + i
            pg, sl = int(table[b, pos // page]), pos % page
            p64 = torch.tensor([float(pos)], dtype=torch.float64, device=DEV)
            for j, x in enumerate((k, v)):
                y = x[s + i:s + i + 1].double()
                size = y.abs()
                noise = 0.0
                if j == 0 and freq is not None:
                    y, size = rotate64(y, p64, freq, interleaved)
                    noise = 16 * F32  # sine, cosine, their angle's last bit, three roundings
                z = 1.0
                if f8:
                    z = 1.0 if scales is None else scales[j].double()[None, :, None]
                    y = (y / z).clamp(-448, 448)
                    noise += 2 * F32
                out[j][pg, :, sl] = y[0]
                exact = not f8 and not (j == 0 and freq is not None)
                t = u * y.abs() + noise * (size / z) * (1 + u) + (2.0 ** -10 if f8 else 2.0 ** -25)
                tol[j][pg, :, sl] = 0.0 if exact else t[0]
    return out, tol


CASES = [
    # counts, cached, Hq, Hkv, D, page, rot, interleaved, dtype, cache, heads_inner
    ([1], [0], 4, 1, 64, 16, 64, False, torch.bfloat16, None, False),
    ([1, 1, 1], [15, 16, 17], 8, 8, 128, 16, 128, False, torch.bfloat16, None, True),
    ([8, 8], [123, 60], 8, 2, 128, 64, 64, False, torch.float16, None, False),
    ([3, 0, 17, 1], [5, 9, 0, 31], 5, 5, 64, 7, 32, True, torch.bfloat16, None, False),
    ([9, 2], [1, 100], 6, 3, 256, 24, 256, True, torch.float16, None, True),
    ([16, 5], [40, 0], 4, 2, 256, 1, 128, False, torch.bfloat16, None, False),
    ([4, 4, 4], [11, 0, 200], 8, 4, 128, 48, 128, False, torch.bfloat16, torch.float8_e4m3fn, True),
    ([2, 33], [3, 7], 2, 2, 64, 32, 48, True, torch.float16, torch.float8_e4m3fn, False),
    ([6], [1000], 16, 2, 256, 100, 16, False, torch.bfloat16, torch.float8_e4m3fn, False),
    ([5], [50], 3, 1, 128, 16, 0, False, torch.bfloat16, None, False),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
@pytest.mark.parametrize("with_q", [True, False])
def test_matches_the_definition(dv, case, with_q):
    counts, cached, Hq, Hkv, D, page, rot, inter, dtype, cdt, inner = case
    cdt = cdt or dtype
    g, table, caches, q, k, v = setup(len(counts) + D + page, counts, cached, Hq, Hkv, D, page, dtype, cdt, inner)
    scales = None
    if cdt == torch.float8_e4m3fn:
        scales = [torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.004 for _ in range(2)]  # some saturate
    freq = 1e4 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot) if rot else None
    want, tol = expected(caches, table, k, v, counts, cached, page, freq, inter, scales)
    pc = dv.PagedCache(caches[0], caches[1], table, *(scales or (None, None)))
    uniform = len(set(counts)) == 1
    starts = None if uniform else torch.tensor(starts_of(counts), dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q0 = q.clone()
    out = dv.kv_append(pc, k, v, torch.tensor(cached, dtype=torch.int32, device=DEV), q_start=starts,
                       q=q if with_q else None, phases=None if freq is None else dv.rope_phases(freq),
                       interleaved=inter, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for c, w, t in zip(caches, want, tol):
        assert bool(((c.double() - w).abs() <= t).all()), float((c.double() - w).abs().max())
    assert torch.equal(q, q0)
    if not with_q:
        assert out is None
        return
    pos = torch.cat([torch.arange(c, c + n, device=DEV, dtype=torch.float64) for c, n in zip(cached, counts)])
    y, size = rotate64(q.double(), pos, freq, inter) if freq is not None else (q.double(), q.double() * 0)
    assert bool(((out.double() - y).abs() <= U[dtype] * y.abs() * (freq is not None) + 17 * F32 * size).all())


def test_far_positions(dv):
    """Position 2^31 - 50 of a long table: the angle is still exact to 2^-25 of
    a turn (fp32 radians would be off by 64)."""
    D, page = 128, 1 << 20
    pos = 2 ** 31 - 50
    width = 2048
    table = torch.zeros((1, width), dtype=torch.int32, device=DEV)
    c = [torch.zeros((1, 1, 1, D), dtype=torch.bfloat16, device=DEV).expand(1, 1, page, D) for _ in range(2)]
    pc = dv.PagedCache(c[0], c[1], table)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    q = torch.randn((1, 2, D), generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    k = torch.randn((1, 1, D), generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    freq = 1e6 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    out = dv.kv_append(pc, k, k, torch.tensor([pos], dtype=torch.int32, device=DEV), q=q, phases=dv.rope_phases(freq))
    y, size = rotate64(q.double(), torch.tensor([float(pos)], dtype=torch.float64, device=DEV), freq, False)
    # the reference's own angle: pos * w in fp64 is off by up to 2^31 2^-53 radians
    tol = U[torch.bfloat16] * y.abs() + (17 * F32 + 2.0 ** -21) * size
    assert bool(((out.double() - y).abs() <= tol).all())


def test_rotation_in_place_on_a_side_stream(dv):
    counts, cached = [4, 4], [10, 3]
    g, table, caches, q, k, v = setup(5, counts, cached, 6, 2, 128, 16, torch.bfloat16, torch.bfloat16, False)
    freq = 1e4 ** (-torch.arange(0, 128, 2, device=DEV, dtype=torch.float64) / 128)
    ph = dv.rope_phases(freq)
    lens = torch.tensor(cached, dtype=torch.int32, device=DEV)
    ref = [c.clone() for c in caches]
    want = dv.kv_append(dv.PagedCache(ref[0], ref[1], table), k, v, lens, q=q, phases=ph)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dv.kv_append(dv.PagedCache(caches[0], caches[1], table), k, v, lens, q=q, phases=ph, q_out=q, stream=s)
    s.synchronize()
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    assert torch.equal(caches[0], ref[0]) and torch.equal(caches[1], ref[1])


def test_special_values_reach_the_cache(dv):
    """Infinities and NaN are stored (e4m3: infinities saturate, NaN stays)."""
    D = 64
    x = torch.zeros((1, 1, D), dtype=torch.bfloat16, device=DEV)
    x[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e38])
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    for cdt in (torch.bfloat16, torch.float8_e4m3fn):
        c = [torch.zeros((1, 1, 16, D), device=DEV).to(cdt) for _ in range(2)]
        dv.kv_append(dv.PagedCache(c[0], c[1], table), x, x, lens)
        for y in c:
            y = y[0, 0, 0, :4].float()
            if cdt == torch.bfloat16:
                assert torch.equal(y[:2], x[0, 0, :2].float()) and y[3] == x[0, 0, 3].float()
            else:
                assert y[0] == 448 and y[1] == -448 and y[3] == 448
            assert bool(y[2].isnan())


def test_bad_pages_lengths_and_offsets(dv):
    """What lies outside is skipped and reported; the rest is written."""
    counts, cached = [4, 4, 4], [0, 14, 3]
    g, table, caches, q, k, v = setup(9, counts, cached, 2, 2, 64, 16, torch.bfloat16, torch.bfloat16, False)
    before = [c.clone() for c in caches]
    lens = torch.tensor(cached, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = table.clone()
    bad[1, 1] = -1                       # request 1's second page: positions 16, 17
    bad[2, 0] = caches[0].shape[0]       # request 2's only page
    dv.kv_append(dv.PagedCache(caches[0], caches[1], bad), k, v, lens, status=st)
    assert int(st) == dv.STATUS_BAD_PAGE
    want, _ = expected(before, table, k, v, counts, cached, 16, None, False, None)
    for b, pos in [(1, 16), (1, 17), (2, 3), (2, 4), (2, 5), (2, 6)]:
        for j in range(2):
            want[j][int(table[b, pos // 16]), :, pos % 16] = before[j][int(table[b, pos // 16]), :, pos % 16].double()
    for c, w in zip(caches, want):
        assert torch.equal(c.double(), w)
    # lengths below zero or past the table
    cap = table.shape[1] * 16
    for bad_len in ([-1, -5, -2 ** 31], [cap, cap + 7, 2 ** 31 - 1]):
        now = [c.clone() for c in caches]
        st.zero_()
        dv.kv_append(dv.PagedCache(caches[0], caches[1], table), k, v,
                     torch.tensor(bad_len, dtype=torch.int64).to(torch.int32).to(DEV), status=st)
        assert int(st) & dv.STATUS_BAD_LENGTH
        if bad_len[0] > 0:
            assert all(torch.equal(a, b) for a, b in zip(now, caches))
    # offsets that leave the packed tokens: nothing outside is touched
    st.zero_()
    dv.kv_append(dv.PagedCache(caches[0], caches[1], table), k, v, lens, status=st,
                 q_start=torch.tensor([0, 4, 100, 200], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert int(st) & dv.STATUS_BAD_LENGTH


def test_cache_beyond_32_bit_offsets(dv):
    """A cache of more than 2^32 elements: rows at its far end."""
    D, page, H = 256, 64, 8
    pages = (1 << 32) // (page * H * D) + 5
    c = [torch.empty((pages, H, page, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    k = torch.randn((3, H, D), device=DEV).to(torch.bfloat16)
    dv.kv_append(dv.PagedCache(c[0], c[1], table), k, k * 2, torch.tensor([62], dtype=torch.int32, device=DEV))
    for x, y in ((c[0], k), (c[1], k * 2)):
        assert torch.equal(x[pages - 1, :, 62:].float(), y[:2].to(torch.float8_e4m3fn).transpose(0, 1).float())
        assert torch.equal(x[pages - 2, :, 0].float(), y[2].to(torch.float8_e4m3fn).float())
