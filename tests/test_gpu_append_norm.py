"""kv_append with norms against the definition in 64 bits: tokens of both types, weights
in the tokens' type, in fp32 and absent, from a token a request to prompts of thousands of
tokens, where a block takes several tokens and a thread several heads."""
import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


CASES = [
    # tokens of each request, cached, Hq, Hk, D, page, rot, interleaved, tokens' type, cache's, weights' (q, k), q_out over q
    ([1, 1, 1], [0, 7, 64], 6, 2, 64, 16, 64, False, HF, None, (HF, HF), False),
    ([9, 0, 3], [5, 1, 30], 8, 8, 128, 7, 64, True, BF, None, (F, F), False),
    ([5, 40], [100, 0], 4, 1, 256, 24, 48, False, HF, None, (F, None), True),
    ([17], [3], 3, 3, 128, 16, 0, False, BF, None, (None, None), False),
    ([8, 8], [0, 9], 8, 2, 128, 16, 128, False, HF, F8, (None, F), False),
    # more than 2^17 pairs of vectors: head_dim 64, 128 and 256
    ([4001, 33], [9, 500], 6, 2, 64, 16, 64, False, BF, None, (F, F), False),
    ([300, 1, 250], [0, 40, 11], 32, 8, 128, 64, 128, False, BF, None, (BF, BF), False),
    ([700], [123], 32, 8, 128, 16, 64, True, HF, None, (F, F), True),
    ([401, 7, 99], [0, 3, 77], 16, 4, 256, 32, 256, False, HF, None, (HF, None), False),
    ([1500, 2], [17, 1], 16, 4, 64, 100, 32, False, BF, F8, (F, F), False),
    ([512, 90], [1, 2], 24, 8, 128, 16, 128, True, HF, F8, (HF, HF), True),
    ([450], [2], 12, 4, 256, 16, 0, False, BF, F8, (None, None), False),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_the_definition(dv, case):
    counts, cached, Hq, Hk, D, page, rot, inter, dtype, cdt, wtypes, over = case
    cdt, eps, T = cdt or dtype, 1e-5, sum(counts)
    many = T * (Hq + 2 * Hk) * (D // 16) > 1 << 17
    assert many == (sum(counts) > 300)  # (both ways of sharing the work are met)
    g = torch.Generator(device=DEV)
    g.manual_seed(T + D + page)
    qkv = (torch.randn((T, Hq + 2 * Hk, D), generator=g, device=DEV) * 1.5).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    q0, k0, v0 = (t.double() for t in (q, k, v))
    w = [None if t is None else (1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(t) for t in wtypes]
    B, width = len(counts), max(-(-(c + n) // page) for c, n in zip(cached, counts))
    table = torch.randperm(B * width + 2, generator=g, device=DEV)[:B * width].view(B, width).to(torch.int32)
    caches = [torch.randn((B * width + 2, Hk, page, D), generator=g, device=DEV).to(cdt) for _ in range(2)]
    before = [c.clone() for c in caches]
    scales = [torch.rand(Hk, generator=g, device=DEV) * 0.05 + 0.02 for _ in range(2)] if cdt == F8 else [None, None]
    cache = dv.PagedCache(*caches, table, *scales)
    starts = torch.tensor([sum(counts[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV)
    lens = torch.tensor(cached, dtype=torch.int32, device=DEV)
    freq = 1e4 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot) if rot else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = dv.kv_append(cache, k, v, lens, q_start=starts, q=q, phases=None if freq is None else dv.rope_phases(freq, DEV),
                       interleaved=inter, q_out=q if over else None, status=status, eps=eps, q_weight=w[0], k_weight=w[1])
    assert int(status) == 0 and (got.data_ptr() == q.data_ptr()) == over
    assert torch.equal(v.double(), v0) and torch.equal(k.double(), k0) and (over or torch.equal(q.double(), q0))

    request = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(counts, device=DEV))
    pos = torch.arange(T, device=DEV) - starts[request].long() + lens[request].long()
    pages, slots = table[request, pos // page].long(), pos % page
    one = torch.ones(D, device=DEV, dtype=torch.float64)
    for x, y, wt, z in ((q0, got, w[0], None), (k0, caches[0], w[1], scales[0])):
        r, e = refs.norm64(x, one if wt is None else wt.double(), eps, pos, freq, inter)
        if y is not got:
            y = y.view(torch.uint8 if cdt == F8 else cdt)[pages, :, slots].view(cdt)
        if y.dtype == F8:
            z = z.double()[:, None]
            e, r = e / z + 2 * refs.F32 * (r / z).abs(), (r / z).clamp(-448, 448)
            bound = e + 2.0 ** -4 * (r.abs() + e) + 2.0 ** -10
        else:
            bound = refs.rounded(r, e, dtype)
        assert ((y.double() - r).abs() <= bound).all()
    # values are not normed, and the rest of the cache stays
    if cdt != F8:
        assert torch.equal(caches[1][pages, :, slots].double(), v0)
    else:
        y = caches[1].view(torch.uint8)[pages, :, slots].view(cdt).double()
        r = (v0 / scales[1].double()[:, None]).clamp(-448, 448)
        assert ((y - r).abs() <= 2.0 ** -4 * r.abs() + 2.0 ** -10).all()
    for c, b in zip(caches, before):
        c, b = c.view(torch.uint8), b.view(torch.uint8)
        c[pages, :, slots] = b[pages, :, slots]
        assert torch.equal(c, b)
