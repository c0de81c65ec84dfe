"""dflash_paged_attention against softmax attention in 64 bits: shared heads,
blocks and single tokens, ragged and empty requests, pages of any size and
order, both cache layouts, 8-bit caches, masked infinities and NaN, splits
over many SMs, graphs and streams."""
import math

import pytest

torch = pytest.importorskip("torch")
from operator_refs import F32, U, attend64, starts_of  # noqa: E402

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


def make(seed, counts, lens, Hq, Hkv, D, page, dtype, cdt, inner, qscale=2.0, fill=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B = len(counts)
    width = max(1, max(-(-n // page) for n in lens))
    pages = B * width + 2
    table = torch.randperm(pages, generator=g, device=DEV)[:B * width].view(B, width).to(torch.int32)
    shape = (pages, page, Hkv, D) if inner else (pages, Hkv, page, D)
    caches = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV).to(cdt)
        caches.append(x.transpose(1, 2) if inner else x)
    if fill is not None:  # every slot no request uses
        used = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
        for b in range(B):
            for j in range(lens[b]):
                used[int(table[b, j // page]), j % page] = True
        for x in caches:
            y = x.transpose(1, 2)
            (y.view(torch.uint8) if cdt == F8 else y)[~used] = 0x7F if cdt == F8 else fill
    q = (torch.randn((sum(counts), Hq, D), generator=g, device=DEV) * qscale).to(dtype)
    scales = [torch.rand(Hkv, generator=g, device=DEV) + 0.5 for _ in range(2)] if cdt == F8 else None
    return table, caches, q, scales


def rows(cache, table, b, L, page, scale=None):
    """[L, heads, D] fp64 of a request."""
    pos = torch.arange(L, device=DEV)
    y = cache.transpose(1, 2)
    y = y.view(torch.uint8) if cache.dtype == F8 else y
    x = y[table[b].long()[pos // page], pos % page]
    x = (x.view(F8).float() if cache.dtype == F8 else x).double()
    return x if scale is None else x * scale.double()[None, :, None]


def rows_of(y, at):
    return y.view(torch.uint8)[at].view(F8) if y.dtype == F8 else y[at]


def check(dv, table, caches, q, scales, counts, lens, page, causal, scale=None, seen=None, **kw):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    pc = dv.PagedCache(caches[0], caches[1], table, *(scales or (None, None)))
    starts = None if len(set(counts)) == 1 else torch.tensor(starts_of(counts), dtype=torch.int32, device=DEV)
    out, lse = dv.paged_attention(pc, q, torch.tensor(lens, dtype=torch.int32, device=DEV), q_start=starts, scale=scale,
                                  causal=causal, return_lse=True, **kw)
    torch.cuda.synchronize()
    # the weights are rounded to the products' type: the tokens', or f16 for the
    # 8-bit caches of few rows (or head_dim 256)
    rows_each = -(-q.shape[0] // len(counts)) * (q.shape[1] // caches[0].shape[1])
    up = U[torch.float16] if caches[0].dtype == F8 and (rows_each <= 32 or D == 256) else U[q.dtype]
    for b, s in enumerate(starts_of(counts)[:-1]):
        n, L = counts[b], lens[b]
        if n == 0:
            continue
        vis = torch.ones((n, L), dtype=torch.bool, device=DEV)
        if causal:
            vis &= torch.arange(L, device=DEV)[None] <= (L - n + torch.arange(n, device=DEV))[:, None]
        if seen is not None:
            vis &= seen[b][None, :L]
        k = rows(caches[0], table, b, L, page, scales and scales[0])
        v = rows(caches[1], table, b, L, page, scales and scales[1])
        want, want_lse, spread, dx = attend64(q[s:s + n].double(), k, v, scale, vis)
        # sums over L positive weights, in runs of a warp's share; exponentials good to 2^-22
        acc = (L / 16 + 200) * F32 + 2.0 ** -21
        got, got_lse = out[s:s + n].double(), lse[s:s + n].double()
        none = want_lse == -math.inf
        assert torch.equal(got_lse == -math.inf, none)
        tol = U[q.dtype] * want.abs() + (up + 2 * dx[..., None] + 2 * acc) * spread * (1 + U[q.dtype]) \
            + (2.0 ** -25 if q.dtype == torch.float16 else 1e-38)
        err = (got - want).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()))
        ltol = dx + acc + 4 * F32 * (1 + want_lse.abs())
        lerr = (got_lse - want_lse).abs()
        assert bool((lerr[~none] <= ltol[~none]).all()), (b, float(lerr[~none].max()))
    return out, lse


BF, HF = torch.bfloat16, torch.float16
CASES = [
    # counts, lens, Hq, Hkv, D, page, causal, dtype, cache, heads_inner
    ([1], [1], 1, 1, 64, 16, True, BF, BF, False),
    ([1], [2], 8, 1, 128, 16, True, BF, BF, True),
    ([1, 1, 1, 1], [63, 64, 65, 0], 8, 2, 128, 16, True, BF, BF, False),
    ([1, 1], [1000, 333], 6, 1, 64, 7, True, HF, HF, False),
    ([1], [5000], 16, 1, 256, 64, True, BF, BF, True),
    ([1, 1], [129, 3001], 40, 8, 128, 128, True, BF, F8, False),
    ([1, 1], [77, 260], 12, 2, 64, 24, True, HF, F8, True),
    ([1], [900], 4, 4, 256, 1, True, BF, F8, False),
    ([8, 8], [8, 700], 8, 2, 128, 64, True, BF, BF, False),
    ([8, 8, 8], [100, 9, 64], 32, 2, 128, 16, True, HF, HF, True),
    ([3, 0, 17, 1], [50, 40, 17, 4000], 6, 2, 64, 32, True, BF, BF, False),
    ([16, 16], [16, 500], 8, 4, 64, 24, False, HF, HF, False),
    ([5, 33], [700, 90], 3, 3, 128, 48, False, BF, BF, True),
    ([9, 4], [300, 1025], 16, 2, 256, 16, True, HF, HF, False),
    ([8, 2], [250, 64], 24, 4, 256, 32, True, BF, F8, False),
    ([16], [2050], 16, 1, 128, 100, True, BF, F8, True),
    ([130], [130], 4, 2, 64, 16, True, BF, BF, False),      # a whole prompt
    ([4, 4], [2, 1], 2, 1, 64, 16, True, BF, BF, False),     # fewer positions than tokens: rows that see none
    ([1] * 70, [1 + 13 * b for b in range(70)], 4, 2, 128, 16, True, BF, BF, False),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_the_definition(dv, case):
    counts, lens, Hq, Hkv, D, page, causal, dtype, cdt, inner = case
    # slots past each request's length hold NaN: they must not reach the sums
    table, caches, q, scales = make(len(lens) + D + page, counts, lens, Hq, Hkv, D, page, dtype, cdt, inner,
                                    fill=float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    check(dv, table, caches, q, scales, counts, lens, page, causal, status=st)
    assert int(st) == 0


@pytest.mark.parametrize("D,cdt", [(64, BF), (128, BF), (128, F8), (256, F8)])
def test_long_and_split(dv, D, cdt):
    """One request over every SM: partial results of many CTAs joined."""
    lens = [70001]
    table, caches, q, scales = make(D, [2], lens, 8, 2, D, 64, BF, cdt, False)
    a, la = check(dv, table, caches, q, scales, [2], lens, 64, True)
    b, lb = check(dv, table, caches, q, scales, [2], lens, 64, True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("cdt", [BF, F8])
def test_extreme_scores(dv, cdt):
    """Scores in the hundreds of thousands and tiny ones; q far outside f16."""
    for qscale in (1e-6, 3e5):
        table, caches, q, scales = make(3, [2, 2], [90, 200], 4, 2, 128, 16, BF, cdt, False, qscale=qscale)
        check(dv, table, caches, q, scales, [2, 2], [90, 200], 16, True)


@pytest.mark.parametrize("cdt", [BF, HF, F8])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_masked_values_never_count(dv, cdt, bad):
    """Non-finite keys and values of later tokens of the block: earlier tokens
    do not see them. Rows that do see them are not finite."""
    dtype = BF if cdt == F8 else cdt
    counts, lens, page = [6, 6], [40, 70], 16
    table, caches, q, scales = make(8, counts, lens, 4, 2, 64, page, dtype, cdt, False)
    first = 3  # tokens 3, 4, 5 hold the bad values
    clean = [c.clone() for c in caches]
    for b in range(2):
        for i in range(first, 6):
            j = lens[b] - 6 + i
            for n, c in enumerate(caches):
                if cdt == F8:
                    c.view(torch.uint8)[int(table[b, j // page]), :, j % page, n::3] = 0x7F
                else:
                    c[int(table[b, j // page]), :, j % page, n::3] = bad
    pc = dv.PagedCache(caches[0], caches[1], table, *(scales or (None, None)))
    pr = dv.PagedCache(clean[0], clean[1], table, *(scales or (None, None)))
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got, gl = dv.paged_attention(pc, q, ln, return_lse=True)
    want, wl = dv.paged_attention(pr, q, ln, return_lse=True)
    g, w = got.view(2, 6, 4, 64), want.view(2, 6, 4, 64)
    # the seen keys are the same; their sums may run in another order
    tol = 4 * U[dtype] * w[:, :first].float().abs().clamp_min(0.05)
    assert bool(((g[:, :first].float() - w[:, :first].float()).abs() <= tol).all())
    assert bool(((gl.view(2, 6, 4)[:, :first] - wl.view(2, 6, 4)[:, :first]).abs() <= 1e-5).all())
    if not (cdt != F8 and bad == -float("inf")):  # a score of -inf weighs nothing
        assert not bool(g[:, first:].float().isfinite().all(-1).any())


BLOCKS = [
    # counts, lens, Hq, Hkv, D, page, causal, dtype: 17 to 128 rows a head and more, every
    # head_dim, lengths around a tile's 64 and 128 keys
    ([17], [17], 1, 1, 128, 16, True, BF),
    ([5, 5], [127, 128], 8, 2, 128, 64, True, BF),
    ([5, 5], [129, 640], 8, 2, 64, 5, False, HF),
    ([8, 8], [63, 1000], 8, 2, 256, 16, True, BF),
    ([8, 8, 8], [64, 65, 192], 16, 2, 128, 48, True, HF),
    ([8] * 3, [2000, 8, 333], 64, 8, 128, 64, True, BF),
    ([8] * 2, [256, 300], 8, 1, 64, 16, True, BF),
    ([7] * 2, [300, 129], 9, 1, 256, 7, False, BF),
    ([16] * 2, [1000, 16], 16, 2, 128, 64, True, BF),
    ([16] * 2, [255, 257], 16, 2, 64, 32, False, HF),
    ([16] * 2, [127, 450], 8, 1, 256, 128, True, HF),
    ([33, 20, 1, 0], [400, 20, 300, 5], 12, 2, 128, 16, True, BF),
    ([300], [300], 2, 1, 128, 16, True, BF),
    ([6] * 2, [4, 3], 8, 1, 128, 16, True, BF),           # rows that see no key
    ([8] * 90, [1 + 17 * b for b in range(90)], 8, 2, 64, 16, False, BF),
]


@pytest.mark.parametrize("case", BLOCKS, ids=range(len(BLOCKS)))
@pytest.mark.parametrize("inner", [False, True])
@pytest.mark.parametrize("f8", [False, True])
def test_blocks_match_the_definition(dv, case, inner, f8):
    counts, lens, Hq, Hkv, D, page, causal, dtype = case
    table, caches, q, scales = make(len(lens) + D + page, counts, lens, Hq, Hkv, D, page, dtype, F8 if f8 else dtype,
                                    inner, fill=float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = check(dv, table, caches, q, scales, counts, lens, page, causal, status=st)
    b = check(dv, table, caches, q, scales, counts, lens, page, causal, status=st)
    assert int(st) == 0 and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D,rows,cdt", [(64, 32, BF), (64, 128, BF), (128, 32, BF), (128, 64, BF), (128, 128, BF),
                                        (256, 64, BF), (64, 64, F8), (128, 32, F8), (128, 128, F8)])
def test_long_blocks_are_split(dv, D, rows, cdt):
    """One request over every SM, its rising scores moving the reference again and again."""
    n, lens = rows // 8, [70001]
    table, caches, q, scales = make(D + rows, [n], lens, 16, 2, D, 64, BF, cdt, False)
    grow = torch.linspace(0.05, 3.0, lens[0], device=DEV)
    pos = torch.arange(lens[0], device=DEV)
    y = caches[0].transpose(1, 2)
    at = table[0].long()[pos // 64], pos % 64
    grown = (rows_of(y, at).float() * grow[:, None, None]).to(cdt)
    if cdt == F8:
        y.view(torch.uint8)[at] = grown.view(torch.uint8)
    else:
        y[at] = grown
    a, la = check(dv, table, caches, q, scales, [n], lens, 64, True)
    b, lb = check(dv, table, caches, q, scales, [n], lens, 64, True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 8), (256, 16)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_masked_values_never_count_in_blocks(dv, dtype, D, G, bad):
    """As test_masked_values_never_count, for 24 to 96 rows a head."""
    counts, lens, page, first, n = [6, 6], [140, 70], 16, 3, 6
    table, caches, q, _ = make(8, counts, lens, 2 * G, 2, D, page, dtype, dtype, False)
    clean = [c.clone() for c in caches]
    for b in range(2):
        for i in range(first, n):
            j = lens[b] - n + i
            for k, c in enumerate(caches):
                c[int(table[b, j // page]), :, j % page, k::3] = bad
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got, gl = dv.paged_attention(dv.PagedCache(caches[0], caches[1], table), q, ln, return_lse=True)
    want, wl = dv.paged_attention(dv.PagedCache(clean[0], clean[1], table), q, ln, return_lse=True)
    g, w = got.view(2, n, 2 * G, D), want.view(2, n, 2 * G, D)
    assert torch.equal(g[:, :first], w[:, :first])
    assert torch.equal(gl.view(2, n, 2 * G)[:, :first], wl.view(2, n, 2 * G)[:, :first])
    if bad != -float("inf"):
        assert not bool(g[:, first:].float().isfinite().all(-1).any())
    # only values: finite scores, so a row is infinite exactly where a value it sees is
    caches[0].copy_(clean[0])
    got = dv.paged_attention(dv.PagedCache(caches[0], caches[1], table), q, ln).view(2, n, 2 * G, D)
    assert torch.equal(got[:, :first], w[:, :first])
    where = torch.zeros(D, dtype=torch.bool, device=DEV)
    where[1::3] = True
    assert bool((~got[:, first:].float().isfinite() == where).all())


@pytest.mark.parametrize("D", [64, 128])
def test_masked_nan_never_counts_in_8_bit_blocks(dv, D):
    counts, lens, page, first, n, G = [6, 6], [140, 70], 16, 3, 6, 8
    table, caches, q, scales = make(8, counts, lens, 2 * G, 2, D, page, BF, F8, False)
    clean = [c.clone() for c in caches]
    for b in range(2):
        for i in range(first, n):
            j = lens[b] - n + i
            caches[1].view(torch.uint8)[int(table[b, j // page]), :, j % page, 1::3] = 0x7F if i % 2 else 0xFF
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got, gl = dv.paged_attention(dv.PagedCache(caches[0], caches[1], table, *scales), q, ln, return_lse=True)
    want, wl = dv.paged_attention(dv.PagedCache(clean[0], clean[1], table, *scales), q, ln, return_lse=True)
    g, w = got.view(2, n, 2 * G, D), want.view(2, n, 2 * G, D)
    assert torch.equal(g[:, :first], w[:, :first]) and torch.equal(gl, wl)
    where = torch.zeros(D, dtype=torch.bool, device=DEV)
    where[1::3] = True
    assert bool((g[:, first:].isnan() == where).all())


@pytest.mark.parametrize("counts", [[1, 1], [6, 6]])
def test_scales_of_any_sign(dv, counts):
    """Scales below and at zero: the stored values stand for themselves times the scale."""
    lens, page, D = [300, 77], 16, 128
    table, caches, q, _ = make(31, counts, lens, 12, 3, D, page, BF, F8, False)
    scales = [torch.tensor([-0.7, 0.0, 1.3], device=DEV), torch.tensor([1.1, -2.0, 0.0], device=DEV)]
    check(dv, table, caches, q, scales, counts, lens, page, True)


def test_blocks_with_extreme_scores(dv):
    for qscale in (1e-6, 3e4):
        table, caches, q, _ = make(3, [8, 8], [90, 300], 8, 2, 128, 16, BF, BF, False, qscale=qscale)
        check(dv, table, caches, q, None, [8, 8], [90, 300], 16, True)


def test_lowest_and_infinite_scores(dv):
    """Keys whose score is -inf weigh nothing; a row of them alone gives 0, -inf."""
    D, page, L = 64, 16, 40
    table, caches, q, _ = make(4, [1, 1], [L, L], 2, 1, D, page, BF, BF, False)
    q.fill_(1.0)
    pos = torch.arange(L, device=DEV)
    for b, hidden in ((0, pos % 3 == 0), (1, pos >= 0)):
        at = table[b].long()[pos // page], pos % page
        caches[0].transpose(1, 2)[at[0][hidden], at[1][hidden]] = -float("inf")
    pc = dv.PagedCache(caches[0], caches[1], table)
    out, lse = dv.paged_attention(pc, q, torch.tensor([L, L], dtype=torch.int32, device=DEV), return_lse=True)
    assert bool((lse[1] == -math.inf).all()) and bool((out[1] == 0).all())
    k = rows(caches[0], table, 0, L, page)
    v = rows(caches[1], table, 0, L, page)
    ok = pos % 3 != 0
    want, wl, spread, dx = attend64(q[:1].double(), k[ok], v[ok], D ** -0.5,
                                    torch.ones((1, int(ok.sum())), dtype=torch.bool, device=DEV))
    assert bool(((out[:1].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * dx[..., None] + 1e-4)
                 * spread).all())


def test_bad_pages_lengths_and_offsets(dv):
    counts, lens, page = [2, 2, 2], [40, 64, 20], 16
    table, caches, q, _ = make(6, counts, lens, 4, 2, 128, page, BF, BF, False)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = table.clone()
    bad[0, 1] = -1
    bad[1, 0] = 2 ** 31 - 1
    seen = [torch.ones(64, dtype=torch.bool, device=DEV) for _ in range(3)]
    seen[0][16:32] = False
    seen[1][0:16] = False
    safe = bad.clone()
    safe[0, 1] = safe[1, 0] = 0  # for the reference alone
    pc = dv.PagedCache(caches[0], caches[1], bad)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = dv.paged_attention(pc, q, ln, return_lse=True, status=st)
    assert int(st) == dv.STATUS_BAD_PAGE
    for b in range(3):
        L = lens[b]
        vis = torch.arange(L, device=DEV)[None] <= (L - 2 + torch.arange(2, device=DEV))[:, None]
        vis &= seen[b][None, :L]
        want, wl, spread, dx = attend64(q[2 * b:2 * b + 2].double(), rows(caches[0], safe, b, L, page),
                                        rows(caches[1], safe, b, L, page), 128 ** -0.5, vis)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * dx[..., None] + 1e-4) * spread
        assert bool(((out[2 * b:2 * b + 2].double() - want).abs() <= tol).all())
    # lengths: negative ones count as 0, ones past the table as the table's end
    st.zero_()
    good = dv.PagedCache(caches[0], caches[1], table)
    out, lse = dv.paged_attention(good, q, torch.tensor([-7, 64, 20], dtype=torch.int32, device=DEV), return_lse=True,
                                  status=st)
    assert int(st) == dv.STATUS_BAD_LENGTH
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
    st.zero_()
    cap = table.shape[1] * page
    a = dv.paged_attention(good, q, torch.tensor([2 ** 31 - 1, cap + 1, 20], dtype=torch.int32, device=DEV), status=st)
    b = dv.paged_attention(good, q, torch.tensor([cap, cap, 20], dtype=torch.int32, device=DEV))
    assert int(st) == dv.STATUS_BAD_LENGTH and torch.equal(a, b)
    # offsets outside the packed tokens are clamped
    st.zero_()
    dv.paged_attention(good, q, ln, q_start=torch.tensor([-4, 3, 1, 1000], dtype=torch.int32, device=DEV), status=st)
    torch.cuda.synchronize()
    assert int(st) == dv.STATUS_BAD_LENGTH


def test_rows_of_no_request_are_left_alone(dv):
    counts, lens, page = [2, 3], [20, 30], 16
    table, caches, q, _ = make(2, counts + [4], lens + [30], 4, 2, 64, page, BF, BF, False)
    pc = dv.PagedCache(caches[0], caches[1], table[:2])
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    dv.paged_attention(pc, q, torch.tensor(lens, dtype=torch.int32, device=DEV), out=out, lse=lse,
                       q_start=torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV))
    assert bool((out[5:] == 7).all()) and bool((lse[5:] == 7).all())
    want = dv.paged_attention(pc, q[:5], torch.tensor(lens, dtype=torch.int32, device=DEV),
                              q_start=torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV))
    assert torch.equal(out[:5], want)


def test_strided_queries_outputs_and_tables(dv):
    counts, lens, page = [2, 2], [100, 37], 16
    table, caches, q, _ = make(12, counts, lens, 8, 2, 128, page, BF, BF, False)
    wide = torch.full((2, table.shape[1] + 3), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    want = dv.paged_attention(dv.PagedCache(caches[0], caches[1], table), q,
                              torch.tensor(lens, dtype=torch.int32, device=DEV))
    big = torch.zeros((4, 12, 128), dtype=BF, device=DEV)
    big[:, 2:10] = q
    heads_first = torch.zeros((8, 4, 128), dtype=BF, device=DEV)
    got = dv.paged_attention(dv.PagedCache(caches[0], caches[1], wide[:, :table.shape[1]]), big[:, 2:10],
                             torch.tensor(lens, dtype=torch.int32, device=DEV), out=heads_first.transpose(0, 1))
    assert torch.equal(got, want)


def test_side_stream_and_graph(dv):
    """On another stream, and captured: a replay reads the tensors' contents at
    its time (lengths, table, queries)."""
    counts, lens, page = [1, 1], [500, 90], 16
    table, caches, q, _ = make(21, counts, lens, 8, 2, 128, page, BF, BF, False)
    pc = dv.PagedCache(caches[0], caches[1], table)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = dv.paged_attention(pc, q, ln)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dv.paged_attention(pc, q, ln, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        dv.paged_attention(pc, q, ln, out=out)
    q2 = torch.randn_like(q.float()).to(BF)
    want2 = dv.paged_attention(pc, q2, ln - 30)
    q.copy_(q2)
    ln.sub_(30)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_cache_beyond_32_bit_offsets(dv):
    D, page, H = 256, 64, 8
    pages = (1 << 32) // (page * H * D) + 5
    c = [torch.empty((pages, H, page, D), dtype=F8, device=DEV) for _ in range(2)]
    for x in c:
        x[-3:] = torch.randn((3, H, page, D), device=DEV).to(F8)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 8, D), device=DEV).to(BF)
    got = dv.paged_attention(dv.PagedCache(c[0], c[1], table), q, torch.tensor([150], dtype=torch.int32, device=DEV))
    small = [x[-3:].clone() for x in c]
    t2 = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    want = dv.paged_attention(dv.PagedCache(small[0], small[1], t2), q, torch.tensor([150], dtype=torch.int32, device=DEV))
    assert torch.equal(got, want)


def test_append_then_attend_equals_a_plain_decoder(dv):
    """Token by token or as a block: the same keys, the same attention."""
    D, H, Hq, page, n = 128, 2, 8, 16, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    qkv = torch.randn((n, Hq + 2 * H, D), generator=g, device=DEV).to(BF)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    freq = 1e4 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    ph = dv.rope_phases(freq)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    outs = []
    for block in (True, False):
        c = [torch.zeros((3, H, page, D), dtype=BF, device=DEV) for _ in range(2)]
        pc = dv.PagedCache(c[0], c[1], table)
        steps = [(0, n)] if block else [(i, i + 1) for i in range(n)]
        got = []
        for lo, hi in steps:
            at = torch.tensor([13 + lo], dtype=torch.int32, device=DEV)
            qr = dv.kv_append(pc, k[lo:hi], v[lo:hi], at, q=q[lo:hi], phases=ph)
            got.append(dv.paged_attention(pc, qr, at + (hi - lo)))
        outs.append(torch.cat(got).float())
    # the same sums over the same keys, which may fall to other lanes: P's and the output's rounding
    assert float((outs[0] - outs[1]).abs().max()) <= 2 * 2.0 ** -8 * 4.0


def test_refusals(dv):
    table, caches, q, _ = make(1, [1], [20], 4, 2, 64, 16, BF, BF, False)
    pc = dv.PagedCache(caches[0], caches[1], table)
    ln = torch.tensor([20], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        dv.paged_attention(pc, q.float(), ln)
    with pytest.raises(TypeError):
        dv.paged_attention(pc, q.half(), ln)
    with pytest.raises(TypeError):
        dv.paged_attention(pc, q, ln.long())
    with pytest.raises(ValueError):
        dv.paged_attention(pc, q[..., :32], ln)
    with pytest.raises(ValueError):
        dv.paged_attention(pc, q, ln[:0])
    with pytest.raises(ValueError):
        dv.paged_attention(pc, q.transpose(1, 2).contiguous().transpose(1, 2), ln)
    with pytest.raises(ValueError):
        dv.paged_attention(pc, q, ln, out=torch.empty((2, 4, 64), dtype=BF, device=DEV))
    with pytest.raises(dv.DFlashError):
        dv.paged_attention(pc, q[:, :3], ln)
    with pytest.raises(dv.DFlashError):
        dv.paged_attention(pc, q, ln, scale=-1.0)
    with pytest.raises(dv.DFlashError):
        dv.paged_attention(pc, q, ln, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        dv.PagedCache(caches[0], caches[1].transpose(1, 2), table)
    with pytest.raises(ValueError):
        dv.PagedCache(caches[0], caches[1], table.long())
    with pytest.raises(ValueError):
        dv.PagedCache(caches[0], caches[1], table, k_scale=torch.ones(2, device=DEV))


def test_extents_of_one_and_no_tokens(dv):
    """Strides of extents of one do not matter; no tokens is no work."""
    table, caches, q, _ = make(17, [1], [12], 1, 1, 64, 16, BF, BF, False)
    ln = torch.tensor([12], dtype=torch.int32, device=DEV)
    one = [c[int(table[0, 0])][None] for c in caches]
    t0 = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    want = dv.paged_attention(dv.PagedCache(one[0], one[1], t0), q, ln)
    odd = [c.as_strided(c.shape, (3, 5, c.stride(2), 1), c.storage_offset()) for c in one]
    q1 = q.as_strided(q.shape, (7, 1, 1), q.storage_offset())
    assert torch.equal(dv.paged_attention(dv.PagedCache(odd[0], one[1], t0), q1, ln), want)
    none = dv.paged_attention(dv.PagedCache(one[0], one[1], t0), q[:0], ln)
    assert none.shape == (0, 1, 64)
    assert dv.kv_append(dv.PagedCache(one[0], one[1], t0), q[:0], q[:0], ln) is None
