"""dflash_paged_attention where values of the cache are not finite, and where a
row's weights span many powers of 2: what a row sees decides its result, not
which kernel, tile, copy or SM took the key."""
import math

import pytest

torch = pytest.importorskip("torch")
from operator_refs import F32, U  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


class Case:
    """One request of L positions and n new tokens, 2 key/value heads."""

    def __init__(self, seed, L, n, G, D, dtype, cdt, page=16, H=2):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        width = -(-L // page)
        self.L, self.n, self.G, self.D, self.H, self.page, self.dtype = L, n, G, D, H, page, dtype
        self.table = torch.randperm(width, generator=g, device=DEV).view(1, width).to(torch.int32)
        self.k, self.v = (torch.randn((width, H, page, D), generator=g, device=DEV).to(cdt) for _ in range(2))
        self.q = torch.randn((n, H * G, D), generator=g, device=DEV).to(dtype)
        self.lens = torch.tensor([L], dtype=torch.int32, device=DEV)

    def put(self, cache, pos, value, head=slice(None), col=slice(None)):
        t = cache.view(torch.uint8) if cache.dtype == F8 else cache
        if cache.dtype == F8:
            value = torch.tensor(value, device=DEV).to(F8).view(torch.uint8)
        t[self.table[0, pos // self.page].long(), head, pos % self.page, col] = value

    def attend(self, dv, scales=(None, None), **kw):
        out, lse = dv.paged_attention(dv.PagedCache(self.k, self.v, self.table, *scales), self.q, self.lens,
                                      return_lse=True, **kw)
        return out.view(self.n, self.H, self.G, self.D), lse.view(self.n, self.H, self.G)


# n, G: 8 rows a head (the warps' products), then units of 32, 64 and 128 rows, and two units
ROWS = [(4, 2), (4, 6), (4, 12), (4, 24), (4, 40)]


TYPES = [(64, BF, BF), (128, BF, BF), (128, HF, HF), (256, BF, BF)]
TYPES8 = [(64, BF, F8), (128, HF, F8), (256, BF, F8)]
BAD = [(t, bad, r) for t in TYPES for bad in (NAN, INF, -INF) for r in ROWS[1:]] \
    + [(t, NAN, r) for t in TYPES8[:2] for r in ROWS[2:]]


@pytest.mark.parametrize("types,bad,rows", BAD)
def test_values_in_front_of_the_block_count(dv, types, bad, rows):
    """The block's tile also holds keys in front of the block, which every row
    sees: a value there that is not finite reaches every row."""
    (D, dtype, cdt), (n, G), L, col = types, rows, 200, 5
    tile = 64 if D == 256 else 128
    block = L - n
    for pos in (block - 1, block // tile * tile):
        c = Case(D + G, L, n, G, D, dtype, cdt)
        want, wl = c.attend(dv)
        c.put(c.v, pos, bad, head=1, col=col)
        got, gl = c.attend(dv)
        assert torch.equal(gl, wl)
        assert not bool(got[:, 1, :, col].float().isfinite().any()), (pos, got[:, 1, :, col])
        got[:, 1, :, col] = want[:, 1, :, col]
        assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", ROWS[1:])
@pytest.mark.parametrize("below", [40.0, 200.0])
def test_bad_values_of_other_rows_leave_weak_keys_alone(dv, D, n, G, below):
    """A tile's first half weighs e^-40 or (in 32 bits) nothing against the rest,
    and the block's last token's value is NaN: the tokens before it do not
    notice."""
    L = 64 if D == 256 else 128
    c = Case(G, L, n, G, D, BF, BF)
    c.q.zero_()
    c.q[..., 0] = D ** 0.5
    for pos in range(L // 2):
        c.put(c.k, pos, -below, col=0)
    want, wl = c.attend(dv)
    c.put(c.v, L - 1, NAN, col=slice(0, None, 3))
    got, gl = c.attend(dv)
    assert torch.equal(gl, wl) and torch.equal(got[:-1], want[:-1])
    assert bool(got[-1, :, :, ::3].isnan().all())
    got[-1, :, :, ::3] = want[-1, :, :, ::3]
    assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", ROWS[2:])
def test_bad_values_under_a_scale_of_zero(dv, D, n, G):
    """A head's values scaled by 0: zero for the rows that see finite values only."""
    c = Case(G, 128, n, G, D, BF, F8)
    scales = torch.ones(2, device=DEV), torch.tensor([0.0, 0.5], device=DEV)
    want, _ = c.attend(dv, scales)
    assert bool((want[:, 0] == 0).all())
    c.put(c.v, 127, NAN, col=slice(0, None, 3))
    got, _ = c.attend(dv, scales)
    assert torch.equal(got[:-1], want[:-1])
    assert bool(got[-1, :, :, ::3].isnan().all())


# the rest of the forms: the warps' products
WARPS = [(t, bad, ROWS[0]) for t in TYPES for bad in (NAN, INF, -INF)] \
    + [(t, NAN, r) for t in TYPES8 for r in (ROWS if t[0] == 256 else ROWS[:2])]


@pytest.mark.parametrize("types,bad,rows", WARPS)
def test_other_results_stay_as_they_are(dv, types, bad, rows):
    """A value that is not finite decides its own column of the rows that see it;
    every other result keeps its bits."""
    test_values_in_front_of_the_block_count(dv, types, bad, rows)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("n,G", [(1, 4)] + ROWS)
@pytest.mark.parametrize("L,page", [(300, 16), (70001, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_infinite_values_stay_infinite(dv, D, dtype, n, G, L, page, causal):
    """An infinite value that a row sees, at whatever weight, makes its result
    infinite; infinities of both signs, or a NaN, make it NaN. Over one SM and
    over many."""
    c = Case(D + G, L, n, G, D, dtype, dtype, page)
    want, wl = c.attend(dv, causal=causal)
    c.put(c.v, 3, INF, col=0)
    c.put(c.v, L // 2 + 1, -INF, col=1)
    c.put(c.v, 5, INF, col=2)
    c.put(c.v, L // 2, -INF, col=2)
    c.put(c.v, L // 3, INF, col=D - 1)
    c.put(c.v, 7, NAN, col=D - 2)
    got, gl = c.attend(dv, causal=causal)
    assert torch.equal(gl, wl)
    f = got.float()
    assert bool((f[..., 0] == INF).all()), f[..., 0]
    assert bool((f[..., 1] == -INF).all())
    assert bool(f[..., 2].isnan().all())
    assert bool((f[..., D - 1] == INF).all()) and bool(f[..., D - 2].isnan().all())
    for col in (0, 1, 2, D - 1, D - 2):
        got[..., col] = want[..., col]
    assert torch.equal(got, want)


@pytest.mark.parametrize("n,G", [(1, 4)] + ROWS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("below", [15.0, 60.0, 300.0])
def test_infinite_values_of_weak_keys_stay_infinite(dv, n, G, dtype, below):
    """The key of the infinite value weighs e^-15 to e^-300 of the rest: a finite
    score's weight is not zero, whatever type holds it."""
    D, L = 128, 400
    c = Case(G, L, n, G, D, dtype, dtype)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k[..., 0] = 0.0
    c.put(c.k, 9, -below, col=0)
    want, wl = c.attend(dv, scale=1.0)
    c.put(c.v, 9, INF, col=7)
    got, gl = c.attend(dv, scale=1.0)
    assert torch.equal(gl, wl) and bool((got[..., 7] == INF).all()), got[..., 7]
    got[..., 7] = want[..., 7]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,cdt", [(HF, HF), (BF, F8), (HF, F8), (BF, BF)])
@pytest.mark.parametrize("n,G", [(1, 4), (4, 6), (4, 12), (4, 24)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("below,sink", [(18.0, 0), (18.0, 15000), (12.0, 0)])
def test_many_keys_far_below_one(dv, dtype, cdt, n, G, D, below, sink):
    """One key outweighs each of 20000 others by e^12 or e^18 and has no value
    of its own: the result is what the others add up to. Weights are rounded by
    half a step of their own, in f16 (whose largest weight is 2^15 in the warps'
    products, and at first 2^7 on tensor memory) by no more than 2^-25 at the least.
    (300 requests share the pages, so that each unit lies in few SMs.)"""
    L, B = 20001, 300
    c = Case(1, L, n, G, D, dtype, cdt, page=64)
    c.q.zero_()
    c.q[..., 0] = 1.0
    for t, x in ((c.k, 0.0), (c.v, 1.0)):
        t.copy_(torch.full(t.shape, x, device=DEV).to(t.dtype))
    c.put(c.k, sink, below, col=0)
    c.put(c.v, sink, 0.0)
    c.table, c.lens, c.q = c.table.expand(B, -1).contiguous(), c.lens.expand(B).contiguous(), c.q.repeat(B, 1, 1)
    c.n *= B
    got, lse = c.attend(dv, scale=1.0, causal=False)
    rest = (L - 1) * math.exp(-below)
    want = rest / (1.0 + rest)
    # the weights' type (8-bit caches of up to 32 rows: f16), the output's, sums of L / 16 terms a lane
    up = U[HF] if cdt == F8 and n * G <= 32 else U[dtype]
    small = 0.0 if up != U[HF] else 2.0 ** (-40 if n * G <= (32 if cdt == F8 else 16) else -32)
    tol = max(up, small * math.exp(below)) + U[dtype] + 2 * ((L / 16 + 200) * F32 + 2.0 ** -21)
    err = (got.double() / want - 1.0).abs()
    assert float(err.max()) <= tol, (float(err.max()), tol)
    assert float((lse.double() - (below + math.log1p(rest))).abs().max()) <= 2 * tol
