"""packed_attention against the definitions in 64 bits: lengths, masks that leave
rows empty, head groups, strides, values that are not finite in places that are not
seen, gradients, captured calls."""
import math

import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

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


def starts(counts, first=0):
    s = [first]
    for n in counts:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device=DEV)


def inputs(seed, nq, nk, Hq, Hk, D, dtype, q_scale=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q = (torch.randn((nq, Hq, D), generator=g, device=DEV) * q_scale).to(dtype)
    k, v = (torch.randn((nk, Hk, D), generator=g, device=DEV).to(dtype) for _ in range(2))
    do = torch.randn((nq, Hq, D), generator=g, device=DEV).to(dtype)
    return q, k, v, do


def check(out, lse, grads, q, k, v, do, cq, ck, scale, causal, q0=0, k0=0):
    """Every sequence's outputs (and gradients) against the definition."""
    u = refs.U[q.dtype]
    i, j = q0, k0
    for n, m in zip(cq, ck):
        t, s = slice(i, i + n), slice(j, j + m)
        mask = refs.sees(n, m, causal).to(DEV)
        a = [x.detach().double() for x in (q[t], k[s], v[s])]
        o, l, eo, el, _, _ = refs.attention64(*a, scale, mask, u)
        assert ((out[t].double() - o).abs() <= refs.rounded(o, eo, q.dtype)).all()
        if lse is not None:
            fine = l.isfinite()
            assert torch.equal(fine, lse[t].isfinite()) and (lse[t][~fine] == -math.inf).all()
            assert ((lse[t].double() - l).abs()[fine] <= (el + 4 * refs.F32 * l.abs())[fine]).all()
        if grads is not None:
            want, bound = refs.attention_grad64(*a, scale, mask, do[t].double(), u)
            for got, at, w, b in zip(grads, (t, s, s), want, bound):
                assert ((got[at].double() - w).abs() <= refs.rounded(w, b, q.dtype)).all()
        i, j = i + n, j + m


CASES = [
    # queries, keys (None: the same), q heads, kv heads, head_dim, causal
    ([1], None, 1, 1, 64, True), ([1, 1, 1], None, 8, 2, 128, True), ([7], None, 32, 8, 128, True),
    ([127, 1, 128, 129], None, 4, 2, 64, True), ([255, 256, 257], None, 2, 2, 128, True), ([513], None, 3, 1, 128, True),
    ([5, 0, 300, 2], None, 8, 8, 64, False), ([0, 0, 9], None, 4, 1, 128, False), ([700], None, 5, 5, 128, False),
    ([16, 16, 16], [300, 1, 129], 8, 2, 128, True), ([100, 40], [30, 500], 4, 4, 64, True),
    ([64, 3, 130], [0, 200, 131], 6, 2, 128, True), ([20, 200], [0, 333], 16, 2, 64, False), ([1, 1], [1000, 257], 8, 1, 128, True),
    ([128] * 5, [128] * 5, 2, 1, 128, True), ([384], [640], 2, 1, 64, True),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("cq,ck,Hq,Hk,D,causal", CASES)
def test_values(dv, cq, ck, Hq, Hk, D, causal, dtype):
    q, k, v, do = inputs(len(cq) + sum(cq), sum(cq), sum(ck or cq), Hq, Hk, D, dtype)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    args = dict(kv_start=None if ck is None else starts(ck), causal=causal, status=status)
    out, lse = dv.packed_attention(q, k, v, starts(cq), return_lse=True, **args)
    check(out, lse, None, q, k, v, do, cq, ck or cq, D ** -0.5, causal)
    assert torch.equal(out, dv.packed_attention(q, k, v, starts(cq), **args)) and int(status) == 0


@pytest.mark.parametrize("cq,ck,Hq,Hk,D,causal", CASES)
def test_gradients(dv, cq, ck, Hq, Hk, D, causal):
    q, k, v, do = inputs(len(cq) + sum(cq), sum(cq), sum(ck or cq), Hq, Hk, D, BF)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    for t in (q, k, v):
        t.requires_grad_(True)
    out = dv.packed_attention(q, k, v, starts(cq), kv_start=None if ck is None else starts(ck), causal=causal, status=status)
    grads = torch.autograd.grad(out, (q, k, v), do)
    check(out.detach(), None, grads, q, k, v, do, cq, ck or cq, D ** -0.5, causal)
    assert int(status) == 0


@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_sharp_and_flat_scores(dv, scale):
    """Scores that one key rules, and scores that hardly differ; far references move a row's scale."""
    cq = [300, 70]
    q, k, v, do = inputs(3, 370, 370, 4, 2, 128, BF, 1.0)
    k[150:160] *= 3.0
    for t in (q, k, v):
        t.requires_grad_(True)
    out, lse = dv.packed_attention(q, k, v, starts(cq), scale=scale, return_lse=True)
    grads = torch.autograd.grad(out, (q, k, v), do)
    check(out.detach(), lse, grads, q, k, v, do, cq, cq, scale, True)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rising_scores(dv, dtype):
    """Every tile's scores lie far above those of the tiles before it."""
    n, D = 700, 64
    q, k, v, do = inputs(5, n, n, 2, 1, D, dtype, 1.0)
    q[:, :, 0] = 8.0
    k[:, :, 0] = (torch.arange(n, device=DEV)[:, None] / 20.0).to(dtype)
    out, lse = dv.packed_attention(q, k, v, starts([n]), scale=1.0, causal=False, return_lse=True)
    check(out, lse, None, q, k, v, do, [n], [n], 1.0, False)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("cq,ck,Hq,Hk,D,causal", [
    ([1], None, 8, 1, 64, True), ([33], None, 10, 2, 128, True), ([64], None, 64, 8, 64, True), ([65], None, 5, 1, 128, True),
    ([64], None, 65, 5, 128, False), ([1] * 63, None, 4, 2, 64, True), ([1] * 64, None, 4, 2, 128, True),
    ([3, 0, 17, 9], [20, 5, 1, 38], 6, 3, 128, True), ([2, 40, 0], [0, 31, 33], 4, 4, 64, False)])
def test_few_words(dv, cq, ck, Hq, Hk, D, causal, dtype):
    """Short prompts, at the sizes at which another kernel takes over, between rows of no sequence."""
    nq, nk = sum(cq) + 3, sum(ck or cq) + 3
    q, k, v, do = inputs(nq + Hq, nq, nk, Hq, Hk, D, dtype)
    for t in (q, k, v):
        t[:1], t[-2:] = math.nan, math.inf
    qs, ks = starts(cq, 1), starts(ck or cq, 1)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)

    def run():
        return dv.packed_attention(q, k, v, qs, kv_start=ks, causal=causal, return_lse=True, status=status)

    out, lse = run()
    check(out, lse, None, q, k, v, do, cq, ck or cq, D ** -0.5, causal, 1, 1)
    for rows in (slice(0, 1), slice(-2, None)):
        assert not out[rows].any() and (lse[rows] == -math.inf).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], lse) and int(status) == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_few_words_beside_values_that_are_not_seen(dv, bad):
    q, k, v, do = inputs(4, 50, 50, 4, 2, 64, BF)
    clean, lse = dv.packed_attention(q, k, v, starts([20, 10, 20]), return_lse=True)
    k[20:30], v[20:30], q[20:30], v[45, 1, 5] = bad, bad, bad, bad
    out, lse2 = dv.packed_attention(q, k, v, starts([20, 10, 20]), return_lse=True)
    same = torch.ones((50, 4, 64), device=DEV, dtype=torch.bool)
    same[20:30], same[45:, 2:, 5] = False, False
    assert torch.equal(out[same], clean[same]) and torch.equal(lse2[:20], lse[:20]) and torch.equal(lse2[30:], lse[30:])
    hit = out[45:, 2:, 5].float()
    assert hit.isnan().all() if math.isnan(bad) else (hit == bad).all()


def test_strides_and_fused_projections(dv):
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    cq, Hq, Hk, D = [130, 61], 6, 2, 128
    qkv = torch.randn((191, Hq + 2 * Hk, D), generator=g, device=DEV).to(BF)
    parts = [qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]]
    want = dv.packed_attention(*(t.contiguous() for t in parts), starts(cq))
    assert torch.equal(dv.packed_attention(*parts, starts(cq)), want)
    first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in parts]  # heads outside tokens
    assert torch.equal(dv.packed_attention(*first, starts(cq)), want)
    do = torch.randn((191, Hq, D), generator=g, device=DEV).to(BF)
    grads = []
    for p, up in ((parts, do), (first, do.transpose(0, 1).contiguous().transpose(0, 1)),
                  ([t.contiguous() for t in parts], torch.stack([do, do], -1)[..., 0])):
        leaves = [t.detach().requires_grad_(True) for t in p]
        grads.append(torch.autograd.grad(dv.packed_attention(*leaves, starts(cq)), leaves, up))
    for other in grads[1:]:
        assert all(torch.equal(a, b) for a, b in zip(grads[0], other))


def test_broadcast_keys(dv):
    """One head's keys and values for every head, as an expanded view: the gradients add up over it."""
    q, k, v, do = inputs(7, 90, 90, 4, 1, 64, BF)
    for t in (q, k, v):
        t.requires_grad_(True)
    wide = dv.packed_attention(q, k.expand(90, 4, 64), v.expand(90, 4, 64), starts([90]))
    assert torch.equal(wide, dv.packed_attention(q, k, v, starts([90])))
    dk, = torch.autograd.grad(wide, [k], do)
    (_, want, _), (_, bound, _) = refs.attention_grad64(q.detach().double(), k.detach().double(), v.detach().double(), 0.125,
                                                        refs.sees(90, 90, True).to(DEV), do.double(), refs.U[BF])
    # four rounded parts, added up in bf16
    parts = sum(refs.attention_grad64(q.detach()[:, h:h + 1].double(), k.detach().double(), v.detach().double(), 0.125,
                                      refs.sees(90, 90, True).to(DEV), do[:, h:h + 1].double(), refs.U[BF])[0][1].abs()
                for h in range(4))
    assert ((dk.double() - want).abs() <= bound + 5 * 2.0 ** -8 * (parts + bound)).all()


def test_rows_of_no_sequence(dv):
    """Rows in front of the first sequence and behind the last: outputs and gradients 0, whatever they hold."""
    q, k, v, do = inputs(8, 300, 260, 4, 2, 128, BF)
    qs, ks = starts([100, 120], 30), starts([90, 100], 20)
    for t, lo, hi in ((q, 30, 250), (do, 30, 250), (k, 20, 210), (v, 20, 210)):
        t[:lo], t[hi:] = math.nan, math.inf
    for t in (q, k, v):
        t.requires_grad_(True)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    out, lse = dv.packed_attention(q, k, v, qs, kv_start=ks, return_lse=True, status=status)
    grads = torch.autograd.grad(out, (q, k, v), do)
    check(out.detach(), lse, grads, q, k, v, do, [100, 120], [90, 100], 128 ** -0.5, True, 30, 20)
    assert not out[:30].any() and not out[250:].any() and (lse[:30] == -math.inf).all() and (lse[250:] == -math.inf).all()
    for g, lo, hi in zip(grads, (30, 20, 20), (250, 210, 210)):
        assert not g[:lo].any() and not g[hi:].any()
    assert int(status) == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_seen(dv, bad):
    """What a sequence holds that is not finite does not reach its neighbours, nor rows before it (causal). (The
    rows beside it come from another kernel, so they are held to the definition, not to equal bits.)"""
    cq = [100, 70, 130]
    q, k, v, do = inputs(9, 300, 300, 4, 2, 64, BF)
    k[100:170], v[100:170], q[100:170] = bad, bad, bad
    out, lse = dv.packed_attention(q, k, v, starts(cq), return_lse=True)
    for lo, hi in ((0, 100), (170, 300)):
        check(out[lo:hi], lse[lo:hi], None, q[lo:hi], k[lo:hi], v[lo:hi], do, [hi - lo], [hi - lo], 0.125, True)
    v[250, 1, 5] = bad
    odd, lse2 = dv.packed_attention(q, k, v, starts(cq), return_lse=True)
    assert ((lse2[170:] - lse[170:]).abs() <= 2.0 ** -18 * (1 + lse[170:].abs())).all()
    v[250, 1, 5] = 0.0  # beside it, all is as with any other value there
    o, _, e, _, _, _ = refs.attention64(q[170:].double(), k[170:].double(), v[170:].double(), 0.125,
                                        refs.sees(130, 130, True).to(DEV), refs.U[BF])
    rest = torch.ones((130, 4, 64), device=DEV, dtype=torch.bool)
    rest[80:, 2:, 5] = False
    assert ((odd[170:].double() - o).abs() <= refs.rounded(o, e, BF))[rest].all()
    hit = odd[250:, 2:, 5].float()
    assert hit.isnan().all() if math.isnan(bad) else (hit == bad).all()


def test_gradients_beside_values_that_are_not_seen(dv):
    cq = [100, 70, 130]
    q, k, v, do = inputs(10, 300, 300, 4, 2, 64, BF)

    def grads():
        leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
        return torch.autograd.grad(dv.packed_attention(*leaves, starts(cq)), leaves, do)

    for t in (q, k, v, do):
        t[100:170] = math.nan
    got = grads()
    check(dv.packed_attention(q, k, v, starts(cq))[:100], None, [g[:100] for g in got], q, k, v, do, [100], [100], 0.125, True)
    check(dv.packed_attention(q, k, v, starts(cq)), None, got, q, k, v, do, [130], [130], 0.125, True, 170, 170)
    do[200] = math.inf  # seen by the keys up to its own: the later keys' gradients stay sound
    got = grads()
    assert all(torch.isfinite(g[201:]).all() for g in got[1:]) and torch.isfinite(got[0][170:200]).all()
    assert not torch.isfinite(got[2][170:201]).any()


def test_bad_offsets_are_reported(dv):
    q, k, v, _ = inputs(11, 64, 64, 2, 1, 64, BF)
    for s in ([0, 40, 30, 64], [0, 20, 80, 90], [-5, 10, 20, 64]):
        status = torch.zeros(1, device=DEV, dtype=torch.int32)
        dv.packed_attention(q, k, v, torch.tensor(s, dtype=torch.int32, device=DEV), status=status)
        assert int(status) == dv.STATUS_BAD_LENGTH


def test_no_tokens(dv):
    q, k, v, do = inputs(12, 0, 0, 2, 1, 64, BF)
    out, lse = dv.packed_attention(q, k, v, starts([0, 0]), return_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    q, _, _, do = inputs(12, 9, 0, 2, 1, 64, BF)
    for t in (q, k, v):
        t.requires_grad_(True)
    out, lse = dv.packed_attention(q, k, v, starts([9]), kv_start=starts([0]), return_lse=True)
    dq, dk, dvv = torch.autograd.grad(out, (q, k, v), do)
    assert not out.any() and (lse == -math.inf).all() and not dq.any() and dk.shape == (0, 1, 64)
    q, k, v, _ = inputs(12, 0, 9, 2, 1, 64, BF)
    for t in (q, k, v):
        t.requires_grad_(True)
    out = dv.packed_attention(q, k, v, starts([0]), kv_start=starts([9]))
    _, dk, dvv = torch.autograd.grad(out, (q, k, v), torch.zeros_like(out))
    assert not dk.any() and not dvv.any()


def test_lse_beside_the_gradients(dv):
    """With and without lse the gradients are the same; lse itself carries none."""
    q, k, v, do = inputs(15, 70, 70, 4, 2, 64, BF)
    for t in (q, k, v):
        t.requires_grad_(True)
    alone = dv.packed_attention(q, k, v, starts([70]))
    out, lse = dv.packed_attention(q, k, v, starts([70]), return_lse=True)
    assert torch.equal(out, alone) and not lse.requires_grad and lse.shape == (70, 4)
    a, b = (torch.autograd.grad(o, (q, k, v), do) for o in (alone, out))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    out, lse = dv.packed_attention(q, k, v, starts([70]), return_lse=True)
    (out.float().sum() + lse.sum()).backward()
    assert q.grad.isfinite().all()


def test_repeats_bit_for_bit_on_any_stream(dv):
    cq = [400, 33, 250]
    q, k, v, do = inputs(13, 683, 683, 8, 2, 128, BF)
    runs = []
    for i in range(3):
        stream = torch.cuda.Stream() if i else torch.cuda.current_stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            leaves = [t.detach().requires_grad_(True) for t in (q, k, v)]
            out, lse = dv.packed_attention(*leaves, starts(cq), return_lse=True)
            runs.append([out.detach(), lse, *torch.autograd.grad(out, leaves, do)])
        stream.synchronize()
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_captured_and_replayed(dv):
    """Two captured graphs, replayed in turn with new contents and other offsets."""
    cq, other = [200, 100], [17, 283]
    graphs = []
    for seed in (14, 15):
        q, k, v, do = inputs(seed, 300, 300, 4, 2, 64, BF)
        leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
        s = starts(cq)

        def step(leaves=leaves, s=s, do=do):
            out, lse = dv.packed_attention(*leaves, s, return_lse=True)
            return [out.detach(), lse, *torch.autograd.grad(out, leaves, do)]

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got, step, s))
    for turn in range(2):
        for graph, got, step, s in graphs:
            graph.replay()
        for graph, got, step, s in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, step()))
            s.copy_(starts(other))
