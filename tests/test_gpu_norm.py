"""norm_rotate and kv_append with norms against the definitions in 64 bits:
types, head sizes, rotations, strides, odd counts, gradients, captured calls."""
import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    return m


def frequencies(rot):
    return 1e5 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else None


def inputs(seed, T, Hq, Hk, D, dtype, wtype, far=1000):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    qkv = (torch.randn((T, Hq + 2 * Hk, D), generator=g, device=DEV) * 1.5).to(dtype)
    w = [(1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(wtype) for _ in range(2)]
    pos = torch.randint(-far, far, (T,), generator=g, device=DEV).to(torch.int32)
    up = [torch.randn((T, h, D), generator=g, device=DEV).to(dtype) for h in (Hq, Hk)]
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], w, pos, up


CASES = [
    # tokens, q heads, k heads, head_dim, rot, interleaved, dtype, weights' dtype, farthest position
    (1, 1, 1, 64, 64, False, BF, BF, 10), (1, 64, 8, 128, 128, False, BF, F, 100000), (3, 5, 3, 128, 64, True, HF, HF, 50),
    (33, 8, 8, 256, 256, False, BF, BF, 4000), (257, 7, 1, 64, 16, True, BF, F, 1000), (5, 3, 1, 256, 48, False, HF, F, 2 ** 30),
    (100, 40, 8, 128, 0, False, BF, BF, 10), (9, 2, 2, 64, 48, False, HF, HF, 9), (2449, 2, 1, 64, 64, False, BF, BF, 5000),
]


@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter,dtype,wtype,far", CASES)
def test_values_and_gradients(dv, T, Hq, Hk, D, rot, inter, dtype, wtype, far):
    q, k, _, w, pos, up = inputs(T + D, T, Hq, Hk, D, dtype, wtype, far)
    freq = frequencies(rot)
    ph = dv.rope_phases(freq, DEV) if rot else None
    leaves = [t.detach().requires_grad_(True) for t in (q, k, *w)]
    got = dv.norm_rotate(*leaves, positions=pos, phases=ph, interleaved=inter, eps=1e-5)
    grads = torch.autograd.grad(got, leaves, up)
    f = None if freq is None else freq.to(DEV)
    for i in range(2):
        x, wt = leaves[i].detach().double(), w[i].double()
        y, e = refs.norm64(x, wt, 1e-5, pos, f, inter)
        assert ((got[i].double() - y).abs() <= refs.rounded(y, e, dtype)).all()
        assert got[i].is_contiguous() and got[i].dtype == dtype
        dx, ex, dw, ew = refs.norm_grad64(x, wt, 1e-5, pos, f, inter, up[i].double())
        assert ((grads[i].double() - dx).abs() <= refs.rounded(dx, ex, dtype)).all()
        assert ((grads[2 + i].double() - dw).abs() <= refs.rounded(dw, ew, wtype)).all()
        assert grads[2 + i].dtype == wtype


def test_repeats_bit_for_bit(dv):
    q, k, _, w, pos, up = inputs(1, 3000, 6, 2, 128, BF, F)
    ph = dv.rope_phases(frequencies(128), DEV)
    runs = []
    for _ in range(3):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, *w)]
        got = dv.norm_rotate(*leaves, positions=pos, phases=ph)
        runs.append(list(got) + list(torch.autograd.grad(got, leaves, up)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_one_array_no_weights_no_rotation(dv):
    q, k, _, w, pos, up = inputs(2, 17, 4, 2, 128, BF, BF)
    one, none = dv.norm_rotate(q)
    assert none is None
    y, e = refs.norm64(q.double(), torch.ones(128, device=DEV, dtype=torch.float64), 1e-6, None, None, False)
    assert ((one.double() - y).abs() <= refs.rounded(y, e, BF)).all()
    both = dv.norm_rotate(q, k)
    assert torch.equal(both[0], one)
    none, two = dv.norm_rotate(None, k)
    assert none is None and torch.equal(two, both[1])
    # a gradient of one result alone, and of the weights alone
    kk, wk = k.detach().requires_grad_(True), w[1].requires_grad_(True)
    got = dv.norm_rotate(q, kk, w[0], wk)
    dk, = torch.autograd.grad(got[1], [kk], up[1])
    got = dv.norm_rotate(q, k, w[0], wk)
    dw, = torch.autograd.grad(got[1], [wk], up[1])
    rx, ex, rw, ew = refs.norm_grad64(k.double(), w[1].detach().double(), 1e-6, None, None, False, up[1].double())
    assert ((dk.double() - rx).abs() <= refs.rounded(rx, ex, BF)).all()
    assert ((dw.double() - rw).abs() <= refs.rounded(rw, ew, BF)).all()


def test_no_tokens(dv):
    q = torch.zeros((0, 4, 64), device=DEV, dtype=BF, requires_grad=True)
    w = torch.ones(64, device=DEV, dtype=F, requires_grad=True)
    out, _ = dv.norm_rotate(q, None, w)
    dq, dw = torch.autograd.grad(out, [q, w], torch.zeros_like(out))
    assert out.shape == (0, 4, 64) and dq.shape == (0, 4, 64) and not dw.any()


def test_gradients_of_no_tokens_by_the_library(dv):
    """No tokens, positions or phases: the weights' gradients are 0."""
    lib = dv.load()
    gw = [torch.full((128,), 7.0, device=DEV) for _ in range(2)]
    w = torch.ones(128, device=DEV)
    size = lib.dflash_norm_workspace_bytes(128)
    ws = torch.empty(size, device=DEV, dtype=torch.uint8)
    code = lib.dflash_norm_rotate_grad(None, None, None, None, None, None, dv.DFLASH_BF16, 0, 4, 2, 128, None, w.data_ptr(),
                                       w.data_ptr(), gw[0].data_ptr(), gw[1].data_ptr(), dv.DFLASH_F32, 1e-6, None, None, 64,
                                       0, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert code == dv.OK and not gw[0].any() and not gw[1].any()


def test_many_heads(dv):
    """A token's heads are found by a multiplication: at counts where 32 bits would not do for it."""
    q = torch.randn((3, 40001, 64), device=DEV).to(BF)
    w = torch.ones(64, device=DEV)
    out, _ = dv.norm_rotate(q, None, w)
    want = q.double() * torch.rsqrt(q.double().square().mean(-1, keepdim=True) + 1e-6)
    assert ((out.double() - want).abs() <= refs.rounded(want, 32 * refs.F32 * want.abs(), BF)).all()


def test_strides_broadcast_inputs_and_upstream(dv):
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    x = torch.randn((3, 24, 128), generator=g, device=DEV).to(BF)
    heads_first = x.transpose(0, 1)  # [24 tokens, 3 heads, 128]
    out, _ = dv.norm_rotate(heads_first)
    assert torch.equal(out, dv.norm_rotate(heads_first.contiguous())[0])
    one = x[:1, :1].detach().requires_grad_(True)
    out, _ = dv.norm_rotate(one.expand(5, 7, 128))
    assert torch.equal(out, dv.norm_rotate(one.expand(5, 7, 128).contiguous())[0])
    grad, = torch.autograd.grad(out.sum(), one)  # an upstream gradient without strides
    _, _, _, _ = refs.norm_grad64(one.detach().double(), torch.ones(128, device=DEV).double(), 1e-6, None, None, False,
                                  torch.full((1, 1, 128), 35.0, device=DEV).double())
    dx, ex, _, _ = refs.norm_grad64(one.detach().double(), torch.ones(128, device=DEV).double(), 1e-6, None, None, False,
                                    torch.full((1, 1, 128), 35.0, device=DEV).double())
    # 35 rounded gradients are added up (in bf16 at worst, 35 roundings)
    assert ((grad.double() - dx).abs() <= 35 * refs.U[BF] * (dx.abs() + ex) + 35 * ex + 36 * 2.0 ** -8 * dx.abs().amax()).all()


def test_zero_and_odd_values(dv):
    x = torch.zeros((4, 1, 64), device=DEV, dtype=BF)
    x[1, 0, 3] = float("nan")
    x[2, 0, 5] = float("inf")
    x[3] = 1e-30
    out, _ = dv.norm_rotate(x, eps=1e-6)
    assert not out[0].any() and out[1].isnan().all()
    assert out[2, 0, 5].isnan() and torch.isfinite(out[3]).all()


@pytest.mark.parametrize("cache_dtype", [BF, torch.float8_e4m3fn])
@pytest.mark.parametrize("T,D,rot,inter", [(1, 64, 64, False), (5, 128, 64, True), (70, 128, 128, False), (33, 256, 0, False)])
def test_append_norms_on_the_way(dv, cache_dtype, T, D, rot, inter):
    """The same heads as norm_rotate's, in the cache; without eps nothing is normed."""
    Hq, Hk, page = 6, 2, 16
    q, k, v, w, _, _ = inputs(T, T, Hq, Hk, D, BF, BF)
    lens = torch.arange(T, device=DEV, dtype=torch.int32) % 40
    ph = dv.rope_phases(frequencies(rot), DEV) if rot else None
    table = torch.arange(T * 3, device=DEV, dtype=torch.int32).view(T, 3)
    caches = [torch.zeros((T * 3, Hk, page, D), device=DEV, dtype=cache_dtype) for _ in range(2)]
    cache = dv.PagedCache(*caches, table)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    got = dv.kv_append(cache, k, v, lens, q=q, phases=ph, interleaved=inter, eps=1e-6, q_weight=w[0], k_weight=w[1],
                       status=status)
    wq, wk = dv.norm_rotate(q, k, *w, positions=lens, phases=ph, interleaved=inter, eps=1e-6)
    assert int(status) == 0
    f = None if not rot else frequencies(rot).to(DEV)
    for x, y, wt in ((q, got, w[0]), (k, None, w[1])):
        r, e = refs.norm64(x.double(), wt.double(), 1e-6, lens, f, inter)
        if y is None:
            y = caches[0].view(torch.uint8) if cache_dtype != BF else caches[0]
            y = torch.stack([y[table[t, int(lens[t]) // page], :, int(lens[t]) % page] for t in range(T)])
            y = y.view(cache_dtype) if cache_dtype != BF else y
            bound = refs.rounded(r, e, BF) if cache_dtype == BF else e + 2.0 ** -4 * (r.abs() + e) + 2.0 ** -10
        else:
            bound = refs.rounded(r, e, BF)
        assert ((y.double() - r).abs() <= bound).all()
    assert ((got.double() - wq.double()).abs() <= 2.0 ** -7 * wq.double().abs() + 1e-30).all()  # a rounding either way
    stored = caches[1].float()[table[torch.arange(T), (lens // page).long()].long(), :, (lens % page).long()]
    assert torch.equal(stored, v.to(cache_dtype).float())


def test_captured_and_replayed(dv):
    q, k, _, w, pos, up = inputs(8, 50, 4, 2, 128, BF, F)
    ph = dv.rope_phases(frequencies(128), DEV)
    leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, *w)]

    def step():
        got = dv.norm_rotate(*leaves, positions=pos, phases=ph)
        return [*(t.detach() for t in got), *torch.autograd.grad(got, leaves, up)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        for t in leaves[:2]:
            t.mul_(2.0)  # the norm takes it out again, up to eps
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got[:2], want[:2]):
        assert (a.double() - b.double()).abs().amax() <= 2.0 ** -6 * b.double().abs().amax()
    assert not torch.equal(got[2], want[2])
