"""The training operators' C interface where the binding does not use it: results over
their inputs, outputs inside wider arrays, rows of no sequence left as they were, gradients
without the outputs' low bits, without an upstream gradient, one at a time."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
import training_refs as refs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
CODE = {BF: 0, HF: 2, F: 1}


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_83_gb300 as m

    m.build()
    m.load()
    assert (m.DFLASH_BF16, m.operators.DFLASH_F16, m.DFLASH_F32) == (CODE[BF], CODE[HF], CODE[F])
    return m


def outer(*arrays):
    """Token and head strides, one array behind the other."""
    s = [x for t in arrays for x in t.stride()[:2]]
    return (ctypes.c_int64 * len(s))(*s)


def at(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def scratch(size):
    return torch.empty(size, device=DEV, dtype=torch.uint8)


def randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


# ---- norms
@pytest.mark.parametrize("T,D,dtype", [(1, 64, BF), (37, 128, HF), (2500, 128, BF), (70, 256, BF)])
def test_norms_over_their_inputs(dv, T, D, dtype):
    """q_out over q and k_out over k, inside a fused projection whose values stay; then dq over dq_out, dk over dk_out."""
    lib, Hq, Hk, rot = dv.load(), 5, 2, D // 2
    qkv = randn(T, T, Hq + 2 * Hk, D).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    w = [1 + 0.2 * randn(s, D) for s in (1, 2)]
    pos = torch.arange(T, device=DEV, dtype=torch.int32) * 3
    phases = dv.rope_phases(1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot), DEV)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, *w)]
    want = dv.norm_rotate(*leaves, positions=pos, phases=phases, eps=1e-5)
    up = randn(3, T, Hq + Hk, D).to(dtype)
    grads = torch.autograd.grad(want, leaves, [up[:, :Hq], up[:, Hq:]])
    x, values = [t.clone() for t in (q, k)], v.clone()
    assert lib.dflash_norm_rotate(at(q), at(k), at(q), at(k), CODE[dtype], T, Hq, Hk, D, outer(q, k, q, k), at(w[0]), at(w[1]),
                                  CODE[F], 1e-5, at(pos), at(phases), rot, 0, stream()) == dv.OK
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, values)
    gq, gk = up[:, :Hq], up[:, Hq:]
    gw = [torch.empty(D, device=DEV) for _ in w]
    ws = scratch(lib.dflash_norm_workspace_bytes(D))

    def backward(*gw):
        return lib.dflash_norm_rotate_grad(at(x[0]), at(x[1]), at(gq), at(gk), at(gq), at(gk), CODE[dtype], T, Hq, Hk, D,
                                           outer(*x, gq, gk, gq, gk), at(w[0]), at(w[1]), at(gw[0]), at(gw[1]), CODE[F], 1e-5,
                                           at(pos), at(phases), rot, 0, at(ws), ws.numel(), stream())

    kept = up.clone()
    assert backward(*gw) == dv.OK
    assert all(torch.equal(a, b) for a, b in zip((gq, gk, *gw), grads))
    for i in range(2):  # one of the weights' gradients, or none
        up.copy_(kept)
        part = [torch.full((D,), 7.0, device=DEV) if j == i else None for j in range(2)]
        assert backward(*part) == dv.OK
        assert torch.equal(part[i], grads[2 + i]) and torch.equal(gq, grads[0]) and torch.equal(gk, grads[1])
    up.copy_(kept)
    assert backward(None, None) == dv.OK
    assert torch.equal(gq, grads[0]) and torch.equal(gk, grads[1])


# ---- attention
def batch(dv, qs, ks, nq, nk, Hq, Hk, D, dtype, causal=1, scale=None):
    return dv.training._Batch(at(qs), at(ks), qs.numel() - 1, nq, nk, Hq, Hk, D, CODE[dtype], causal, scale or D ** -0.5)


def starts(counts, first):
    return torch.tensor([first + sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device=DEV)


def wide(n, heads, D, dtype, value=7.0):
    """Heads in the middle of a wider array that holds one value."""
    whole = torch.full((n, heads + 3, D), value, device=DEV, dtype=dtype)
    return whole, whole[:, 1:1 + heads]


@pytest.mark.parametrize("cq,ck,D,dtype,low", [
    (*shape, t, low) for t, low in ((BF, False), (BF, True), (HF, False))  # (low bits are bf16's)
    for shape in (([9, 3], [12, 7], 64), ([9, 3], [12, 7], 128), ([300, 130], [200, 140], 128), ([257, 40], [400, 3], 64))])
def test_rows_of_no_sequence_stay(dv, cq, ck, D, dtype, low):
    """Without `fill`, rows in front of the first sequence and behind the last keep what they hold, and so does what
    lies between the outputs' heads."""
    lib, Hq, Hk, q0, k0 = dv.load(), 4, 2, 5, 3
    nq, nk = sum(cq) + 14, sum(ck) + 9
    q, k, v = (randn(i, n, h, D).to(dtype) for i, n, h in ((1, nq, Hq), (2, nk, Hk), (3, nk, Hk)))
    for t in (q, k, v):
        t[:3], t[-4:] = math.nan, math.inf
    qs, ks = starts(cq, q0), starts(ck, k0)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    whole, out = wide(nq, Hq, D, dtype)
    lse = torch.full((nq, Hq), 7.0, device=DEV)
    bits = torch.full((nq, Hq, D), 7, device=DEV, dtype=torch.int8) if low else None
    b = batch(dv, qs, ks, nq, nk, Hq, Hk, D, dtype)
    ws = scratch(lib.dflash_packed_workspace_bytes(ctypes.byref(b), 0))
    assert lib.dflash_packed_attention(ctypes.byref(b), at(q), at(k), at(v), at(out), outer(q, k, v, out), at(lse), at(bits), 0,
                                       at(ws), ws.numel(), at(status), stream()) == dv.OK
    end = q0 + sum(cq)
    for t in (out, lse) + ((bits,) if low else ()):
        assert (t[:q0] == 7).all() and (t[end:] == 7).all()
    assert (whole[:, 0] == 7).all() and (whole[:, 1 + Hq:] == 7).all()
    with torch.set_grad_enabled(low):  # (the kernel that keeps low bits is the one of calls with a gradient)
        want, wl = dv.packed_attention(q.clone().requires_grad_(low), k, v, qs, kv_start=ks, return_lse=True)
    assert torch.equal(out[q0:end], want[q0:end]) and torch.equal(lse[q0:end], wl[q0:end])
    assert not want[:q0].any() and not want[end:].any() and int(status) == 0


@pytest.mark.parametrize("cq,ck,D", [([9, 3], [12, 7], 64), ([300, 130], [200, 140], 128), ([257, 0, 40], [400, 30, 3], 64)])
@pytest.mark.parametrize("low", [True, False])
def test_gradients_left_and_without_low_bits(dv, cq, ck, D, low):
    """fill = 0, gradients inside wider arrays; without the outputs' low bits their rounding reaches dq and dk."""
    lib, Hq, Hk, q0, k0 = dv.load(), 4, 2, 5, 3
    nq, nk = sum(cq) + 14, sum(ck) + 9
    q, k, v, do = (randn(i, n, h, D).to(BF) for i, n, h in ((1, nq, Hq), (2, nk, Hk), (3, nk, Hk), (4, nq, Hq)))
    qs, ks = starts(cq, q0), starts(ck, k0)
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    out, lse = torch.empty((nq, Hq, D), device=DEV, dtype=BF), torch.empty((nq, Hq), device=DEV)
    bits = torch.empty((nq, Hq, D), device=DEV, dtype=torch.int8) if low else None
    b = batch(dv, qs, ks, nq, nk, Hq, Hk, D, BF)
    ws = scratch(lib.dflash_packed_workspace_bytes(ctypes.byref(b), 0))
    assert lib.dflash_packed_attention(ctypes.byref(b), at(q), at(k), at(v), at(out), outer(q, k, v, out), at(lse), at(bits), 1,
                                       at(ws), ws.numel(), at(status), stream()) == dv.OK
    (wq, dq), (wk, dk), (wv, dvv) = wide(nq, Hq, D, BF), wide(nk, Hk, D, BF), wide(nk, Hk, D, BF)
    ws = scratch(lib.dflash_packed_workspace_bytes(ctypes.byref(b), 1))
    assert lib.dflash_packed_attention_grad(ctypes.byref(b), at(q), at(k), at(v), at(out), at(lse), at(bits), at(do), at(dq),
                                            at(dk), at(dvv), outer(q, k, v, out, do, dq, dk, dvv), 0, at(ws), ws.numel(),
                                            at(status), stream()) == dv.OK
    for t, first, n in ((wq, q0, sum(cq)), (wk, k0, sum(ck)), (wv, k0, sum(ck))):
        assert (t[:first] == 7).all() and (t[first + n:] == 7).all() and (t[:, 0] == 7).all() and (t[:, -2:] == 7).all()
    assert int(status) == 0
    if low:  # as the binding calls it
        leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
        want = torch.autograd.grad(dv.packed_attention(*leaves, qs, kv_start=ks), leaves, do)
        for got, w, first, n in zip((dq, dk, dvv), want, (q0, k0, k0), (sum(cq), sum(ck), sum(ck))):
            assert torch.equal(got[first:first + n], w[first:first + n])
        return
    i, j = q0, k0
    for n, m in zip(cq, ck):
        t, s = slice(i, i + n), slice(j, j + m)
        want, bound = refs.attention_grad64(q[t].double(), k[s].double(), v[s].double(), D ** -0.5,
                                            refs.sees(n, m, True).to(DEV), do[t].double(), refs.U[BF], low=refs.U[BF] * 1.01)
        for got, where, w, e in zip((dq, dk, dvv), (t, s, s), want, bound):
            assert ((got[where].double() - w).abs() <= refs.rounded(w, e, BF)).all()
        i, j = i + n, j + m


# ---- cross entropy
@pytest.mark.parametrize("N,V,K", [(5, 300, 64), (200, 1001, 136)])
def test_upstream_gradients_and_one_gradient_alone(dv, N, V, K):
    """No upstream gradient (1), one that all rows share, one of every other value; statistics not asked for."""
    lib = dv.load()
    h, w = randn(1, N, K).to(BF), (randn(2, V, K) * 0.2).to(BF)
    labels = torch.arange(N, device=DEV, dtype=torch.int32) * 7 % V
    labels[1] = -1
    status = torch.zeros(1, device=DEV, dtype=torch.int32)
    head = at(h), K, at(w), K, N, V, K, at(labels), None
    loss, stats = torch.empty(N, device=DEV), torch.empty((N, 2), device=DEV)
    ws = scratch(lib.dflash_linear_entropy_workspace_bytes(N, V, K, 0))
    assert lib.dflash_linear_entropy(*head, at(loss), at(stats), at(ws), ws.numel(), at(status), stream()) == dv.OK
    alone = torch.empty(N, device=DEV)
    assert lib.dflash_linear_entropy(*head, at(alone), None, at(ws), ws.numel(), at(status), stream()) == dv.OK
    assert torch.equal(loss, alone) and torch.equal(loss, dv.linear_cross_entropy(h, w, labels))
    ws = scratch(lib.dflash_linear_entropy_workspace_bytes(N, V, K, 1))

    def backward(up, step, want_h=True, want_w=True):
        dh = torch.full((N, K), 7.0, device=DEV, dtype=BF) if want_h else None
        dw = torch.full((V, K), 7.0, device=DEV, dtype=BF) if want_w else None
        assert lib.dflash_linear_entropy_grad(*head, at(stats), at(up), step, at(dh), at(dw), at(ws), ws.numel(), at(status),
                                              stream()) == dv.OK
        return dh, dw

    x, y = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    two = randn(5, 2 * N)
    for up, step, same in ((None, 1, torch.ones(N, device=DEV)), (None, 0, torch.ones(N, device=DEV)),
                           (torch.full((1,), 0.3, device=DEV), 0, torch.full((N,), 0.3, device=DEV)),
                           (two, 2, two[::2].contiguous())):
        want = torch.autograd.grad(dv.linear_cross_entropy(x, y, labels), (x, y), same)
        got = backward(up, step)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(backward(up, step, want_w=False)[0], want[0])
        assert torch.equal(backward(up, step, want_h=False)[1], want[1])
    assert int(status) == 0
