"""The operators' argument checks: the library's on the host, before any CUDA
call (fake pointers), and the binding's on CPU tensors."""
import ctypes

import pytest

import speculative_decoding_verification_83_gb300 as dv
from speculative_decoding_verification_83_gb300 import operators as ops

torch = pytest.importorskip("torch")

P, ODD = 1 << 20, (1 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    dv.build()
    return dv.load()


def cache(**kw):
    c = dict(k=P, v=P, page_table=P, k_scale=None, v_scale=None, page_stride=16 * 8 * 128, head_stride=16 * 128,
             slot_stride=128, table_stride=4, num_pages=10, page_size=16, kv_heads=8, head_dim=128,
             dtype=dv.DFLASH_BF16, batch=2, max_pages=4)
    c.update(kw)
    return ops._CacheStruct(*[c[n] for n, _ in ops._CacheStruct._fields_])


def append(lib, c=None, k=P, v=P, q=P, qo=P, dtype=0, tokens=2, hq=16, strides=(1024, 128) * 4, lens=P, rot=128,
           phases=P):
    c = cache() if c is None else c
    return lib.dflash_kv_append(ctypes.byref(c), k, v, q, qo, dtype, tokens, hq, (ctypes.c_int64 * 8)(*strides), lens,
                                None, phases, rot, 0, None, None)


def attend(lib, c=None, q=P, out=P, dtype=0, tokens=2, hq=16, strides=(2048, 128) * 2, lens=P, scale=0.1, ws=P,
           nbytes=1 << 40):
    c = cache() if c is None else c
    return lib.dflash_paged_attention(ctypes.byref(c), q, out, None, dtype, tokens, hq, (ctypes.c_int64 * 4)(*strides),
                                      lens, None, scale, 1, ws, nbytes, None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(k=None), 1, "null"), (dict(page_table=None), 1, "null"),
    (dict(dtype=dv.DFLASH_F32), 1, "dtype"), (dict(dtype=dv.DFLASH_F16), 1, "dtype"),
    (dict(head_dim=96), 2, "head_dim"), (dict(head_dim=0), 2, "head_dim"),
    (dict(batch=0), 1, "batch"), (dict(batch=2049), 1, "batch"),
    (dict(num_pages=0), 1, "num_pages"), (dict(page_size=0), 1, "page_size"), (dict(max_pages=-1), 1, "max_pages"),
    (dict(kv_heads=0), 1, "kv_heads"), (dict(v=ODD), 1, "aligned"),
    (dict(slot_stride=100), 1, "stride"), (dict(head_stride=-128), 1, "stride"),
    (dict(page_stride=1 << 33), 2, "64 GiB"), (dict(table_stride=-1), 1, "table_stride"),
])
def test_cache_is_checked(lib, kw, code, word):
    for call in (append, attend):
        assert call(lib, c=cache(**kw)) == code
        assert word in lib.dflash_last_error().decode()


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=1), 1, "dtype"), (dict(tokens=-1), 1, "tokens"), (dict(tokens=3), 1, "q_start"),
    (dict(lens=None), 1, "null"), (dict(k=ODD), 1, "k must"), (dict(v=None), 1, "null v"),
    (dict(q=None), 1, "together"), (dict(hq=0), 1, "q_heads"),
    (dict(strides=(1024, 100) + (1024, 128) * 3), 1, "k: strides"),
    (dict(strides=(1024, 128) * 3 + (-8, 128)), 1, "q_out: strides"),
    (dict(rot=24), 2, "rot_dim"), (dict(rot=144), 2, "rot_dim"), (dict(phases=None), 1, "phases"),
])
def test_append_is_checked(lib, kw, code, word):
    assert append(lib, **kw) == code
    assert word in lib.dflash_last_error().decode()


@pytest.mark.parametrize("kw,code,word", [
    (dict(hq=12), 1, "q_heads"), (dict(hq=0), 1, "q_heads"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"), (dict(scale=float("inf")), 1, "scale"), (dict(lens=None), 1, "null"),
    (dict(q=ODD), 1, "q must"), (dict(out=None), 1, "null out"), (dict(strides=(2048, 128, 2048, 4)), 1, "out: strides"),
    (dict(ws=None), 1, "workspace"), (dict(nbytes=1000), 1, "workspace"), (dict(ws=P + 16), 1, "256-byte"),
    (dict(tokens=1 << 30), 2, "rows"),
])
def test_attention_is_checked(lib, kw, code, word):
    assert attend(lib, **kw) == code
    assert word in lib.dflash_last_error().decode()


def test_attention_workspace(lib):
    n = lib.dflash_attention_workspace_bytes(32, 128)
    assert n > 0 and lib.dflash_attention_workspace_bytes(2048, 256) > n
    assert lib.dflash_attention_workspace_bytes(0, 128) == 0
    assert lib.dflash_attention_workspace_bytes(4, 100) == 0
    with pytest.raises(dv.DFlashError):
        dv.attention_workspace_bytes(4, 100)


def distill(lib, name, z=P, stride=100, rows=2, V=100, dtype=0, ids=P, teacher=P, K=4, T=1.0, tail=None):
    tail = {"loss": (None, P, None, None, None), "grad": (None, P, None, 1, P, 100, None),
            "loss_grad": (None, P, P, 100, None, None)}[name] if tail is None else tail
    return getattr(lib, "dflash_distill_" + name)(z, stride, rows, V, dtype, ids, teacher, K, T, *tail)


@pytest.mark.parametrize("kw,word", [
    (dict(z=None), "null"), (dict(ids=None), "null"), (dict(teacher=None), "null"), (dict(rows=-1), "rows"),
    (dict(V=0), "V=0"), (dict(K=0), "K=0"), (dict(K=257), "K=257"), (dict(dtype=2), "dtype"),
    (dict(stride=-1), "stride"), (dict(T=0.0), "temperature"), (dict(T=float("nan")), "temperature"),
    (dict(T=float("inf")), "temperature"), (dict(T=-1.0), "temperature"), (dict(z=P + 1), "aligned"),
    (dict(z=P + 2, dtype=1), "aligned"),
])
@pytest.mark.parametrize("name", ["loss", "grad", "loss_grad"])
def test_distillation_is_checked(lib, name, kw, word):
    assert distill(lib, name, **kw) == dv.ERR_INVALID_ARG
    assert word in lib.dflash_last_error().decode()


def test_distillation_outputs_are_checked(lib):
    assert distill(lib, "loss", tail=(None, None, None, None, None)) == dv.ERR_INVALID_ARG
    assert distill(lib, "grad", tail=(None, None, None, 1, P, 100, None)) == dv.ERR_INVALID_ARG
    assert distill(lib, "grad", tail=(None, P, None, 1, P, 99, None))\
        == dv.ERR_INVALID_ARG
    assert distill(lib, "grad", tail=(None, P, P, -1, P, 100, None)) == dv.ERR_INVALID_ARG
    assert distill(lib, "loss_grad", tail=(None, P, None, 100, None, None)) == dv.ERR_INVALID_ARG
    assert distill(lib, "loss_grad", tail=(None, P, P + 1, 100, None, None)) == dv.ERR_INVALID_ARG


def test_empty_calls_do_nothing(lib):
    """No tokens, no rows: accepted without a launch (no GPU needed)."""
    assert append(lib, tokens=0, k=None, v=None) == 0
    assert attend(lib, tokens=0, q=None) == 0
    for name in ("loss", "grad", "loss_grad"):
        assert distill(lib, name, rows=0) == 0
        assert distill(lib, name, rows=0, z=None, ids=None, teacher=None,
                       tail={"loss": (None, None, None, None, None), "grad": (None, None, None, 1, None, 100, None),
                             "loss_grad": (None, None, None, 100, None, None)}[name]) == 0


def test_binding_refuses_before_the_library(lib):
    k = torch.zeros((4, 8, 16, 64), dtype=torch.bfloat16)
    t = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dv.PagedCache(k, k, t)
    with pytest.raises(TypeError, match="cache must be"):
        dv.PagedCache(k.float(), k.float(), t)
    with pytest.raises(ValueError, match="one dtype"):
        dv.PagedCache(k, k[:3], t)
    z, ids, lg = torch.zeros((2, 10)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        dv.distill_loss(z, ids, lg)
    with pytest.raises(TypeError, match="student"):
        dv.distill_loss(z.half(), ids, lg)
    with pytest.raises(ValueError, match="detach"):
        dv.distill_loss(z, ids, lg.requires_grad_(True))


def test_rope_phases_are_exact_fractions():
    """Each entry is round(w 2^64 / 2 pi): within half a unit of the exact
    fraction, so n * entry is within n / 2^65 of a turn."""
    from fractions import Fraction

    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937511")
    w = [1.0, 0.5, 1e-6, 123.25, 0.0] + [10000.0 ** (-2 * j / 128) for j in range(64)]
    got = dv.rope_phases(w, device="cpu")
    assert got.dtype == torch.int64 and got.numel() == len(w)
    for x, g in zip(w, got.tolist()):
        turn = Fraction(x) / two_pi
        turn -= turn.numerator // turn.denominator
        d = abs(Fraction(g % (1 << 64), 1 << 64) - turn)
        assert min(d, 1 - d) <= Fraction(1, 1 << 65)
    assert torch.equal(dv.rope_phases(torch.tensor(w, dtype=torch.float64), device="cpu"), got)
