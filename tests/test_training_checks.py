"""The training operators' argument checks: the library's on the host, before any
CUDA call (fake pointers), and the binding's on CPU tensors."""
import ctypes
import re

import pytest

import speculative_decoding_verification_83_gb300 as dv
from speculative_decoding_verification_83_gb300 import operators as ops
from speculative_decoding_verification_83_gb300 import training as tr

torch = pytest.importorskip("torch")

P, ODD = 1 << 20, (1 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    dv.build()
    return dv.load()


def array(strides):
    return (ctypes.c_int64 * len(strides))(*strides)


def norm(lib, q=P, k=P, qo=P, ko=P, dtype=0, tokens=2, hq=4, hk=2, dim=128, strides=(768, 128) * 2 + (512, 128) * 2, wq=P,
         wk=P, wtype=0, eps=1e-6, pos=P, phases=P, rot=128):
    return lib.dflash_norm_rotate(q, k, qo, ko, dtype, tokens, hq, hk, dim, array(strides), wq, wk, wtype, eps, pos, phases,
                                  rot, 0, None)


def norm_grad(lib, q=P, k=P, qo=P, ko=P, dtype=0, tokens=2, hq=4, hk=2, dim=128, strides=(768, 128) * 2 + (512, 128) * 2,
              wq=P, wk=P, wtype=0, eps=1e-6, pos=P, phases=P, rot=128, ws=P, nbytes=1 << 40):
    return lib.dflash_norm_rotate_grad(q, k, qo, ko, P, P, dtype, tokens, hq, hk, dim, array(tuple(strides) + (512, 128) * 2),
                                       wq, wk, None, None, wtype, eps, pos, phases, rot, 0, ws, nbytes, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=dv.DFLASH_F32), 1, "dtype"), (dict(dtype=7), 1, "dtype"), (dict(dim=96), 2, "head_dim"),
    (dict(dim=512), 2, "head_dim"), (dict(tokens=-1), 1, "tokens"), (dict(hq=0, hk=0), 1, "heads"), (dict(hk=-1), 1, "heads"),
    (dict(hq=1 << 20), 2, "heads"), (dict(tokens=(1 << 30) + 1), 2, "tokens"), (dict(wtype=dv.DFLASH_F16), 1, "weight_dtype"), (dict(wq=ODD), 1, "weights"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(eps=float("inf")), 1, "eps"),
    (dict(rot=24), 2, "rot_dim"), (dict(rot=144), 2, "rot_dim"), (dict(phases=None), 1, "phases"), (dict(pos=None), 1, "positions"),
    (dict(q=None), 1, "null q"), (dict(k=ODD), 1, "k must"), (dict(strides=(768, 128, 768, 100) + (512, 128) * 2), 1, "k: strides"),
    (dict(strides=(64, 128) + (768, 128) + (512, 128) * 2), 1, "q: strides"),
    (dict(strides=(-768, 128) + (768, 128) + (512, 128) * 2), 1, "q: strides"),
])
def test_norm_is_checked(lib, kw, code, word):
    for call in (norm, norm_grad):
        assert call(lib, **kw) == code
        assert word in lib.dflash_last_error().decode()


def test_norm_workspace_is_checked(lib):
    assert lib.dflash_norm_workspace_bytes(96) == 0
    need = lib.dflash_norm_workspace_bytes(128)
    for kw, word in ((dict(ws=None), "workspace"), (dict(nbytes=need - 1), "workspace"), (dict(ws=P + 16), "256-byte")):
        assert norm_grad(lib, **kw) == 1 and word in lib.dflash_last_error().decode()
    assert norm(lib, tokens=0, q=None, k=None) == 0


def cache(**kw):
    c = dict(k=P, v=P, page_table=P, k_scale=None, v_scale=None, page_stride=16 * 8 * 128, head_stride=16 * 128,
             slot_stride=128, table_stride=4, num_pages=10, page_size=16, kv_heads=8, head_dim=128, dtype=0, batch=2, max_pages=4)
    c.update(kw)
    return ops._CacheStruct(*[c[n] for n, _ in ops._CacheStruct._fields_])


@pytest.mark.parametrize("kw,word", [(dict(eps=-1.0), "eps"), (dict(eps=float("inf")), "eps"), (dict(wtype=2), "weight_dtype"),
                                     (dict(wq=ODD), "weights"), (dict(k=None), "null k"), (dict(lens=None), "null")])
def test_append_with_norms_is_checked(lib, kw, word):
    a = dict(k=P, lens=P, wq=P, wtype=1, eps=1e-6)
    a.update(kw)
    c = cache()
    rc = lib.dflash_kv_append_norm(ctypes.byref(c), a["k"], P, P, P, 0, 2, 16, array((1024, 128) * 4), a["lens"], None, a["wq"],
                                   P, a["wtype"], a["eps"], P, 128, 0, None, None)
    assert rc == 1 and word in lib.dflash_last_error().decode()


def packed(**kw):
    b = dict(q_start=P, kv_start=P, batch=2, q_tokens=10, kv_tokens=12, q_heads=8, kv_heads=2, head_dim=128, dtype=0, causal=1,
             scale=0.1)
    b.update(kw)
    return tr._Batch(*[b[n] for n, _ in tr._Batch._fields_])


def attend(lib, b=None, q=P, k=P, v=P, out=P, strides=(1024, 128) + (256, 128) * 2 + (1024, 128), low=None, ws=P,
           nbytes=1 << 40):
    b = packed() if b is None else b
    return lib.dflash_packed_attention(ctypes.byref(b), q, k, v, out, array(strides), None, low, 0, ws, nbytes, None, None)


def attend_grad(lib, b=None, q=P, k=P, v=P, out=P, lse=P, strides=(1024, 128) + (256, 128) * 2 + (1024, 128), ws=P,
                nbytes=1 << 40):
    b = packed() if b is None else b
    more = (1024, 128) * 2 + (256, 128) * 2
    return lib.dflash_packed_attention_grad(ctypes.byref(b), q, k, v, out, lse, None, P, P, P, P, array(tuple(strides) + more),
                                            0, ws, nbytes, None, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(q_start=None), 1, "null"), (dict(kv_start=None), 1, "null"), (dict(dtype=1), 1, "dtype"),
    (dict(head_dim=256), 2, "head_dim"), (dict(head_dim=32), 2, "head_dim"), (dict(batch=0), 1, "batch"),
    (dict(batch=2049), 1, "batch"), (dict(q_tokens=-1), 1, "q_tokens"), (dict(kv_tokens=(1 << 24) + 1), 1, "kv_tokens"),
    (dict(q_heads=9), 1, "q_heads"), (dict(kv_heads=0), 1, "q_heads"), (dict(q_heads=2048), 2, "q_heads"),
    (dict(scale=0.0), 1, "scale"), (dict(scale=-1.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
])
def test_packed_batch_is_checked(lib, kw, code, word):
    b = packed(**kw)
    for call in (attend, attend_grad):
        assert call(lib, b=b) == code
        assert word in lib.dflash_last_error().decode()
    assert lib.dflash_packed_workspace_bytes(ctypes.byref(b), 0) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(q=None), "null q"), (dict(k=ODD), "k must"), (dict(v=None), "null v"), (dict(out=ODD), "out must"),
    (dict(strides=(1024, 100) + (256, 128) * 2 + (1024, 128)), "q: strides"),
    (dict(strides=(1024, 128) + (256, 64) + (256, 128) + (1024, 128)), "k: strides"),
    (dict(strides=(1024, 128) + (256, 128) + (0, 128) + (1024, 128)), "v: strides"),
    (dict(ws=None), "workspace"), (dict(nbytes=100), "workspace"), (dict(ws=P + 64), "256-byte"),
])
def test_packed_arrays_are_checked(lib, kw, word):
    for call in (attend, attend_grad):
        assert call(lib, **kw) == 1
        assert word in lib.dflash_last_error().decode()


def test_packed_gradient_is_bf16(lib):
    assert attend_grad(lib, b=packed(dtype=dv.DFLASH_F16)) == 2 and b"bf16" in lib.dflash_last_error()
    assert attend_grad(lib, lse=None) == 1 and b"lse" in lib.dflash_last_error()
    assert attend(lib, low=ODD) == 1 and b"out_low" in lib.dflash_last_error()
    assert attend(lib, b=packed(dtype=dv.DFLASH_F16), low=P) == 1 and b"out_low" in lib.dflash_last_error()
    assert attend(lib, b=packed(q_tokens=0), q=None, out=None) == 0


def entropy(lib, h=P, w=P, hs=64, wst=64, rows=4, V=100, K=64, labels=P, loss=P, stats=P, ws=P, nbytes=1 << 40):
    return lib.dflash_linear_entropy(h, hs, w, wst, rows, V, K, labels, None, loss, stats, ws, nbytes, None, None)


def entropy_grad(lib, h=P, w=P, hs=64, wst=64, rows=4, V=100, K=64, labels=P, stats=P, up_stride=1, dh=P, dw=P, ws=P,
                 nbytes=1 << 40):
    return lib.dflash_linear_entropy_grad(h, hs, w, wst, rows, V, K, labels, None, stats, P, up_stride, dh, dw, ws, nbytes, None,
                                          None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), 1, "rows"), (dict(rows=(1 << 20) + 1), 1, "rows"), (dict(V=0), 1, "V="), (dict(V=(1 << 24) + 1), 1, "V="),
    (dict(K=0), 2, "K="), (dict(K=60, hs=64), 2, "K="), (dict(K=(1 << 16) + 8), 2, "K="), (dict(h=None), 1, "null"),
    (dict(w=None), 1, "null"), (dict(labels=None), 1, "null"), (dict(h=ODD), 1, "aligned"), (dict(w=ODD), 1, "aligned"),
    (dict(hs=32), 1, "strides"), (dict(wst=68), 1, "strides"), (dict(ws=None), 1, "workspace"), (dict(nbytes=8), 1, "workspace"),
    (dict(ws=P + 128), 1, "256-byte"), (dict(stats=P + 4), 1, "row_stats"),
])
def test_entropy_is_checked(lib, kw, code, word):
    for call in (entropy, entropy_grad):
        assert call(lib, **kw) == code
        assert word in lib.dflash_last_error().decode()


def test_entropy_edges(lib):
    assert entropy(lib, rows=0, h=None, labels=None, loss=None) == 0
    assert entropy(lib, loss=None) == 1 and b"loss" in lib.dflash_last_error()
    assert entropy_grad(lib, rows=0) == 1 and b"rows" in lib.dflash_last_error()
    assert entropy_grad(lib, dh=None, dw=None) == 0
    assert entropy_grad(lib, dh=ODD) == 1 and entropy_grad(lib, up_stride=-1) == 1
    for args in ((0, 10, 64), (10, 0, 64), (10, 10, 12), (1 << 21, 10, 64)):
        assert lib.dflash_linear_entropy_workspace_bytes(*args, 1) == 0


def test_workspaces_follow_the_sizes(lib):
    """The logits' gradients come in pieces: their workspace stays below the logits' size."""
    whole = 16384 * 248320 * 2
    assert lib.dflash_linear_entropy_workspace_bytes(16384, 248320, 1024, 1) < whole // 4
    assert lib.dflash_linear_entropy_workspace_bytes(1 << 20, 248320, 64, 0) == \
        lib.dflash_linear_entropy_workspace_bytes(1 << 14, 248320, 64, 0)  # rows go in runs of 2^14
    for n in (lib.dflash_packed_workspace_bytes(ctypes.byref(packed()), i) for i in (0, 1)):
        assert n > 0 and n % 256 == 0


# ---- the binding, on CPU tensors
def heads(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,error,word", [
    (lambda: dv.norm_rotate(None, None), ValueError, "neither"),
    (lambda: dv.norm_rotate(heads(2, 4, 64, dtype=torch.float32)), TypeError, "bfloat16 or float16"),
    (lambda: dv.norm_rotate(heads(2, 64)), ValueError, "shape"),
    (lambda: dv.norm_rotate(heads(2, 4, 64)), ValueError, "CUDA"),
    (lambda: dv.packed_attention(heads(2, 4, 64, dtype=torch.float32), heads(2, 2, 64), heads(2, 2, 64),
                                 torch.tensor([0, 2], dtype=torch.int32)), TypeError, "bfloat16 or float16"),
    (lambda: dv.packed_attention(heads(2, 4, 64), heads(2, 2, 64), heads(2, 2, 64), torch.tensor([0, 2], dtype=torch.int32)),
     ValueError, "CUDA"),
    (lambda: dv.packed_attention(heads(2, 4, 64, dtype=torch.float16).requires_grad_(True), heads(2, 2, 64), heads(2, 2, 64),
                                 torch.tensor([0, 2], dtype=torch.int32)), TypeError, "bfloat16 only"),
    (lambda: dv.linear_cross_entropy(heads(2, 64, dtype=torch.float32), heads(10, 64), torch.zeros(2, dtype=torch.int32)),
     TypeError, "bfloat16"),
    (lambda: dv.linear_cross_entropy(heads(2, 64), heads(10, 64), torch.zeros(2, dtype=torch.int32)), ValueError, "CUDA"),
    (lambda: dv.linear_cross_entropy(heads(2, 64), heads(10, 64), torch.zeros(2, dtype=torch.int32),
                                     row_weight=torch.ones(2, requires_grad=True)), ValueError, "row_weight"),
])
def test_binding_refuses(lib, call, error, word):
    with pytest.raises(error, match=word):
        call()


def test_every_launch_goes_through_the_device_check():
    """Calls run on their tensors' device, whichever is current."""
    with open(tr.__file__) as f:
        s = f.read()
    names = {"norm_rotate", "norm_rotate_grad", "packed_attention", "packed_attention_grad", "linear_entropy",
             "linear_entropy_grad"}
    found = re.findall(r"(_call\([\w.]+, )?(?:_ops\._library\(\)|lib)\.dflash_(\w+),", s)
    assert {n for c, n in found if c} == names and not [n for c, n in found if not c and n in names]
