"""Arguments at the ends of their ranges, checked on the host before any CUDA call
(fake pointers)."""
import ctypes

import pytest

import speculative_decoding_verification_83_gb300 as dv
from speculative_decoding_verification_83_gb300 import operators as ops

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    dv.build()
    return dv.load()


@pytest.mark.parametrize("name,tail", [("loss", (None, P, None, None, None)),
                                       ("grad", (None, P, None, 1, P, 100, None)),
                                       ("loss_grad", (None, P, P, 100, None, None))])
@pytest.mark.parametrize("T", [1e-45, 1e-40, 4e-39])
def test_temperatures_without_a_finite_inverse_are_refused(lib, name, tail, T):
    """1 / (T ln 2) scales every exponent: where it is infinite nothing is defined."""
    rc = getattr(lib, "dflash_distill_" + name)(P, 100, 2, 100, 0, P, P, 4, ctypes.c_float(T), *tail)
    assert rc == dv.ERR_INVALID_ARG and "temperature" in lib.dflash_last_error().decode()


@pytest.mark.parametrize("kv,hq", [(1 << 28, 0), (1 << 30, 0), (2 ** 31 - 1, 0), (8, 2 ** 31 - 1), (8, 1 << 24)])
def test_more_heads_than_a_grid_holds_are_refused(lib, kv, hq):
    """(Heads may share memory, so that their number has no other limit.)"""
    c = ops._CacheStruct(P, P, P, None, None, 16 * 128, 0, 128, 4, 10, 16, kv, 128, dv.DFLASH_BF16, 2, 4)
    q = P if hq else None
    rc = lib.dflash_kv_append(ctypes.byref(c), P, P, q, q, dv.DFLASH_BF16, 2, hq, (ctypes.c_int64 * 8)(*[128, 0] * 4), P,
                              None, None, 0, 0, None, None)
    assert rc == dv.ERR_UNSUPPORTED and "heads" in lib.dflash_last_error().decode()
