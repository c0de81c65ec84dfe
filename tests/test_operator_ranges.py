"""Arguments at the ends of their ranges, checked on the host before any CUDA call
(fake pointers)."""
import ctypes

import pytest

import speculative_decoding_verification_83_gb300 as dv

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
