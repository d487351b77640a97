"""Rows of linear attention at the C ABI, without a GPU.  The pointers are made up, so only
calls that fail validation or have nothing to do are made."""

import ctypes

import pytest

import rwkv_wkv7_delta_amd as wk
from tests.test_linattn_cpu import FAKE, L, LA_OK  # noqa: F401  (L: a fixture)

C = ctypes.byref


def test_clear_rest_refusals(L):
    def clear(desc=None, starts=FAKE, values=FAKE, queries=FAKE, keys=FAKE, decays=FAKE):
        d = None if desc is None else C(wk.LinattnDesc(**dict(LA_OK, packed=1, tokens=5, **desc)))
        return L.wkv7_linattn_clear_rest(d, starts, values, queries, keys, decays, None)

    assert clear() == wk.WKV7_ERR_INVALID_ARG
    padded = C(wk.LinattnDesc(**LA_OK))
    assert L.wkv7_linattn_clear_rest(padded, FAKE, FAKE, None, None, None, None) == wk.WKV7_ERR_INVALID_ARG
    for over in (dict(starts=None), dict(starts=FAKE + 2), dict(values=FAKE + 8), dict(queries=FAKE + 4),
                 dict(keys=FAKE + 2), dict(decays=FAKE + 8)):
        assert clear({}, **over) == wk.WKV7_ERR_INVALID_ARG, over
    assert clear(dict(N=48)) == wk.WKV7_ERR_UNSUPPORTED and clear(dict(scale=float("nan"))) == wk.WKV7_ERR_INVALID_ARG
    assert clear({}, values=None, queries=None, keys=None, decays=None) == wk.WKV7_OK
    none = wk.LinattnDesc(**dict(LA_OK, packed=1, tokens=0))
    assert L.wkv7_linattn_clear_rest(C(none), FAKE, FAKE, None, None, None, None) == wk.WKV7_OK
