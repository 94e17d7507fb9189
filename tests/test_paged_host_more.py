"""More of the paged-cache calls on the host.  No call here launches work."""
import ctypes as C
import math

import pytest

from dictionary_sparse_kv_gb300 import build as B
from dictionary_sparse_kv_gb300 import fadkv as F
from tests.test_paged_host import FAKE, _paged

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    B.build()
    return F.lib()


@pytest.mark.parametrize("name,arrays,positions", [("attend", 8, 4), ("prefill", 9, 5)])
def test_planned_calls_refuse(L, name, arrays, positions, monkeypatch):
    fn = getattr(L, f"fadkv_paged_{name}_planned")
    lse = arrays - 1
    assert fn(C.byref(_paged(T=-1)), *[FAKE] * (arrays + 1), 1 << 30, None) == 1
    for i in range(arrays):
        args = [FAKE] * (arrays + 1)
        args[i] = FAKE + 2
        assert fn(C.byref(_paged()), *args, 1 << 30, None) == 1, i
        if i not in (lse, positions):                         # both may be null
            args[i] = None
            assert fn(C.byref(_paged()), *args, 1 << 30, None) == 1, i
    assert fn(C.byref(_paged(B=0, T=0)), *[FAKE] * (arrays + 1), 1 << 30, None) == 0
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert fn(C.byref(_paged()), *[FAKE] * (arrays + 1), 1 << 30, None) == 4
    assert f"fadkv_paged_{name}_planned" in F.last_error()


def test_status_refusals(L, monkeypatch):
    word = C.c_uint64(7)
    for ws in (None, FAKE + 16):
        assert L.fadkv_paged_status(ws, C.byref(word), 1, None) == 1
    assert L.fadkv_paged_status(FAKE, None, 1, None) == 1
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert L.fadkv_paged_status(FAKE, C.byref(word), 1, None) == 4 and "fadkv_paged_status" in F.last_error()
    assert word.value == 7
