"""Workspaces of the prefill and of prompts: one for the largest step serves the smaller ones (host only)."""
import ctypes as C
import itertools

import pytest

from dictionary_sparse_kv_gb300 import build as B
from dictionary_sparse_kv_gb300 import fadkv as F

FAKE = 0x10000
HEADS = [(1, 1), (2, 1), (8, 1), (24, 8), (7, 7), (40, 40), (300, 2), (60, 60)]
ROWS = [1, 2, 16, 43, 128, 129, 300, 1151, 1152, 1500, 4000, 8192, 20000, 200000]
WINDOWS = [(0, 0), (64, 4), (900, 4), (4096, 0)]


@pytest.fixture(scope="module")
def L():
    B.build()
    return F.lib()


def _prompt(b, t, hq, hkv, d, window):
    return F.PromptParams(b, t, hq, hkv, d, F.F16, *window, 0.1, hq * d, hkv * d, hkv * d, hq * d)


def _paged(b, t, hq, hkv, d, window, max_pages):
    return F.PagedParams(b, t, hq, hkv, d, F.F16, 16, 10, max_pages, *window, 0.1, hq * d, hq * d, hkv * 16 * d, 16 * d, d)


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("heads", HEADS)
def test_a_workspace_for_more_rows_serves_fewer(L, heads, window, monkeypatch):
    """Prompts: any number of prompts and rows up to those that it was sized for."""
    monkeypatch.setenv("FADKV_FAULT", "cuda")                 # every check is passed, nothing is launched
    sizes = {}
    for b, t, d in itertools.product((1, 3, 256, 300), ROWS, (64, 128)):
        sizes[b, t, d] = F.prompt_attend_workspace_bytes(_prompt(b, t, *heads, d, window))
    for (b, t, d), n in sizes.items():
        for (b1, t1, d1), n1 in sizes.items():
            if d1 == d and b1 <= b and t1 <= t:
                assert n1 <= n, (b, t, b1, t1)
                p = _prompt(b1, t1, *heads, d, window)
                assert L.fadkv_prompt_attend(C.byref(p), *[FAKE] * 8, n, 0) == 4, (b, t, b1, t1)


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("heads", HEADS)
def test_a_workspace_of_the_prefill_for_more_rows_serves_fewer(L, heads, window, monkeypatch):
    """The prefill over pages: any number of requests, rows and pages a request up to those that it was sized for."""
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    sizes = {}
    for b, t, m in itertools.product((1, 3, 256, 300), ROWS, (1, 63, 64, 2000)):
        sizes[b, t, m] = F.paged_prefill_workspace_bytes(_paged(b, t, *heads, 64, window, m))
    for (b, t, m), n in sizes.items():
        for (b1, t1, m1), n1 in sizes.items():
            if b1 <= b and t1 <= t and m1 <= m:
                assert n1 <= n, (b, t, m, b1, t1, m1)
                p = _paged(b1, t1, *heads, 64, window, m1)
                assert L.fadkv_paged_prefill(C.byref(p), *[FAKE] * 9, n, 0) == 4, (b, t, m, b1, t1, m1)


def test_a_workspace_of_many_rows_of_few_heads(L):
    """Two heads over one of 128: whatever a prompt of 1500 rows needs, one of 8192 has asked for."""
    size = lambda t: F.prompt_attend_workspace_bytes(_prompt(1, t, 2, 1, 128, (0, 0)))
    assert size(8192) >= size(4000) >= size(1500) > size(300)
