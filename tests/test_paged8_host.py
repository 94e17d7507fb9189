"""The 8-bit paged cache and prompts on the host: refusals, workspace sizes, the binding's checks, and the plain implementation
that the GPU tests go by.  No call here launches work."""
import ctypes as C
import itertools

import numpy as np
import pytest

from dictionary_sparse_kv_gb300 import build as B
from dictionary_sparse_kv_gb300 import fadkv as F
from tests import paged8_util as V

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    B.build()
    return F.lib()


def _status(call, *args, **kw):
    with pytest.raises(F.FadkvError) as e:
        call(*args, **kw)
    return e.value.status


def _make(cls, base, **kw):
    v = {**base, **kw}
    return cls(*[v[n] for n, _ in cls._fields_])


POOL = dict(Hkv=8, d=128, format=F.E4M3, page_size=16, num_pages=10, block=16, page_stride=8 * 16 * 128, head_stride=16 * 128, token_stride=128)
BAD_POOL = [(dict(Hkv=0), 1), (dict(format=F.F16), 1), (dict(format=5), 1), (dict(format=-1), 1), (dict(d=96), 2),
            (dict(page_size=8), 2), (dict(page_size=24), 2), (dict(page_size=2048), 2), (dict(block=8), 2), (dict(block=24), 2), (dict(block=0), 2),
            (dict(block=32), 2), (dict(num_pages=-1), 1), (dict(num_pages=2 ** 28), 2), (dict(page_stride=-128), 1),
            (dict(head_stride=64), 1), (dict(token_stride=136), 1), (dict(token_stride=2 ** 40), 1)]


def _append(**kw):
    return _make(F.Append8Params, dict(T=4, k_dtype=F.F16, v_dtype=F.F32, k_stride=1024, v_stride=40 * 128, **POOL), **kw)


def _read(**kw):
    return _make(F.Read8Params, dict(B=4, max_pages=8, out_dtype=F.BF16, out_pages=32, out_page_stride=8 * 16 * 128, out_head_stride=16 * 128,
                                     out_token_stride=128, **POOL), **kw)


def _attend(**kw):
    return _make(F.Paged8Params, dict(B=4, Hq=24, dtype=F.F16, max_pages=8, window=0, sinks=0, scale=0.1, q_stride=24 * 128, out_stride=24 * 128, **POOL), **kw)


def _prompt(**kw):
    return _make(F.PromptParams, dict(B=2, T=100, Hq=24, Hkv=8, d=128, dtype=F.BF16, window=0, sinks=0, scale=0.1, q_stride=40 * 128,
                                      k_stride=1024, v_stride=40 * 128, out_stride=24 * 128), **kw)


def _pointers(call, n, optional, wide):
    """Each needed pointer missing; each one off its alignment (16 bytes for `wide`, 4 for the others)."""
    for i in range(n):
        if i not in optional:
            assert _status(call, [FAKE] * i + [None] + [FAKE] * (n - i - 1)) == 1, i
        assert _status(call, [FAKE] * i + [FAKE + (8 if i in wide else 2)] + [FAKE] * (n - i - 1)) == 1, i


def test_append_refusals(L, monkeypatch):
    call = lambda ptrs=None, p=None: F.paged8_append(p or _append(), *(ptrs or [FAKE] * 7), stream=0)
    for kw, status in BAD_POOL + [(dict(Hkv=4100), 2), (dict(T=-1), 1), (dict(k_dtype=F.E4M3), 1), (dict(v_dtype=-1), 1), (dict(k_stride=1016), 1),
                                  (dict(v_stride=1028), 1)]:
        assert _status(call, p=_append(**kw)) == status, kw
    _pointers(call, 7, (), {0, 1, 3, 4})
    F.paged8_append(_append(T=0), *[None] * 7, stream=0)                       # nothing to do, nothing wanted
    F.paged8_append(_append(num_pages=0, page_stride=0), *[None] * 7, stream=0)
    assert L.fadkv_paged8_append(None, *[FAKE] * 8) == 1
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert _status(call) == 4 and "fadkv_paged8_append" in F.last_error()


def test_read_refusals(L, monkeypatch):
    call = lambda ptrs=None, p=None: F.paged8_read(p or _read(), *(ptrs or [FAKE] * 10), stream=0)
    for kw, status in BAD_POOL + [(dict(Hkv=4100), 2), (dict(B=-1), 1), (dict(B=12289), 2), (dict(max_pages=0), 1), (dict(max_pages=2 ** 28), 2), (dict(out_pages=-1), 1),
                                  (dict(out_dtype=F.I8), 1), (dict(out_token_stride=64), 1), (dict(out_head_stride=132), 1), (dict(out_page_stride=0), 1)]:
        assert _status(call, p=_read(**kw)) == status, kw
    _pointers(call, 10, {6, 7}, {0, 1, 8, 9})
    for kw in (dict(B=0), dict(num_pages=0), dict(out_pages=0)):
        F.paged8_read(_read(**kw), *[None] * 10, stream=0)
    assert L.fadkv_paged8_read(None, *[FAKE] * 11) == 1
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert _status(call) == 4 and "fadkv_paged8_read" in F.last_error()


def test_attend_refusals(L, monkeypatch):
    need = F.paged8_attend_workspace_bytes(_attend())
    assert need > 0 and F.paged8_attend_workspace_bytes(_attend(d=64)) > 0

    def call(ptrs=None, p=None, workspace=FAKE, nbytes=None):
        q = list(ptrs or [FAKE] * 10)                   # k v ks vs table lengths positions q out lse
        p = p or _attend()
        rc = F.lib().fadkv_paged8_attend(C.byref(p), *q, workspace, need if nbytes is None else nbytes, 0)
        if rc:
            raise F.FadkvError("fadkv_paged8_attend", rc)
    bad = BAD_POOL + [(dict(B=-1), 1), (dict(B=12289), 2), (dict(Hq=0), 1), (dict(Hq=25), 1), (dict(Hq=8 * 1000), 2), (dict(Hq=4100, Hkv=4100), 2), (dict(dtype=F.F32), 2),
                      (dict(dtype=F.E4M3), 1), (dict(max_pages=0), 1), (dict(max_pages=2 ** 28), 2), (dict(num_pages=0), 1), (dict(window=-1), 1),
                      (dict(sinks=-1), 1), (dict(scale=float("inf")), 1), (dict(q_stride=24 * 128 - 8), 1), (dict(out_stride=24 * 128 + 4), 1)]
    for kw, status in bad:
        assert _status(call, p=_attend(**kw)) == status, kw
        out = C.c_size_t(7)
        assert L.fadkv_paged8_attend_workspace_bytes(C.byref(_attend(**kw)), C.byref(out)) == status and out.value == 7
    _pointers(call, 10, {6, 9}, {0, 1, 7, 8})
    assert _status(call, nbytes=need - 1) == 5 and _status(call, workspace=None) == 5 and _status(call, workspace=FAKE + 128) == 1
    assert L.fadkv_paged8_attend(None, *[FAKE] * 11, need, 0) == 1
    assert L.fadkv_paged8_attend_workspace_bytes(C.byref(_attend()), None) == 1
    F.paged8_attend(_attend(B=0), *[None] * 6, None, None, None, FAKE, stream=0)
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert _status(call) == 4 and "fadkv_paged8_attend" in F.last_error()


def test_prompt_refusals(L, monkeypatch):
    need = F.prompt_attend_workspace_bytes(_prompt())
    assert need > 0

    def call(ptrs=None, p=None, workspace=FAKE, nbytes=None):
        q = list(ptrs or [FAKE] * 7)                    # q k v starts positions out lse
        p = p or _prompt()
        rc = F.lib().fadkv_prompt_attend(C.byref(p), *q, workspace, need if nbytes is None else nbytes, 0)
        if rc:
            raise F.FadkvError("fadkv_prompt_attend", rc)
    for kw, status in [(dict(B=-1), 1), (dict(T=-1), 1), (dict(B=12289), 2), (dict(T=2 ** 31 - 1), 2), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=25), 1),
                       (dict(d=96), 2), (dict(dtype=F.F32), 2), (dict(dtype=F.I8), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
                       (dict(scale=float("nan")), 1), (dict(q_stride=24 * 128 - 8), 1), (dict(k_stride=1028), 1), (dict(v_stride=1016), 1), (dict(out_stride=0), 1)]:
        assert _status(call, p=_prompt(**kw)) == status, kw
        assert L.fadkv_prompt_attend_workspace_bytes(C.byref(_prompt(**kw)), C.byref(C.c_size_t())) == status
    _pointers(call, 7, {4, 6}, {0, 1, 2, 5})
    assert _status(call, nbytes=need - 1) == 5 and _status(call, workspace=None) == 5 and _status(call, workspace=FAKE + 128) == 1
    assert L.fadkv_prompt_attend(None, *[FAKE] * 8, need, 0) == 1
    for kw in (dict(B=0), dict(T=0)):
        F.prompt_attend(_prompt(**kw), None, None, None, None, None, None, FAKE, stream=0)
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert _status(call) == 4 and "fadkv_prompt_attend" in F.last_error()


def test_structs_are_told_apart(L):
    """The direct calls take no struct of another call."""
    calls = ((F.paged8_append, _append(T=0), [None] * 7), (F.paged8_read, _read(B=0), [None] * 10),
             (F.paged8_attend, _attend(B=0), [None] * 9 + [FAKE]), (F.prompt_attend, _prompt(B=0), [None] * 6 + [FAKE]))
    for (call, _, args), (_, p, _) in itertools.permutations(calls, 2):
        with pytest.raises((TypeError, F.FadkvError, C.ArgumentError)):
            call(p, *args, stream=0)


def test_binding_checks(L):
    torch = pytest.importorskip("torch")
    pool = lambda **kw: torch.zeros((5, 2, 32, 64), dtype=kw.get("dtype", torch.int8))
    k = torch.zeros((3, 2, 64), dtype=torch.float16)
    s = torch.ones((5, 2, 2))
    p = F.append8_params(k, k.float(), pool(), "head", s, pool(), s)
    assert (p.T, p.Hkv, p.d, p.k_dtype, p.v_dtype, p.format, p.page_size, p.num_pages, p.block) == (3, 2, 64, F.F16, F.F32, F.I8, 32, 5, 16)
    assert (p.k_stride, p.page_stride, p.head_stride, p.token_stride) == (128, 4096, 2048, 64)
    assert F.append8_params(k, k, pool(dtype=torch.float8_e4m3fn).transpose(1, 2), "token", s).format == F.E4M3
    q = torch.zeros((4, 6, 64), dtype=torch.bfloat16)
    table = torch.zeros((4, 9), dtype=torch.int32)
    a = F.paged8_params(q, q, pool(), s, "head", table, 7, 1)
    assert (a.B, a.Hq, a.Hkv, a.d, a.dtype, a.max_pages, a.window, a.sinks, a.block) == (4, 6, 2, 64, F.BF16, 9, 7, 1, 16)
    full = torch.zeros((8, 32, 2, 64), dtype=torch.float32)
    r = F.read8_params(pool(), s, full, table, "head", "token")
    assert (r.B, r.out_dtype, r.out_pages, r.out_page_stride, r.out_head_stride, r.out_token_stride) == (4, F.F32, 8, 4096, 64, 128)
    t = F.prompt_params(q, k[:0].expand(0, 2, 64).new_zeros((4, 2, 64)).bfloat16(), torch.zeros((4, 2, 64), dtype=torch.bfloat16), q, 2)
    assert (t.B, t.T, t.Hq, t.Hkv, t.k_stride, t.v_stride) == (2, 4, 6, 2, 128, 128)
    bad = [lambda: F.append8_params(k, k, pool(dtype=torch.uint8), "head", s), lambda: F.append8_params(k, k, pool(), "head", s[:4]),
           lambda: F.append8_params(k, k, pool(), "head", s.double()), lambda: F.append8_params(k, k[:2], pool(), "head", s),
           lambda: F.append8_params(k, k, pool(), "head", torch.ones((5, 2, 3))), lambda: F.append8_params(k, k, pool(), "head", s, pool()[:4]),
           lambda: F.append8_params(k.transpose(0, 1), k, pool(), "head", s), lambda: F.append8_params(k, k, pool(), "other", s),
           lambda: F.append8_params(k, k, pool(), "head", s, pool(), s[:, :1]),
           lambda: F.read8_params(pool(), s, full[:, :16], table, "head", "token"), lambda: F.read8_params(pool(), s, full, table[:, ::2], "head", "token"),
           lambda: F.read8_params(pool(), s, full, table, "head", "token", out_table=table[:3]),
           lambda: F.read8_params(pool(), s, full, table, "head", "token", v_out=full.half()),
           lambda: F.paged8_params(q, q.half(), pool(), s, "head", table), lambda: F.paged8_params(q[:3], q[:3], pool(), s, "head", table),
           lambda: F.paged8_params(q, q, pool(), s, "head", table.long()), lambda: F.paged8_params(q, q, pool(), s, "head", table, lse=torch.zeros(4, 5)),
           lambda: F.prompt_params(q, q[:, :2], q[:, :2].half(), q, 2), lambda: F.prompt_params(q, q[:3, :2], q[:3, :2], q, 2),
           lambda: F.prompt_params(q, q[:, :2], q[:, :2], q[:, :4], 2)]
    for call in bad:
        with pytest.raises(ValueError):
            call()


# --- the plain implementation -----------------------------------------------------

def test_codes():
    t = V.TABLE
    assert t[0x38] == 1.0 and t[0x7e] == 448.0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and np.isnan(t[0x7f]) and t[0xb8] == -1.0
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(V.encode(t[codes], "e4m3"), codes)
    mid = (t[:126] + t[1:127]) / 2
    assert np.array_equal(V.encode(mid, "e4m3") % 2, np.zeros(126))              # ties to the even code
    assert V.encode(np.array([np.inf, np.nan]), "e4m3").tolist() == [127, 127]
    x = np.array([0.5, 1.5, -2.5, 127.4, np.nan, np.inf, -np.inf, -126.5])
    assert V.encode(x, "i8").view(np.int8).tolist() == [0, 2, -2, 127, 0, 127, -127, -126]


def test_codes_as_torch_has_them():
    torch = pytest.importorskip("torch")
    x = torch.from_numpy(np.random.default_rng(0).standard_normal(20000) * 2.0 ** np.random.default_rng(1).integers(-12, 7, 20000)).float().clamp(-448, 448)
    assert np.array_equal(x.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), V.encode(x.double().numpy(), "e4m3"))


def test_scales():
    for fmt, m in (("e4m3", 448.0), ("i8", 127.0)):
        for a in (m, np.nextafter(m, 0), np.nextafter(m, 1e9), 0.0, 1.0, m * 2.0 ** -126, m * 2.0 ** -125, 3e38):
            t = V.least_scale(a, fmt)
            assert a <= m * t and (t == 2.0 ** -126 or a > m * t / 2)
