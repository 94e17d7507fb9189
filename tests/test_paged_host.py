"""Paged-cache calls on the host: refusals, workspace sizes and the rotation's
table.  No call here launches work."""
import ctypes as C
import math

import numpy as np
import pytest

from dictionary_sparse_kv_gb300 import build as B
from dictionary_sparse_kv_gb300 import fadkv as F
from tests import paged_util as U

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    B.build()
    return F.lib()


def _status(call, *args, **kw):
    with pytest.raises(F.FadkvError) as e:
        call(*args, **kw)
    return e.value.status


def test_plan_reference_by_hand():
    """Two pages of 8 are free (7 on top), request 1 ends and returns page 3, request 0 crosses a page, request 2
    asks for three pages and is refused, request 3 takes the last two."""
    table = np.array([[5, -1, -1], [3, -1, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    free = np.array([2, 7, 0, 0, 0, 0, 0, 0], np.int32)
    r = U.plan([2, -1, 24, 9], [7, 4, 0, 0], table, free, 2, 8, 40)
    assert r["free"][:3].tolist() == [2, 7, 3]
    assert r["table"].tolist() == [[5, 3, -1], [3, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    # request 3's two pages come after the three that request 2 asked for: refused too
    assert r["lengths"].tolist() == [9, 0, 0, 0] and r["refused"].tolist() == [2] and r["count"].tolist() == [2]
    assert r["starts"].tolist() == [0, 2, 2, 26, 35]
    assert r["positions"][:3].tolist() == [7, 8, -1] and r["slots"][:3].tolist() == [47, 24, -1]
    assert (r["slots"][2:] == -1).all()


def test_page_plan_refusals(L, monkeypatch):
    ok = dict(B=4, page_size=16, num_pages=64, max_pages=8, max_tokens=32)
    def call(ptrs=None, **kw):
        F.page_plan(F.page_params(**{**ok, **kw}), *(ptrs or [FAKE] * 11), stream=0)
    for kw, status in ((dict(B=-1), 1), (dict(num_pages=-1), 1), (dict(max_pages=0), 1), (dict(max_tokens=-1), 1),
                       (dict(page_size=12), 2), (dict(page_size=4), 2), (dict(page_size=2048), 2),
                       (dict(B=12289), 2), (dict(num_pages=2 ** 28), 2), (dict(max_pages=2 ** 28), 2)):
        assert _status(call, **kw) == status, kw
    for i in range(11):
        assert _status(call, ptrs=[FAKE] * i + [None] + [FAKE] * (10 - i)) == 1
        assert _status(call, ptrs=[FAKE] * i + [FAKE + 2] + [FAKE] * (10 - i)) == 1
    assert L.fadkv_page_plan(None, *[FAKE] * 12) == 1
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert _status(call) == 4 and "fadkv_page_plan" in F.last_error()


def test_strides_of_single_rows_pages_and_heads(L):
    """One row, page or head: torch's stride of that dimension says nothing and is not refused."""
    torch = pytest.importorskip("torch")
    d = 64
    q = torch.zeros(4, 1, d, dtype=torch.float16).transpose(0, 1)           # [1][4][d], stride(0) = d
    kv = torch.zeros(1, 2, d, dtype=torch.float16).as_strided((1, 2, d), (7, d, 1))
    pool = torch.zeros(16 * 2 * d, dtype=torch.float16).as_strided((1, 2, 16, d), (3, 16 * d, d, 1))
    p = F.qk_params(q, kv, kv, q, pool)
    assert (p.q_stride, p.k_stride, p.v_stride, p.page_stride, p.head_stride, p.token_stride) == (4 * d, 2 * d, 2 * d, d, 16 * d, d)
    table = torch.zeros(1, 1, dtype=torch.int32)
    assert F.paged_attend_workspace_bytes(F.paged_params(q, q, pool, "head", table)) > 0
    one_head = torch.zeros(3 * 16 * d, dtype=torch.float16).as_strided((3, 1, 16, d), (16 * d, 0, d, 1))
    p = F.paged_params(q, q, one_head, "head", table)
    assert p.q_stride == p.out_stride == 4 * d and (p.page_stride, p.head_stride) == (16 * d, d)
    assert F.paged_prefill_workspace_bytes(p) > 0


@pytest.mark.parametrize("scaling", ["plain", "linear", "stretch", "parts"])
@pytest.mark.parametrize("rd", [16, 32, 128])
def test_rope_table(L, scaling, rd):
    kw = dict(base=500000.0, factor=8.0, original=8192.0, slow=1.0, fast=4.0)
    r = F.rope_init(128, rd, scaling=scaling, amplitude=1.25, **kw)
    f = U.frequencies(rd, scaling=scaling, **kw)
    got = np.array([t / 2.0 ** 64 for t in r.turns[:rd // 2]])
    assert np.allclose(got, f / (2 * math.pi), rtol=2e-14, atol=2.0 ** -63)
    assert r.amplitude == 1.25 and r.rotary_dim == rd and not any(r.turns[rd // 2:])


def test_rope_refusals(L):
    for kw, status in ((dict(d=96), 2), (dict(rotary_dim=24), 2), (dict(rotary_dim=144), 1), (dict(rotary_dim=-16), 1),
                       (dict(base=1.0), 1), (dict(base=math.inf), 1), (dict(base=math.nan), 1),
                       (dict(scaling="linear", factor=0.5), 1), (dict(scaling="parts", factor=2.0, slow=4.0), 1),
                       (dict(scaling="parts", factor=2.0, original=0.0), 1), (dict(amplitude=math.inf), 1)):
        assert _status(F.rope_init, **{**dict(d=128, rotary_dim=64), **kw}) == status, kw
    with pytest.raises(KeyError):
        F.rope_init(128, 64, scaling="other")
    assert L.fadkv_rope_init(None, None) == 1


def _qk(**kw):
    d = kw.get("d", 128)
    v = dict(T=4, Hq=24, Hkv=8, d=d, dtype=F.F16, q_dtype=F.F32, kv_dtype=F.F16, page_size=16, num_pages=10, eps=1e-6,
             q_stride=40 * d, k_stride=40 * d, v_stride=40 * d, page_stride=8 * 16 * d, head_stride=16 * d, token_stride=d)
    v.update(kw)
    return F.QkParams(*[v[n] for n, _ in F.QkParams._fields_])


def test_qk_refusals(L, monkeypatch):
    rope = F.rope_init(128, 128)
    def call(p, ptrs=None, r=rope):
        F.qk_norm_rope(p, r, *(ptrs or [FAKE] * 11), stream=0)
    for kw, status in ((dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(dtype=3), 1), (dict(q_dtype=-1), 1),
                       (dict(kv_dtype=9), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(d=96), 2),
                       (dict(d=64), 1), (dict(Hq=5000), 2), (dict(q_stride=24 * 128 - 8), 1), (dict(k_stride=1025), 1),
                       (dict(v_stride=0), 1), (dict(page_size=24), 2), (dict(num_pages=-1), 1), (dict(head_stride=64), 1),
                       (dict(token_stride=132), 1), (dict(page_stride=-1024), 1)):
        assert _status(call, _qk(**kw)) == status, kw
    #       q k v wq wk positions slots q_out k_out k_pages v_pages
    needed = {0, 1, 2, 5, 7, 9, 10}
    for i in range(11):
        if i in needed:
            assert _status(call, _qk(), ptrs=[FAKE] * i + [None] + [FAKE] * (10 - i)) == 1, i
        assert _status(call, _qk(), ptrs=[FAKE] * i + [FAKE + 2] + [FAKE] * (10 - i)) == 1, i
    bad = F.rope_init(128, 128)
    bad.rotary_dim = 136
    assert _status(call, _qk(), r=bad) == 1
    call(_qk(T=0))                                        # nothing to launch
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert _status(call, _qk()) == 4 and "fadkv_qk_norm_rope" in F.last_error()


def _paged(**kw):
    d = kw.get("d", 128)
    v = dict(B=4, T=4, Hq=24, Hkv=8, d=d, dtype=F.F16, page_size=16, num_pages=10, max_pages=4, window=0, sinks=0, scale=0.1,
             q_stride=24 * d, out_stride=24 * d, page_stride=8 * 16 * d, head_stride=16 * d, token_stride=d)
    v.update(kw)
    return F.PagedParams(*[v[n] for n, _ in F.PagedParams._fields_])


BAD_PAGED = [(dict(B=-1), 1), (dict(T=-1), 1), (dict(Hq=25), 1), (dict(Hkv=0), 1), (dict(d=96), 2), (dict(dtype=F.F32), 2),
             (dict(dtype=5), 1), (dict(page_size=20), 2), (dict(num_pages=-2), 1), (dict(max_pages=0), 1),
             (dict(max_pages=2 ** 28), 2), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=math.nan), 1),
             (dict(q_stride=100), 1), (dict(out_stride=24 * 128 + 4), 1), (dict(head_stride=0), 1),
             (dict(B=12289, T=12289), 2)]


@pytest.mark.parametrize("prefill", [False, True])
def test_paged_refusals(L, prefill, monkeypatch):
    ask = F.paged_prefill_workspace_bytes if prefill else F.paged_attend_workspace_bytes
    fn = L.fadkv_paged_prefill if prefill else L.fadkv_paged_attend
    arrays = 8 if prefill else 7
    for kw, status in BAD_PAGED:
        p = _paged(**kw)
        assert _status(ask, p) == status, kw
        assert fn(C.byref(p), *[FAKE] * (arrays + 1), 1 << 30, None) == status, kw
    p = _paged()
    need = ask(p)
    for i in range(arrays):
        args = [FAKE] * (arrays + 1)
        args[i] = FAKE + 2
        assert fn(C.byref(p), *args, 1 << 30, None) == 1, i
        if i != arrays - 1:                               # lse may be null
            args[i] = None
            assert fn(C.byref(p), *args, 1 << 30, None) == 1, i
    if need:
        assert fn(C.byref(p), *[FAKE] * (arrays + 1), need - 1, None) == 5
        assert fn(C.byref(p), *[FAKE] * arrays, FAKE + 16, need, None) == 1
        assert fn(C.byref(p), *[FAKE] * arrays, None, need, None) == 5
    if not prefill:
        assert fn(C.byref(_paged(T=3)), *[FAKE] * (arrays + 1), 1 << 30, None) == 1
    assert fn(C.byref(_paged(B=0, T=0)), *[FAKE] * (arrays + 1), 1 << 30, None) == 0
    monkeypatch.setenv("FADKV_FAULT", "cuda")
    assert fn(C.byref(p), *[FAKE] * (arrays + 1), 1 << 30, None) == 4


def test_tensor_helpers_refuse(L):
    import torch
    q = torch.zeros(4, 24, 128, dtype=torch.float16)
    pool = torch.zeros(10, 8, 16, 128, dtype=torch.float16)
    table = torch.zeros(4, 3, dtype=torch.int32)
    p = F.paged_params(q, torch.empty_like(q), pool, "head", table)
    assert (p.B, p.T, p.Hkv, p.page_size, p.max_pages, p.head_stride) == (4, 4, 8, 16, 3, 16 * 128)
    p = F.paged_params(q, torch.empty_like(q), pool.transpose(1, 2).contiguous(), "token", table)
    assert (p.Hkv, p.page_size, p.head_stride, p.token_stride) == (8, 16, 128, 8 * 128)
    for bad in (dict(layout="other"), dict(block_table=table[:, :2]), dict(k_pages=pool.float()), dict(out=q[:3]),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(k_pages=pool[..., ::2])):
        with pytest.raises(ValueError):
            F.paged_params(**{**dict(q=q, out=torch.empty_like(q), k_pages=pool, layout="head", block_table=table), **bad})
    k = torch.zeros(4, 8, 128, dtype=torch.float16)
    for bad in (dict(k=k.float()), dict(v=k[:, :4]), dict(q=q[..., ::2])):
        with pytest.raises(ValueError):
            F.qk_params(**{**dict(q=q, k=k, v=k, q_out=q, k_pages=pool), **bad})


def test_direct_calls_check_their_arguments(L):
    """The binding's own module: other structs and objects are refused before the library is called."""
    p, r = _qk(), F.rope_init(128, 128)
    with pytest.raises(TypeError):
        F.qk_norm_rope(F.page_params(1, 8, 1, 1, 1), r, *[FAKE] * 11, stream=0)
    with pytest.raises(TypeError):
        F.qk_norm_rope(p, p, *[FAKE] * 11, stream=0)
    with pytest.raises(AttributeError):
        F.qk_norm_rope(p, r, "q", *[FAKE] * 10, stream=0)
    with pytest.raises(OverflowError):
        F.qk_norm_rope(p, r, 1 << 70, *[FAKE] * 10, stream=0)
    with pytest.raises(TypeError):
        F._calls.paged_attend(F._direct["paged_attend"], _paged())
    with pytest.raises(AttributeError):
        F.paged_prefill(_paged(), *[FAKE] * 8, workspace=object(), stream=0)
