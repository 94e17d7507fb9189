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


def _rows(T, H, d, dtype=torch.float16):
    return torch.zeros((T, H, d), dtype=dtype)


def test_qk_params_refuses_outputs_that_the_kernel_would_overrun():
    """q_out and k_out are written as dense rows of q's and k's shape: fewer heads or rows, padded rows and other types
    are refused, as are a pool of another head dimension and pools that differ."""
    T, d = 4, 128
    q, k, pool = _rows(T, 24, d), _rows(T, 8, d), torch.zeros((10, 8, 16, d), dtype=torch.float16)
    ok = dict(q=q, k=k, v=k, q_out=_rows(T, 24, d, torch.float32), k_pages=pool)
    padded = torch.zeros((T, 24 * d + 64), dtype=torch.float16)[:, :24 * d].view(T, 24, d)
    for bad in (dict(q_out=_rows(T, 12, d)), dict(q_out=_rows(T - 1, 24, d)), dict(q_out=padded), dict(q_out=_rows(T, 24, 64)),
                dict(k_pages=torch.zeros((10, 8, 16, 64), dtype=torch.float16)),
                dict(k_pages=torch.zeros((10, 8, 16, 256), dtype=torch.float16)),
                dict(v_pages=pool[:9]), dict(v_pages=pool.bfloat16()), dict(v_pages=pool.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(k_out=_rows(T, 7, d)), dict(k_out=_rows(T, 8, d, torch.float32)), dict(k_out=padded[:, :8]),
                dict(wq=torch.zeros(d)), dict(wk=torch.zeros(64, dtype=torch.float16)), dict(wk=torch.zeros(2 * d, dtype=torch.float16)[::2])):
        with pytest.raises(ValueError):
            F.qk_params(**{**ok, **bad})
    w = torch.zeros(d, dtype=torch.float16)
    p = F.qk_params(**ok, k_out=_rows(T, 8, d), v_pages=torch.zeros_like(pool), wq=w, wk=w)
    assert bytes(p) == bytes(F.qk_params(**ok)) == bytes(F.qk_params(**{**ok, "q_out": _rows(T + 3, 24, d, torch.float32)}))
    one = torch.zeros((1, 8, 16, d), dtype=torch.float16)                     # a single page: its stride says nothing
    F.qk_params(**{**ok, "k_pages": one}, v_pages=one.as_strided(one.shape, (8, 16 * d, d, 1)))
    assert F.qk_params(q, k, k, ok["q_out"], None, kv_dtype=F.BF16, k_out=_rows(T, 8, d, torch.bfloat16)).kv_dtype == F.BF16


def test_paged_params_refuses_other_tables_and_pools():
    q, pool, table = _rows(4, 24, 128), torch.zeros((10, 8, 16, 128), dtype=torch.float16), torch.zeros((4, 3), dtype=torch.int32)
    ok = dict(q=q, out=torch.empty_like(q), k_pages=pool, block_table=table)
    for bad in (dict(block_table=table.long()), dict(block_table=table[0]), dict(v_pages=pool[:9]), dict(v_pages=pool.bfloat16()),
                dict(v_pages=pool.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=torch.zeros(4, 8)),
                dict(lse=torch.zeros(4, 24, dtype=torch.float64)), dict(lse=torch.zeros(24, 4).T)):
        with pytest.raises(ValueError):
            F.paged_params(**{**ok, **bad})
    p = F.paged_params(**ok, v_pages=torch.zeros_like(pool), lse=torch.zeros(4, 24))
    assert bytes(p) == bytes(F.paged_params(**ok))


def test_structs_of_one_size_are_told_apart(L):
    """QkParams and PagedParams have as many bytes; the direct calls take each for what it is."""
    from tests.test_paged_host import _qk
    assert C.sizeof(F.QkParams) == C.sizeof(F.PagedParams)
    rope = F.rope_init(128, 128)
    with pytest.raises(TypeError):
        F.qk_norm_rope(_paged(T=0), rope, *[FAKE] * 11, stream=0)
    for call, arrays in ((F.paged_attend, 8), (F.paged_prefill, 9)):
        with pytest.raises(TypeError):
            call(_qk(T=0), *[FAKE] * (arrays - 1), workspace=torch.zeros(1), stream=0)
    with pytest.raises(TypeError):
        F._calls.types(F.PageParams, F.QkParams, F.Rope)
    with pytest.raises(TypeError):
        F._calls.types(F.PageParams, F.QkParams, F.Rope, 5)

    class Mine(F.QkParams):
        pass

    p = Mine.from_buffer_copy(bytes(_qk(T=0)))                # a class derived from it is one
    F.qk_norm_rope(p, rope, *[FAKE] * 11, stream=0)


def test_addresses_and_streams_of_other_objects(L, monkeypatch):
    """Integers of any class are addresses; objects without a device are passed over in the search for a stream."""
    import enum

    class Place(enum.IntEnum):
        A = 0x1000

    class Array:                                              # an address and nothing else
        def data_ptr(self):
            return 0x2000

    class Cuda:                                               # a device, but not a tensor's way to ask for it
        device = torch.device("cuda", 0)

    assert F._addr(Place.A) == 0x1000 and F._addr(True) == 1 and F._addr(Array()) == 0x2000 and F._addr(None) is None
    stream = type("S", (), {"cuda_stream": 77})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    assert F._stream(None, Place.A, None, 5, Array(), torch.zeros(1)) == 77
    assert F._stream(None, Array(), Cuda()) == 77
    assert F._stream(stream, Array()) == 77 and F._stream(3) == 3
    class Tensor:
        def get_device(self):
            return 2
    monkeypatch.setattr(F, "_raw_stream", lambda d: 1000 + d)
    assert F._stream(None, None, Array(), torch.zeros(1), Tensor()) == 1002


def test_workspaces_given_as_addresses(L, monkeypatch):
    """As for the other arrays: an integer is an address, its size what the call needs."""
    monkeypatch.setenv("FADKV_FAULT", "cuda")                 # every check is passed, nothing is launched
    for call, arrays in ((F.paged_attend, 7), (F.paged_prefill, 8)):
        with pytest.raises(F.FadkvError) as e:
            call(_paged(), *[FAKE] * arrays, workspace=FAKE, stream=0)
        assert e.value.status == 4
        with pytest.raises(F.FadkvError) as e:
            call(_paged(), *[FAKE] * arrays, workspace=None, stream=0)
        assert e.value.status == 5


def test_rope_amplitude_has_to_be_finite_in_32_bits(L):
    for amplitude in (1e39, -1e39, math.inf, math.nan):
        with pytest.raises(F.FadkvError) as e:
            F.rope_init(128, 64, amplitude=amplitude)
        assert e.value.status == 1
    assert F.rope_init(128, 64, amplitude=3e38).amplitude == pytest.approx(3e38)
