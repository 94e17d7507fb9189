"""The 8-bit paged cache and the prompts' attention at the calls that the documentation allows and the other tests do not make:
output pools 16 bytes off a sector, lengths far below what long tables have room for, scales that are not
finite (needs a GPU)."""
import numpy as np
import pytest

from tests import paged8_util as V
from tests.test_gpu_paged8 import DEV, TYPES, _attend, _attend_state, _check_attend, _i32, _np, _random_codes, _tables, _to_pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    B.build()


# --- read -----------------------------------------------------------------------

def _off(shape, dtype, elements):
    """A pool that begins `elements` elements into an allocation."""
    n = int(np.prod(shape))
    return torch.full((n + elements,), -123.0, dtype=dtype, device=DEV)[elements:].view(shape)


@pytest.mark.parametrize("k_off,v_off", [(4, 4), (4, 0), (0, 4), (8, 8)])
@pytest.mark.parametrize("fmt,d,layout", [("e4m3", 128, "head"), ("i8", 64, "token")])
def test_read_to_32_bits_16_bytes_off_a_sector(k_off, v_off, fmt, d, layout):
    """Output pools are 16-byte aligned: bases 16 bytes past a multiple of 32, of either pool."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(k_off + v_off)
    lens, first, hkv, ps, block = [100, 33, 0, 250], [90, 0, 0, 17], 3, 32, 16
    table, P = _tables(rng, lens, ps)
    codes = [_random_codes(rng, (P, ps, hkv, d), fmt) for _ in range(2)]
    scales = [np.exp(rng.normal(0, 2, (P, hkv, ps // block))).astype(np.float32) for _ in range(2)]
    pools = [_to_pool(c, layout, fmt) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    B, mp = table.shape
    shape = (B * mp, hkv, ps, d) if layout == "head" else (B * mp, ps, hkv, d)
    out = [_off(shape, TYPES["f32"], n) for n in (k_off, v_off)]
    assert [o.data_ptr() % 32 for o in out] == [n * 4 % 32 for n in (k_off, v_off)]
    p = F.read8_params(pools[0], pools[2], out[0], _i32(table), layout, None, pools[1], pools[3], out[1])
    F.paged8_read(p, *pools, _i32(table), _i32(lens), _i32(first), None, *out)
    torch.cuda.synchronize()
    for c, s, got in zip(codes, scales, out):
        want = np.full((B * mp, ps, hkv, d), -123.0, np.float32)
        for b in range(B):
            for j in range(first[b], lens[b]):
                page = int(table[b, j // ps])
                want[b * mp + j // ps, j % ps] = V.decode(c[page, j % ps], fmt).astype(np.float32) * s[page, :, j % ps // block][:, None]
        got = got.cpu().transpose(1, 2) if layout == "head" else got.cpu()
        assert torch.equal(got, torch.from_numpy(want))


# --- attention of single tokens -----------------------------------------------------

@pytest.mark.parametrize("length", [0, 1, 65, 100, 128, 300])
@pytest.mark.parametrize("hkv,d", [(65, 64), (70, 128)])
def test_attend_short_requests_in_very_long_tables(hkv, d, length):
    """Tables of 2^31 tokens (units counted in 64 bits) and a request of a few blocks: fewer units than CTAs."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(length)
    ps, fmt, P = 1024, "i8", 2
    table = np.array([[1, -1]], np.int32)
    codes = [rng.integers(-127, 128, (P, ps, hkv, d), np.int8).view(np.uint8) for _ in range(2)]
    scales = [np.exp(rng.normal(-4.6, 1, (P, hkv, 8))).astype(np.float32) for _ in range(2)]
    pools = [_to_pool(c, "head", fmt) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    wide = torch.full((1, (1 << 21) - 5), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = _i32(table)
    q = torch.randn((1, hkv, d), generator=torch.Generator().manual_seed(7)).half().to(DEV)
    out, lse = torch.empty_like(q), torch.empty((1, hkv), device=DEV)
    p = F.paged8_params(q, out, pools[0], pools[2], "head", wide)
    ws = torch.zeros(F.paged8_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    want = V.attend(_np(q), codes[0], codes[1], scales[0], scales[1], table, [length], 0, 0, d ** -0.5, fmt)
    for _ in range(3):                                  # the workspace is left fit for the next call
        out.fill_(9), lse.fill_(9)
        F.paged8_attend(p, *pools, wide, _i32([length]), q, out, lse, ws)
        torch.cuda.synchronize()
        _check_attend((out, lse), want, max(length, 1), d, torch.float16)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("fmt,d", [("e4m3", 64), ("i8", 64), ("e4m3", 128), ("i8", 128)])
def test_attend_scales_that_are_not_finite(fmt, d, sign, bad):
    """A seen block's scale that is not finite makes what it enters NaN, whatever the products' signs: of the keys, the rows and
    lse of the heads that read it; of the values, the rows alone.  Nothing else changes."""
    rng = np.random.default_rng(2)
    lens, hkv, ps = [40, 300], 2, 16
    table, P, codes, scales = _attend_state(rng, lens, hkv, d, fmt, ps, 16, "head")
    positive = np.abs(V.decode(codes[0], fmt)) + 1
    codes[0] = V.encode(positive.clip(1, 127), fmt)
    q = sign * torch.rand((2, 2 * hkv, d), generator=torch.Generator().manual_seed(1)).add(0.5).half().to(DEV)
    pools = [_to_pool(c, "head", fmt) for c in codes] + [torch.from_numpy(s.copy()).to(DEV) for s in scales]
    out0, lse0 = _attend(q, pools, "head", table, lens)
    assert out0.isfinite().all() and lse0.isfinite().all()
    rows = torch.zeros((2, 2 * hkv), dtype=torch.bool, device=DEV)
    rows[0, 2:] = True                                  # request 0, the heads over KV head 1
    for which in (2, 3):                                # of the keys, of the values
        was = pools[which][table[0, 1], 1, 0].clone()
        pools[which][table[0, 1], 1, 0] = bad
        out, lse = _attend(q, pools, "head", table, lens)
        assert torch.equal(out.isnan(), rows[..., None].expand_as(out)) and torch.equal(out[~rows], out0[~rows])
        if which == 2:
            assert torch.equal(lse.isnan(), rows) and torch.equal(lse[~rows], lse0[~rows])
        else:
            assert torch.equal(lse, lse0)
        pools[which][table[0, 1], 1, 0] = was
