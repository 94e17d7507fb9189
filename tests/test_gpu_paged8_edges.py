"""The 8-bit paged cache and the prompts' attention at the calls that the documentation allows and the other tests do not make:
output pools 16 bytes off a sector, lengths far below what long tables have room for (needs a GPU)."""
import numpy as np
import pytest

from tests import paged8_util as V
from tests.test_gpu_paged8 import DEV, TYPES, _attend_state, _check_attend, _i32, _np, _random_codes, _tables, _to_pool

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
    ps, fmt = 1024, "e4m3"
    table, P, codes, scales = _attend_state(rng, [length], hkv, d, fmt, ps, 128, "head")
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
