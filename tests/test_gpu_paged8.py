"""The 8-bit paged cache (append, read back, attention of single tokens) and the attention of packed prompts, against plain
implementations in 64 bits, through the C ABI (needs a GPU).

Codes and scales: equal.  What is read back: equal to the 32-bit product, rounded once.  Attention: the bounds of
paged8_util.bounds and paged_util.bounds, element by element.
"""
import numpy as np
import pytest

from tests import paged8_util as V
from tests import paged_util as U

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HELD = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    B.build()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(DEV)


def _np(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _codes(pool, layout):
    """[pages][ps][Hkv][d] uint8 of a pool."""
    x = pool.detach().view(torch.uint8).cpu().numpy()
    return np.ascontiguousarray(x.transpose(0, 2, 1, 3) if layout == "head" else x)


def _to_pool(codes, layout, fmt):
    x = codes.transpose(0, 2, 1, 3) if layout == "head" else codes
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).view(HELD[fmt])


def _random_codes(rng, shape, fmt):
    x = rng.integers(0, 256, shape).astype(np.uint8)
    x[(x & 127) == 127] = 0 if fmt == "e4m3" else 1
    if fmt == "i8":
        x[x == 128] = 3
    return x


def _tables(rng, lens, ps, spare=2):
    need = [-(-int(n) // ps) for n in lens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(1, max(need, default=0)) + 1), -1, np.int32)
    o = 0
    for b, n in enumerate(need):
        table[b, :n] = order[o:o + n]
        o += n
    return table, sum(need) + spare


# --- append -------------------------------------------------------------------

APPENDS = [
    # lengths before, new tokens, Hkv, d, k type, v type, format, page, block, layout
    ([0], [1], 1, 64, "f16", "f16", "e4m3", 16, 16, "head"),
    ([0, 5, 15, 16, 31], [1, 1, 1, 1, 1], 8, 128, "f16", "f16", "e4m3", 16, 16, "head"),
    ([3, 0, 40], [20, 33, 70], 2, 128, "bf16", "f32", "i8", 32, 32, "token"),
    ([0, 7, 100], [200, 130, 29], 5, 64, "f32", "bf16", "e4m3", 64, 16, "token"),
    ([1], [300], 3, 128, "f32", "f32", "i8", 128, 128, "head"),                      # runs longer than what is kept
    ([0, 17], [1100, 1000], 1, 64, "f16", "bf16", "e4m3", 1024, 1024, "head"),       # blocks of many rows
    ([11] * 40, [1] * 40, 4, 64, "bf16", "bf16", "i8", 16, 16, "token"),
    ([0, 9, 60], [900, 400, 700], 8, 128, "bf16", "f16", "e4m3", 32, 16, "head"),    # ranges of 16 rows a warp
    ([2, 0, 5], [2000, 3, 500], 4, 64, "f32", "f16", "i8", 64, 64, "head"),
    ([30, 0], [3000, 700], 1, 128, "f16", "f32", "e4m3", 512, 256, "token"),         # four warps a block of tokens
    ([40, 0], [14500, 900], 8, 64, "f16", "bf16", "i8", 64, 64, "head"),             # more rows a warp than it has lanes
    ([3, 0], [7500, 300], 8, 128, "f16", "f16", "e4m3", 128, 128, "token"),          # the same, four warps a block
]


def _append(k, v, slots, pools, layout):
    from dictionary_sparse_kv_gb300 import fadkv as F
    p = F.append8_params(k, v, pools[0], layout, pools[2], pools[1], pools[3])
    F.paged8_append(p, k, v, slots, *pools)
    torch.cuda.synchronize()


def _slots(table, before, new, ps):
    out = []
    for b, (l, n) in enumerate(zip(before, new)):
        out += [int(table[b, j // ps]) * ps + j % ps for j in range(l, l + n)]
    return out


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append(i):
    before, new, hkv, d, kt, vt, fmt, ps, block, layout = APPENDS[i]
    rng = np.random.default_rng(100 + i)
    table, P = _tables(rng, [a + b for a, b in zip(before, new)], ps)
    slots = _slots(table, before, new, ps)
    # rows that are skipped, between requests and at the end
    slots = [-1] + slots[:new[0]] + [-1, P * ps, 2 ** 31 - 1] + slots[new[0]:] + [-5]
    T = len(slots)
    wide = np.exp(rng.normal(0, 1.5, (T, 1, 1)))
    k = torch.from_numpy(rng.standard_normal((T, hkv, d)) * wide).to(TYPES[kt]).to(DEV)
    # values: one part of wider rows
    v = torch.from_numpy(rng.standard_normal((T, 3 * hkv * d)) * wide[:, :, 0]).to(TYPES[vt]).to(DEV)[:, hkv * d:2 * hkv * d].view(T, hkv, d)
    codes = [_random_codes(rng, (P, ps, hkv, d), fmt) for _ in range(2)]
    scales = [(2.0 ** rng.integers(-9, -3, (P, hkv, ps // block))).astype(np.float32) for _ in range(2)]
    pools = [_to_pool(c, layout, fmt) for c in codes] + [torch.from_numpy(s.copy()).to(DEV) for s in scales]
    for x, c, s in zip((k, v), codes, scales):
        V.append(_np(x), slots, c, s, ps, block, fmt)
    for _ in range(2):                                 # the same again: the same result
        _append(k, v, _i32(slots), pools, layout)
        for n, got, want in (("k", pools[0], codes[0]), ("v", pools[1], codes[1])):
            assert np.array_equal(_codes(got, layout), want), n
        for n, got, want in (("k", pools[2], scales[0]), ("v", pools[3], scales[1])):
            assert np.array_equal(got.cpu().numpy(), want), n


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_append_odd_values(fmt, dt):
    """Zeros, the type's extremes, what is not finite, ties, and blocks of one kind of value; old scales that are no powers of
    two, zero scales."""
    rng = np.random.default_rng(7)
    hkv, d, ps, block, P = 2, 64, 32, 16, 12
    big, tiny = torch.finfo(TYPES[dt]).max, torch.finfo(TYPES[dt]).smallest_normal
    rows = []
    for kind in range(10):
        x = rng.standard_normal((hkv, d))
        if kind == 1: x[:] = 0
        if kind == 2: x[:] = -0.0
        if kind == 3: x[0, 5], x[1, 9] = big, -big
        if kind == 4: x *= tiny / 4
        if kind == 5: x[0, 3], x[0, 4], x[1, 7] = np.inf, -np.inf, np.nan
        if kind == 6: x[:] = np.inf
        if kind == 7: x = rng.integers(-255, 256, (hkv, d)) / 2.0               # ties
        if kind == 8: x[:] = 448 * 2.0 ** -5
        if kind == 9: x[:] = np.nan
        rows.append(x)
    x = torch.from_numpy(np.stack(rows)).to(TYPES[dt]).to(DEV)
    # each alone at the start of a block, and each behind tokens that are there already
    for first in (0, 9):
        slots = [(2 + kind) * ps + (16 if kind % 2 else 0) + first for kind in range(10)]
        codes = [_random_codes(rng, (P, ps, hkv, d), fmt) for _ in range(2)]
        scales = [rng.choice(np.float32([0.0, 0.3, 2.0 ** -126, 0.01, 1.7, 2.0 ** 60]), (P, hkv, ps // block)) for _ in range(2)]
        pools = [_to_pool(c, "head", fmt) for c in codes] + [torch.from_numpy(s.copy()).to(DEV) for s in scales]
        for c, s in zip(codes, scales):
            V.append(_np(x), slots, c, s, ps, block, fmt)
        _append(x, x, _i32(slots), pools, "head")
        for got, want in zip(pools, codes):
            assert np.array_equal(V.decode(_codes(got, "head"), fmt), V.decode(want, fmt), equal_nan=True)
        for got, want in zip(pools[2:], scales):
            assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("ps,block,d,dt", [(32, 32, 64, "f16"), (128, 128, 128, "bf16"), (256, 64, 128, "f32")])
def test_append_in_any_order_within_a_block(ps, block, d, dt):
    """Rows of one block in any order, some with values that are not finite (in a large block too)."""
    rng = np.random.default_rng(block)
    hkv, before, new, fmt = 2, [7, 40], [5 * block + 3, 60], "e4m3"
    table, P = _tables(rng, [a + b for a, b in zip(before, new)], ps)
    slots = np.array(_slots(table, before, new, ps))
    blk = slots // block
    cuts = [0] + (np.flatnonzero(blk[1:] != blk[:-1]) + 1).tolist() + [len(slots)]
    for a, b in zip(cuts, cuts[1:]):
        slots[a:b] = rng.permutation(slots[a:b])
    x = torch.from_numpy(rng.standard_normal((len(slots), hkv, d)) * 3).to(TYPES[dt]).to(DEV)
    x[block + 5, 1, 3], x[2 * block + 9, 0, 0], x[2 * block + 9, 0, d - 1] = float("nan"), float("inf"), float("-inf")
    x[cuts[2]:cuts[3], 1] = float("inf")                # nothing finite in a whole block
    for f in (fmt, "i8"):
        codes = [_random_codes(rng, (P, ps, hkv, d), f) for _ in range(2)]
        scales = [(2.0 ** rng.integers(-12, -3, (P, hkv, ps // block))).astype(np.float32) for _ in range(2)]
        pools = [_to_pool(c, "head", f) for c in codes] + [torch.from_numpy(s.copy()).to(DEV) for s in scales]
        for c, s in zip(codes, scales):
            V.append(_np(x), slots.tolist(), c, s, ps, block, f)
        _append(x, x, _i32(slots), pools, "head")
        for got, want in zip(pools, codes):
            assert np.array_equal(V.decode(_codes(got, "head"), f), V.decode(want, f), equal_nan=True)
        for got, want in zip(pools[2:], scales):
            assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_append_token_by_token_stays_within_a_step(fmt):
    """A block filled one token at a time with growing values: an I8 value ends less than one step of the last scale from its
    input, an E4M3 value within half a step of its own and one of the type's smallest steps (2^-9) of the last scale."""
    rng = np.random.default_rng(3)
    hkv, d, ps = 2, 128, 16
    pools = [torch.zeros((1, hkv, ps, d), dtype=torch.int8, device=DEV).view(HELD[fmt]) for _ in range(2)] + [
        torch.zeros((1, hkv, 1), device=DEV) for _ in range(2)]
    x = torch.from_numpy(rng.standard_normal((ps, hkv, d)) * 1.7 ** np.arange(ps)[:, None, None]).half().to(DEV)
    for t in range(ps):
        _append(x[t:t + 1], x[t:t + 1], _i32([t]), pools, "head")
    s = pools[2].cpu().numpy().astype(np.float64).reshape(1, hkv, 1)
    got = V.decode(_codes(pools[0], "head"), fmt)[0] * s
    want = _np(x)
    err = np.abs(got - want)
    if fmt == "i8":
        assert (err < s).all()
    else:
        assert (err <= np.abs(want) * 2.0 ** -4 + 2.0 ** -9 * s).all()


def test_append_of_nothing():
    from dictionary_sparse_kv_gb300 import fadkv as F
    pools = [torch.zeros((2, 1, 16, 64), dtype=torch.int8, device=DEV) for _ in range(2)] + [torch.ones((2, 1, 1), device=DEV) for _ in range(2)]
    x = torch.ones((0, 1, 64), device=DEV)
    p = F.append8_params(x, x, pools[0], "head", pools[2])
    F.paged8_append(p, x, x, _i32([]), *pools)
    x = torch.ones((3, 1, 64), device=DEV)
    _append(x, x, _i32([-1, 32, -7]), pools, "head")
    assert not any(t.any() for t in pools[:2]) and all((t == 1).all() for t in pools[2:])


# --- read -----------------------------------------------------------------------

READS = [
    # lengths, first, Hkv, d, type, format, page, block, layout, layout of the output, own output table
    ([1], None, 1, 64, "f16", "e4m3", 16, 16, "head", "head", False),
    ([0, 77, 16, 300], None, 8, 128, "f16", "e4m3", 16, 16, "head", "token", False),
    ([100, 33, 0, 250], [90, 40, 0, 17], 3, 64, "f32", "i8", 64, 16, "token", "token", True),
    ([129, 5], [0, 1], 2, 128, "bf16", "i8", 32, 32, "token", "head", True),
    ([40 + b for b in range(150)], [b for b in range(150)], 2, 64, "bf16", "e4m3", 128, 64, "head", "head", True),
]


@pytest.mark.parametrize("i", range(len(READS)))
def test_read(i):
    from dictionary_sparse_kv_gb300 import fadkv as F
    lens, first, hkv, d, dt, fmt, ps, block, layout, out_layout, own = READS[i]
    rng = np.random.default_rng(200 + i)
    B = len(lens)
    table, P = _tables(rng, lens, ps)
    if len(lens) > 1:
        table[1, 0] = (-1, P, -9, P + 5, -1)[i]          # a page that is none
    codes = [_random_codes(rng, (P, ps, hkv, d), fmt) for _ in range(2)]
    codes[0][0, 0] = 0x7f                                # NaN in E4M3
    scales = [np.exp(rng.normal(0, 2, (P, hkv, ps // block))).astype(np.float32) for _ in range(2)]
    pools = [_to_pool(c, layout, fmt) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    mp = table.shape[1]
    out_pages = B * mp + 1 if not own else int((table >= 0).sum())
    out_table = np.arange(B * mp).reshape(B, mp)
    if own:
        out_table = np.full((B, mp), -1)
        flat = np.flatnonzero(table >= 0)
        out_table.reshape(-1)[flat] = rng.permutation(len(flat))
        out_table[B - 1, 0] = out_pages + 3              # no output page: skipped
    shape = (out_pages, hkv, ps, d) if out_layout == "head" else (out_pages, ps, hkv, d)
    out = [torch.full(shape, -123.0, dtype=TYPES[dt], device=DEV) for _ in range(2)]
    ot = _i32(out_table) if own else None
    p = F.read8_params(pools[0], pools[2], out[0], _i32(table), layout, out_layout, pools[1], pools[3], out[1], ot)
    F.paged8_read(p, *pools, _i32(table), _i32(lens), None if first is None else _i32(first), ot, *out)
    torch.cuda.synchronize()
    for c, s, got in zip(codes, scales, out):
        want = np.full((out_pages, ps, hkv, d), -123.0, np.float32)
        for b in range(B):
            for j in range(0 if first is None else first[b], lens[b]):
                page, to = int(table[b, j // ps]), int(out_table[b, j // ps])
                if 0 <= page < P and 0 <= to < out_pages:
                    want[to, j % ps] = V.decode(c[page, j % ps], fmt).astype(np.float32) * s[page, :, j % ps // block][:, None]
        want = torch.from_numpy(want).to(TYPES[dt])
        got = got.cpu().transpose(1, 2) if out_layout == "head" else got.cpu()
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(got.isnan(), want.isnan())


# --- attention of single tokens -----------------------------------------------------

ATTENDS = [
    # lengths, Hq, Hkv, d, type, format, page, block, layout, window, sinks
    ([1], 1, 1, 64, "f16", "e4m3", 16, 16, "head", 0, 0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 300], 24, 8, 128, "f16", "e4m3", 16, 16, "head", 0, 0),
    ([777], 24, 8, 128, "bf16", "i8", 64, 32, "token", 0, 0),
    ([0, 200, 1], 4, 4, 64, "bf16", "e4m3", 32, 16, "token", 0, 0),
    ([500, 33, 70, 1000], 16, 2, 64, "f16", "i8", 128, 128, "head", 64, 4),
    ([500, 33, 70, 1000], 12, 1, 128, "bf16", "e4m3", 16, 16, "token", 50, 37),      # two tiles of heads
    ([300, 90, 201], 40, 2, 64, "f16", "e4m3", 64, 16, "head", 130, 70),             # several pieces of heads, many first tokens
    ([400], 16, 1, 64, "bf16", "i8", 16, 16, "head", 1, 0),                          # the window is the token itself
    ([5000, 3], 3, 1, 128, "f16", "i8", 256, 64, "head", 0, 0),                      # pieces joined
    ([12000], 2, 1, 64, "bf16", "e4m3", 1024, 256, "token", 0, 0),                   # joined in groups
    ([20 + 7 * b for b in range(70)], 6, 2, 128, "f16", "e4m3", 32, 32, "head", 0, 0),   # more requests than a warp has lanes
    ([900] * 33 + [1] * 5, 8, 8, 64, "bf16", "i8", 16, 16, "token", 200, 1),
]


def _attend_state(rng, lens, hkv, d, fmt, ps, block, layout, spread=1.0):
    table, P = _tables(rng, lens, ps)
    codes = [_random_codes(rng, (P, ps, hkv, d), fmt) for _ in range(2)]
    if fmt == "e4m3":
        codes = [V.encode(np.clip(rng.standard_normal((P, ps, hkv, d)) * 100, -448, 448), fmt) for _ in range(2)]
    scales = [np.exp(rng.normal(-4.6, spread, (P, hkv, ps // block))).astype(np.float32) for _ in range(2)]
    return table, P, codes, scales


def _attend(q, pools, layout, table, lens, window=0, sinks=0, scale=None, positions=None, ws=None, lse=True):
    from dictionary_sparse_kv_gb300 import fadkv as F
    out = torch.full_like(q, 99.0)
    l = torch.full(q.shape[:2], 99.0, device=DEV) if lse else None
    t = _i32(table)
    p = F.paged8_params(q, out, pools[0], pools[2], layout, t, window, sinks, scale, pools[1], pools[3], l)
    if ws is None:
        ws = torch.zeros(F.paged8_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    F.paged8_attend(p, *pools, t, _i32(lens), q, out, l, ws, positions=None if positions is None else _i32(positions))
    torch.cuda.synchronize()
    return out, l


def _check_attend(got, want, n, d, dt):
    out, lse, pv, big, most = want
    e_out, e_lse = V.bounds(out, lse, pv, big, n, most, d, torch.finfo(dt).eps)
    o, l = _np(got[0]), _np(got[1])
    assert np.isfinite(o).all() and (np.abs(o - out) <= e_out).all(), (np.abs(o - out) / e_out).max()
    fine = np.isfinite(lse)
    assert np.array_equal(np.isfinite(l), fine)
    assert (np.abs(l[fine] - lse[fine]) <= e_lse[fine]).all(), (np.abs(l[fine] - lse[fine]) / e_lse[fine]).max()


@pytest.mark.parametrize("i", range(len(ATTENDS)))
def test_attend(i):
    lens, Hq, hkv, d, dt, fmt, ps, block, layout, window, sinks = ATTENDS[i]
    rng = np.random.default_rng(300 + i)
    table, P, codes, scales = _attend_state(rng, lens, hkv, d, fmt, ps, block, layout)
    if len(lens) > 2:                                   # pages that are none: not seen
        table[-1, 0] = P
        table[-2, table.shape[1] // 3] = -1
    B = len(lens)
    q = torch.from_numpy(rng.standard_normal((B, Hq + 1, d)) * 1.5).to(TYPES[dt]).to(DEV)[:, :Hq]    # rows apart
    pools = [_to_pool(c, layout, fmt) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    positions = [n - 1 for n in lens] if i % 2 else None
    if positions and B > 1:
        positions[0] = -1                               # refused
    scale = (None, -0.05, 0.2)[i % 3]
    want = V.attend(_np(q), codes[0], codes[1], scales[0], scales[1], table, lens, window, sinks, scale or d ** -0.5, fmt, positions)
    got = _attend(q, pools, layout, table, lens, window, sinks, scale, positions)
    _check_attend(got, want, max(lens), d, TYPES[dt])


def test_attend_blocks_of_very_different_size():
    """Scales from 2^-60 to 2^20 beside one another, the largest where hardly anything is seen: what the small ones give is
    kept."""
    rng = np.random.default_rng(5)
    d, ps, n = 64, 16, 640
    table, P, codes, scales = _attend_state(rng, [n], 1, d, "e4m3", ps, 16, "head")
    q = torch.zeros((1, 2, d), dtype=torch.float16, device=DEV)
    q[:, :, 0] = 8.0
    codes[0][:] = 0
    codes[0][..., 0] = V.encode(np.float64(64.0), "e4m3")
    pages = table[0, :n // ps]
    scales[0][pages[:20]] = 1.0                         # scores 64 * 8 / 8 = 64 ...
    scales[0][pages[20:]] = 2.0 ** -4                   # ... and 4: e^-60 of the others
    scales[1][pages[:20]] = 2.0 ** -12
    scales[1][pages[20:]] = 2.0 ** 20
    scales[1][pages[::3]] = 2.0 ** -60
    pools = [_to_pool(c, "head", "e4m3") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    want = V.attend(_np(q), codes[0], codes[1], scales[0], scales[1], table, [n], 0, 0, d ** -0.5, "e4m3")
    want[4][:] = 2.0 ** -12 * 448                       # the largest weight times value: e^-60 2^20 is far below
    got = _attend(q, pools, "head", table, [n])
    _check_attend(got, want, n, d, torch.float16)


@pytest.mark.parametrize("power", [-126, -110, 100, 112])
def test_attend_values_near_the_ends_of_their_range(power):
    """Scales of the values near 2^-126 and 2^112: bfloat16 holds the result, and the references' difference is as large."""
    rng = np.random.default_rng(14)
    lens, d, ps = [40, 300, 1500], 128, 16
    table, P, codes, scales = _attend_state(rng, lens, 1, d, "e4m3", ps, 16, "head")
    scales[1][:] = 2.0 ** (power + rng.integers(0, 3, scales[1].shape))
    q = torch.from_numpy(rng.standard_normal((3, 3, d))).bfloat16().to(DEV)
    pools = [_to_pool(c, "head", "e4m3") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    want = V.attend(_np(q), codes[0], codes[1], scales[0], scales[1], table, lens, 0, 0, d ** -0.5, "e4m3")
    out, lse = _attend(q, pools, "head", table, lens)
    e_out, _ = V.bounds(*want[:4], 1500, want[4], d, 2.0 ** -7, least=2.0 ** -133)    # bfloat16's smallest step
    assert (np.abs(_np(out) - want[0]) <= e_out).all(), (np.abs(_np(out) - want[0]) / e_out).max()


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_attend_keeps_small_probabilities(fmt):
    """131072 keys 12.1 (in units of the exponent) below one whose value is 0."""
    n, d, ps = 131073, 64, 1024
    P = -(-n // ps)
    one = {"e4m3": 0x38, "i8": 1}[fmt]
    codes = [np.zeros((P, ps, 1, d), np.uint8) for _ in range(2)]
    codes[0][..., 0] = one
    codes[1][:] = one
    scales = [np.ones((P, 1, 1), np.float32) for _ in range(2)]
    q = torch.zeros((1, 1, d), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = -12.125
    codes[0][0, 0], codes[1][0, 0] = 0, 0
    table = np.arange(P, dtype=np.int32)[None]
    pools = [_to_pool(c, "head", fmt) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    out, lse = _attend(q, pools, "head", table, [n], scale=1.0)
    w = 131072 * np.exp(-12.125)
    want = w / (1 + w)
    # bfloat16: half a step; what is lost: 131072 times 2^-36
    assert abs(_np(out) - want).max() <= want * 2.0 ** -8 + 2.0 ** -19
    assert abs(_np(lse) - np.log1p(w)).max() < 1e-5


def test_attend_what_is_not_seen_is_not_used():
    """NaN codes past the lengths, outside the window and on pages that are none; scales of blocks that hold nothing seen; a
    code that is seen touches its element or its row alone."""
    rng = np.random.default_rng(6)
    lens, d, ps, window, sinks = [100, 37, 300, 0], 64, 64, 40, 3
    table, P, codes, scales = _attend_state(rng, lens, 2, d, "e4m3", ps, 16, "head")
    clean = [c.copy() for c in codes]
    live = np.zeros((P, ps), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            if j > n - 1 - window or j < sinks:
                live[table[b, j // ps], j % ps] = True
    for c, s in zip(codes, scales):
        c[~live] = 0x7f
        for page in range(P):
            for part in range(ps // 16):
                if not live[page, part * 16:part * 16 + 16].any():
                    s[page, :, part] = np.nan
    q = torch.from_numpy(rng.standard_normal((4, 6, d))).half().to(DEV)
    pools = [_to_pool(c, "head", "e4m3") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    want = V.attend(_np(q), clean[0], clean[1], np.nan_to_num(scales[0]), np.nan_to_num(scales[1]), table, lens, window, sinks, d ** -0.5, "e4m3")
    got = _attend(q, pools, "head", table, lens, window, sinks)
    _check_attend(got, want, 300, d, torch.float16)
    # a value that is NaN: that element of the heads that read it; a key: the rows of its head
    page, at = table[2, 299 // ps], 299 % ps
    pools[1].view(torch.uint8)[page, 1, at, 17] = 0xff
    out, lse = _attend(q, pools, "head", table, lens, window, sinks)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[2, 3:, 17] = True
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], got[0][~bad]) and torch.equal(lse, got[1])
    pools[0].view(torch.uint8)[page, 0, at, 5] = 0x7f
    out, lse = _attend(q, pools, "head", table, lens, window, sinks)
    assert out[2, :3].isnan().all() and lse[2, :3].isnan().all()
    assert torch.equal(lse[2, 3:], got[1][2, 3:]) and torch.equal(out[:2], got[0][:2])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attend_queries_of_any_size(dt):
    """Queries from the type's smallest to its largest, and ones that are not finite."""
    rng = np.random.default_rng(8)
    d, n, ps = 128, 70, 16
    table, P, codes, scales = _attend_state(rng, [n] * 6, 1, d, "i8", ps, 16, "token")
    q = rng.standard_normal((6, 1, d))
    top = torch.finfo(TYPES[dt]).max
    q[0] *= 1e-6 if dt == "f16" else 1e-38
    q[1] *= top / 8 / np.abs(q[1]).max()
    q[2, 0, 3:] *= 1e-4
    q[3] = 0
    q = torch.from_numpy(q).to(TYPES[dt]).to(DEV)
    q[4, 0, 9], q[5, 0, 11] = float("inf"), float("nan")
    big = 1e-3 if dt == "f16" else 2.0 ** -110
    for s in scales[:1]:
        s *= big if dt == "f16" else 1
    pools = [_to_pool(c, "token", "i8") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    for scale, rows in ((1.0, [0, 2, 3]), (2.0 ** -8 if dt == "f16" else 2.0 ** -124, [0, 1, 2, 3])):
        want = V.attend(_np(q)[rows], codes[0], codes[1], scales[0], scales[1], table[rows], [n] * len(rows), 0, 0, scale, "i8")
        out, lse = _attend(q, pools, "token", table, [n] * 6, scale=scale)
        _check_attend((out[rows], lse[rows]), want, n, d, TYPES[dt])
        assert out[4:].isnan().all()


@pytest.mark.parametrize("Hq", [4, 8, 16])
def test_attend_small_codes(Hq):
    """I8 codes of -2 .. 2 beside one large one a block: the keys enter the product as code + 128, so their sums are rounded at
    that size: 2^-23 of sum |q| (|code| + 128) for each of the product's d / 16 steps and the sums of q, twice."""
    rng = np.random.default_rng(13)
    d, ps, n = 128, 16, 333
    table, P = _tables(rng, [n], ps)
    codes = [rng.integers(-2, 3, (P, ps, 1, d)).astype(np.int8) for _ in range(2)]
    codes[0][:, 3, :, 7] = 127
    codes = [c.view(np.uint8) for c in codes]
    scales = [np.full((P, 1, 1), 0.25, np.float32), np.full((P, 1, 1), 2.0 ** -6, np.float32)]
    q = torch.from_numpy(rng.standard_normal((1, Hq, d))).half().to(DEV)
    pools = [_to_pool(c, "head", "i8") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    want = V.attend(_np(q), codes[0], codes[1], scales[0], scales[1], table, [n], 0, 0, d ** -0.5, "i8")
    most = (np.abs(_np(q)) * (127 + 128)).sum(-1) * 0.25 * d ** -0.5
    want[3] = want[3] + most * 2 * (d / 16 + d + 8) / (d + 8)   # (bounds() multiplies by (d + 8) 2^-23)
    _check_attend(_attend(q, pools, "head", table, [n]), want, n, d, torch.float16)


def test_attend_repeats_bit_for_bit_and_shares_a_workspace():
    """One workspace for the 8-bit and the 16-bit calls in turn, without lse; the same bits every time."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(9)
    lens, d, ps = [4000, 33, 2500, 700], 128, 16
    table, P, codes, scales = _attend_state(rng, lens, 2, d, "i8", ps, 16, "head")
    pools = [_to_pool(c, "head", "i8") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    full = [torch.randn((P, 2, ps, d), device=DEV).half() for _ in range(2)]
    q = torch.randn((4, 8, d), device=DEV).half()
    o16 = torch.empty_like(q)
    p16 = F.paged_params(q, o16, full[0], "head", _i32(table))
    p8 = F.paged8_params(q, q, pools[0], pools[2], "head", _i32(table))
    ws = torch.zeros(max(F.paged_attend_workspace_bytes(p16), F.paged_prefill_workspace_bytes(p16), F.paged8_attend_workspace_bytes(p8)),
                     dtype=torch.uint8, device=DEV)
    first, _ = _attend(q, pools, "head", table, lens, lse=False)
    for _ in range(5):
        out, _ = _attend(q, pools, "head", table, lens, ws=ws, lse=False)
        assert torch.equal(out, first)
        F.paged_attend(p16, *full, _i32(table), _i32(lens), q, o16, None, ws)
        F.paged_prefill(p16, *full, _i32(table), _i32(lens), _i32([0, 1, 2, 3, 4]), q, o16, None, ws)
    assert F.paged_status(ws) == 0


# --- prompts -----------------------------------------------------------------------

PROMPTS = [
    # lengths, Hq, Hkv, d, type, window, sinks
    ([1], 1, 1, 64, "f16", 0, 0),
    ([0, 7, 128, 0, 129, 300], 24, 8, 128, "f16", 0, 0),
    ([200, 1, 513], 6, 2, 64, "bf16", 0, 0),
    ([300, 40], 5, 1, 128, "bf16", 33, 2),
    ([700], 4, 4, 64, "f16", 256, 130),
    ([1500], 2, 1, 128, "f16", 0, 0),                  # cut along its keys
    ([1300, 1100], 2, 1, 64, "bf16", 0, 0),
    ([90] * 40, 4, 2, 128, "bf16", 0, 0),
]


def _prompt(q, k, v, starts, window=0, sinks=0, positions=None, B=None, ws=None, lse=True, scale=None):
    from dictionary_sparse_kv_gb300 import fadkv as F
    out = torch.full_like(q, 99.0)
    l = torch.full(q.shape[:2], 99.0, device=DEV) if lse else None
    p = F.prompt_params(q, k, v, out, len(starts) - 1, window, sinks, scale, l)
    if ws is None:
        ws = torch.zeros(F.prompt_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    F.prompt_attend(p, q, k, v, _i32(starts), out, l, ws, positions=None if positions is None else _i32(positions))
    torch.cuda.synchronize()
    assert F.paged_status(ws) == 0
    return out, l


def _prompt_state(rng, T, Hq, hkv, d, dt):
    q = torch.from_numpy(rng.standard_normal((T, Hq, d)) * 1.5).to(TYPES[dt]).to(DEV)
    k = torch.from_numpy(rng.standard_normal((T, hkv + 1, d))).to(TYPES[dt]).to(DEV)[:, :hkv]
    v = torch.from_numpy(rng.standard_normal((T, 3 * hkv * d))).to(TYPES[dt]).to(DEV)[:, 2 * hkv * d:].view(T, hkv, d)
    return q, k, v


def _check_prompt(got, q, k, v, starts, window, sinks, dt, refused=(), scale=None):
    d = q.shape[2]
    o, l, qn, kn, vn = _np(got[0]), _np(got[1]), _np(q), _np(k), _np(v)
    T = q.shape[0]
    for b in range(len(starts) - 1):
        a, e = min(starts[b], T), min(starts[b + 1], T)
        n = e - a
        if b in refused:
            assert (o[a:e] == 0).all() and (l[a:e] == -np.inf).all()
            continue
        want = U.attend_rows(qn[a:e], kn[a:e], vn[a:e], np.ones(n, bool), list(range(n)), window, sinks, scale or d ** -0.5)
        e_out, e_lse = U.bounds(*want, d, torch.finfo(TYPES[dt]).eps, 1)
        assert (np.abs(o[a:e] - want[0]) <= e_out).all(), b
        fine = np.isfinite(want[1])
        assert (np.abs(l[a:e] - want[1])[fine] <= e_lse[fine]).all() and fine.all(), b
    assert (o[starts[-1]:] == 99).all() and (l[starts[-1]:] == 99).all()


@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompt(i):
    lens, Hq, hkv, d, dt, window, sinks = PROMPTS[i]
    rng = np.random.default_rng(400 + i)
    starts = [0] + np.cumsum(lens).tolist()
    q, k, v = _prompt_state(rng, starts[-1] + 5, Hq, hkv, d, dt)
    got = _prompt(q, k, v, starts, window, sinks)
    _check_prompt(got, q, k, v, starts, window, sinks, dt)


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (64, "f16")])
def test_prompts_keep_apart(d, dt):
    """What is not finite in one prompt, or behind the last one, reaches no other; a refused prompt sees nothing; rows past T
    are left out."""
    rng = np.random.default_rng(11)
    lens = [130, 70, 200, 3, 150]
    starts = [0] + np.cumsum(lens).tolist()
    T = starts[-1]
    q, k, v = _prompt_state(rng, T + 200, 4, 2, d, dt)
    positions = [j for n in lens for j in range(n)] + [-1] * 200
    clean = _prompt(q, k, v, starts, positions=positions)
    k[starts[2]:starts[3]], v[starts[2]:starts[3]], q[starts[2]:starts[3]] = float("nan"), float("inf"), float("-inf")
    k[T:], v[T:] = float("nan"), float("inf")
    for j in range(starts[2], starts[3]):
        positions[j] = -1
    got = _prompt(q, k, v, starts, positions=positions)
    _check_prompt(got, q, k, v, starts, 0, 0, dt, refused=(2,))
    other = [j for j in range(T) if not starts[2] <= j < starts[3]]
    assert torch.equal(got[0][other], clean[0][other]) and torch.equal(got[1][other], clean[1][other])
    # a prompt that passes T, and one behind it
    cut = starts[1] + 40
    part = _prompt(q[:cut], k[:cut], v[:cut], starts)
    assert torch.equal(part[0], clean[0][:cut]) and torch.equal(part[1], clean[1][:cut])


def test_prompts_as_the_pages_answer_them():
    """The same prompts through pages: the same kernel, within rounding of one another."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(12)
    lens, ps, d = [300, 128, 77], 64, 128
    starts = [0] + np.cumsum(lens).tolist()
    q, k, v = _prompt_state(rng, starts[-1], 8, 2, d, "f16")
    got = _prompt(q, k, v, starts, window=100, sinks=5)
    table, P = _tables(rng, lens, ps)
    pools = [torch.zeros((P, ps, 2, d), dtype=torch.float16, device=DEV) for _ in range(2)]
    slots = torch.tensor(_slots(table, [0] * 3, lens, ps), device=DEV)
    for pool, x in zip(pools, (k, v)):
        pool.view(-1, 2, d)[slots] = x
    out = torch.empty_like(q)
    p = F.paged_params(q, out, pools[0], "token", _i32(table), 100, 5)
    ws = torch.zeros(F.paged_prefill_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    F.paged_prefill(p, *pools, _i32(table), _i32(lens), _i32(starts), q, out, None, ws)
    assert torch.equal(out, got[0])


def test_no_prompts():
    q = torch.ones((5, 2, 64), dtype=torch.float16, device=DEV)
    k = torch.ones((5, 1, 64), dtype=torch.float16, device=DEV)
    out, lse = _prompt(q, k, k, [0])
    assert (out == 99).all() and (lse == 99).all()
    out, lse = _prompt(q, k, k, [0, 0, 0])
    assert (out == 99).all() and (lse == 99).all()
    _prompt(q[:0], k[:0], k[:0], [0, 0])
