"""The 8-bit paged cache and the prompts' attention where calls meet one another and at the ends of their ranges (needs a GPU):
strides, offsets past 32 bits, very many tiles, streams, graphs, one workspace for all, waits that run out, and a serving loop of
all of it.
"""
import numpy as np
import pytest

from tests import paged8_util as V
from tests import paged_util as U
from tests.test_gpu_paged8 import (DEV, HELD, TYPES, _append, _attend, _attend_state, _check_attend, _check_prompt, _codes, _i32, _np,
                                   _prompt, _prompt_state, _random_codes, _slots, _tables, _to_pool)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    from dictionary_sparse_kv_gb300 import fadkv as F
    B.build()
    yield
    F.debug_paged_wait_limit(0)


def _spaced(pool, layout, how):
    """The pool's values in a view with gaps: wider tokens, heads and pages; or pages more than 2^31 bytes apart."""
    if how == "gaps":
        n, a, b, d = pool.shape
        big = torch.full((n, a + 1, b + 3, d + 16), 77, dtype=torch.int8, device=DEV).view(pool.dtype)[:, :a, :b, :d]
    else:
        n, a, b, d = pool.shape
        far = (1 << 31) + 4096
        big = torch.empty(((n - 1) * far + a * b * d,), dtype=torch.int8, device=DEV).view(pool.dtype).as_strided((n, a, b, d), (far, b * d, d, 1))
    big.view(torch.uint8).copy_(pool.view(torch.uint8))
    return big


@pytest.mark.parametrize("how", ["gaps", "far"])
@pytest.mark.parametrize("layout,fmt,d", [("head", "e4m3", 128), ("token", "i8", 64)])
def test_strides(how, layout, fmt, d):
    """Append, read and attention through views, against the same through dense pools."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(1)
    lens, new, ps, hkv = [70, 9], [30, 9], 64 if how == "far" else 16, 2
    table, P, codes, scales = _attend_state(rng, lens, hkv, d, fmt, ps, 16, layout)
    before = [a - b for a, b in zip(lens, new)]
    slots = _i32(_slots(table, before, new, ps))
    k, v = (torch.randn((sum(new), hkv, d), device=DEV) for _ in range(2))
    q = torch.randn((2, 4, d), device=DEV).half()
    results = []
    for wide in (False, True):
        pools = [_to_pool(c, layout, fmt) for c in codes]
        if wide:
            pools = [_spaced(p, layout, how) for p in pools]
        pools += [torch.from_numpy(s.copy()).to(DEV) for s in scales]
        _append(k, v, slots, pools, layout)
        out, lse = _attend(q, pools, layout, table, lens)
        full = [torch.zeros((table.size,) + pools[0].shape[1:], dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        if wide and how == "gaps":
            full = [torch.zeros(f.shape[:3] + (d + 8,), dtype=f.dtype, device=DEV)[..., :d] for f in full]
        p = F.read8_params(pools[0], pools[2], full[0], _i32(table), layout, None, pools[1], pools[3], full[1])
        F.paged8_read(p, *pools, _i32(table), _i32(lens), None, None, *full)
        torch.cuda.synchronize()
        results.append([out, lse, *[f.contiguous() for f in full], *[x.contiguous().view(torch.uint8) for x in pools[:2]], *pools[2:]])
        if wide and how == "gaps":                      # nothing in the gaps has been written
            base = pools[0].view(torch.uint8)
            whole = torch.as_strided(base, (pools[0].stride(0) * pools[0].shape[0],), (1,))
            assert int((whole == 77).sum()) >= whole.numel() - pools[0].numel()
    for a, b in zip(*results):
        assert torch.equal(a, b)


# pages of 1024 tokens; lengths in pages
WIDE = [
    ("one piece a CTA", [16400] * 4, 2, 64, None),
    ("many requests", [64] * 1000 + [1200 + 77 * i for i in range(24)], 4, 64, None),
    ("many requests of d = 128", [60] * 600, 2, 128, None),
    ("long tables", [3, 1], 64, 64, (1 << 21) - 5),    # so long that units are counted in 64 bits
]


@pytest.mark.parametrize("name,pages,hkv,d,columns", WIDE, ids=[w[0] for w in WIDE])
def test_very_many_tiles(name, pages, hkv, d, columns):
    """The block tables repeat three pages, so that the result is that over those: the same weights, a log-sum-exp larger by
    the log of the repeats."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    ps, distinct, fmt = 1024, 3, "e4m3"
    rng = np.random.default_rng(len(pages))
    B = len(pages)
    codes = [V.encode(np.clip(rng.standard_normal((distinct, ps, hkv, d)) * 100, -448, 448), fmt) for _ in range(2)]
    scales = [(2.0 ** rng.integers(-8, -5, (distinct, hkv, 8))).astype(np.float32) for _ in range(2)]
    pools = [_to_pool(c, "head", fmt) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    kp, vp = (torch.from_numpy(V.decode(c, fmt)).to(DEV).transpose(1, 2) * torch.from_numpy(s).to(DEV).double().repeat_interleave(ps // 8, 2)[..., None]
              for c, s in zip(codes, scales))           # [page][head][token][d]
    table = torch.full((B, columns or max(pages)), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = (torch.arange(n) + b) % distinct
    table = table.to(DEV)
    q = torch.randn((B, hkv, d), generator=torch.Generator().manual_seed(5)).half().to(DEV)
    out, lse = torch.full_like(q, 9), torch.full((B, hkv), 9.0, device=DEV)
    p = F.paged8_params(q, out, pools[0], pools[2], "head", table)
    ws = torch.zeros(F.paged8_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    for _ in range(2):                                  # the counters are back at zero after the first
        out.fill_(9), lse.fill_(9)
        F.paged8_attend(p, *pools, table, _i32([n * ps for n in pages]), q, out, lse, ws)
    torch.cuda.synchronize()
    x = torch.einsum("bhd,phtd->bhpt", q.double(), kp) * d ** -0.5
    repeats = torch.tensor([[(n - (s - b) % distinct + distinct - 1) // distinct for s in range(distinct)] for b, n in enumerate(pages)],
                           dtype=torch.float64, device=DEV).clamp(min=0)     # times page s is among the first n
    assert repeats.sum(1).tolist() == [float(n) for n in pages]
    x = x + repeats.log()[:, None, :, None]
    z = torch.logsumexp(x.flatten(2), -1)
    w = torch.exp(x - z[..., None, None])
    want, mass = torch.einsum("bhpt,phtd->bhd", w, vp), torch.einsum("bhpt,phtd->bhd", w, vp.abs())
    # scores and exponents as in paged8_util.bounds; sums: a product of 16 tokens for each tile of a warp's part (a CTA has an even
    # share, or a (request, heads) in equal parts), 2^-23 each, twice (l too)
    big = torch.einsum("bhd,phtd->bhpt", q.double().abs(), kp.abs()).amax((2, 3)) * d ** -0.5
    delta = (d + 8) * 2.0 ** -23 * big + 3 * 2.0 ** -24 * (1.45 * big + 140) + 2.0 ** -21
    units = sum(-(-n * ps // 64) for n in pages) * hkv
    chain = 2 * (units / 300 + 200) * 2.0 ** -23 + 2.0 ** -18
    lost = torch.tensor(pages, device=DEV).double()[:, None, None] * ps * 2.0 ** -36 * 448 * 2.0 ** -6    # weights below 2^-36
    eps = torch.finfo(torch.float16).eps
    tol = eps / 2 * want.abs() * 1.01 + 2 * (2 * delta[..., None] + chain) * mass + 2.0 ** -24 + lost * w.amax((2, 3))[..., None]
    assert ((out.double() - want).abs() <= tol).all(), ((out.double() - want).abs() / tol).max()
    assert ((lse.double() - z).abs() <= 2 * delta + chain + z.abs() * 2.0 ** -22).all()


def test_read_of_long_tables():
    """Tables of 2^21 pages: only what the lengths name is looked at."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(2)
    ps, hkv, d, columns = 1024, 2, 64, (1 << 21) - 5
    codes = [_random_codes(rng, (3, ps, hkv, d), "i8") for _ in range(2)]
    pools = [_to_pool(c, "token", "i8") for c in codes] + [torch.full((3, hkv, 4), 0.5, device=DEV) for _ in range(2)]
    table = torch.full((3, columns), 2, dtype=torch.int32, device=DEV)
    to = torch.full((3, columns), -1, dtype=torch.int32, device=DEV)
    first = [5, (columns - 1) * ps - 100, 7]
    lens = [20, columns * ps + 50, 7]                   # the second one is cut at the table's end
    to[0, 0], to[1, columns - 2], to[1, columns - 1] = 0, 1, 2
    out = [torch.zeros((3, ps, hkv, d), device=DEV) for _ in range(2)]
    p = F.read8_params(pools[0], pools[2], out[0], table, "token", None, pools[1], pools[3], out[1], to)
    F.paged8_read(p, *pools, table, _i32(lens), _i32(first), to, *out)
    torch.cuda.synchronize()
    for c, o in zip(codes, out):
        want = np.zeros((3, ps, hkv, d))
        want[0, 5:20] = V.decode(c[2, 5:20], "i8") / 2
        want[1, ps - 100:] = V.decode(c[2, ps - 100:], "i8") / 2
        want[2] = V.decode(c[2], "i8") / 2
        assert np.array_equal(_np(o), want)


def test_on_another_stream_and_in_a_graph():
    """Every call on a side stream and captured, with the outputs overwritten in between: the same bits."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(3)
    lens, hkv, d, ps = [500, 33, 1, 0], 2, 128, 32
    table, P, codes, scales = _attend_state(rng, lens, hkv, d, "i8", ps, 32, "head")
    pools = [_to_pool(c, "head", "i8") for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    q = torch.randn((4, 8, d), device=DEV).bfloat16()
    new = [20, 5, 1, 0]
    slots = _i32(_slots(table, [a - b for a, b in zip(lens, new)], new, ps))
    pq, pk, pv = _prompt_state(rng, 300, 6, 2, d, "f16")
    out, po = torch.empty_like(q), torch.empty_like(pq)
    full = [torch.zeros((table.size, hkv, ps, d), dtype=torch.float16, device=DEV) for _ in range(2)]
    t, ln, starts = _i32(table), _i32(lens), _i32([0, 100, 300])
    pa = F.append8_params(pk[:26], pv[:26], pools[0], "head", pools[2])
    pr = F.read8_params(pools[0], pools[2], full[0], t, "head")
    p8 = F.paged8_params(q, out, pools[0], pools[2], "head", t)
    pp = F.prompt_params(pq, pk, pv, po, 2)
    ws = torch.zeros(max(F.paged8_attend_workspace_bytes(p8), F.prompt_attend_workspace_bytes(pp)), dtype=torch.uint8, device=DEV)

    def step():
        F.paged8_append(pa, pk[:26], pv[:26], slots, *pools)
        F.paged8_read(pr, *pools, t, ln, None, None, *full)
        F.paged8_attend(p8, *pools, t, ln, q, out, None, ws)
        F.prompt_attend(pp, pq, pk, pv, starts, po, None, ws)
    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (*pools, *full, out, po)]
    clear = lambda: [x.fill_(3) for x in (*full, out, po)]

    def check():
        torch.cuda.synchronize()
        for a, b in zip((*pools, *full, out, po), want):
            assert torch.equal(a, b) or (a.dtype == torch.float16 and torch.equal(a[b != 0], b[b != 0]))
    clear()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    check()
    clear()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        clear()
        g.replay()
        check()


def test_waits_of_prompts_run_out_and_the_workspace_recovers():
    """As for the prefill over pages: waits of a nanosecond; 64 heads over 16000 tokens are some milliseconds of work."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    T = 16000
    q, k = torch.randn((T, 64, 64), device=DEV).half(), torch.randn((T, 64, 64), device=DEV).half()
    out, lse = torch.empty_like(q), torch.empty((T, 64), device=DEV)
    p = F.prompt_params(q, k, k, out, 1, lse=lse)
    ws = torch.zeros(F.prompt_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    starts = _i32([0, T])
    call = lambda: F.prompt_attend(p, q, k, k, starts, out, lse, ws)
    call()
    assert F.paged_status(ws) == 0
    want, wl = out.clone(), lse.clone()
    F.debug_paged_wait_limit(1)
    for _ in range(3):
        call()
    assert F.paged_status(ws) in (0, F.DEV_TIMEOUT)     # (most waits are over at their first look)
    F.debug_paged_wait_limit(0)
    out.fill_(5), lse.fill_(5)
    call()
    assert F.paged_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_a_serving_loop():
    """Prompts, decode steps (the last ones replayed from a graph) and a chunk: planned, rotated, prompts answered from their own
    rows, everything kept in 8 bits, single tokens answered from there, the chunk from what is read back.  One request asks for
    more pages than there are and is refused."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    rng = np.random.default_rng(4)
    B, Hq, Hkv, d, ps, mp, P, block, fmt = 4, 6, 2, 128, 32, 8, 20, 16, "i8"
    prompts, steps, chunk = [61, 140, 17, 300], 6, [30, 0, 45, 0]
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)
    table, free, count = torch.full((B, mp), -1, dtype=torch.int32, device=DEV), torch.arange(P, dtype=torch.int32, device=DEV), _i32([P])
    lens, starts, refused = z(B), z(B + 1), z(1)
    pools = [torch.zeros((P, Hkv, ps, d), dtype=torch.int8, device=DEV).view(HELD[fmt]) for _ in range(2)] + [
        torch.zeros((P, Hkv, ps // block), device=DEV) for _ in range(2)]
    rope = F.rope_init(d, d)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    keys, values = [[] for _ in range(B)], [[] for _ in range(B)]
    codes = [np.zeros((P, ps, Hkv, d), np.uint8) for _ in range(2)]
    scales = [np.zeros((P, Hkv, ps // block), np.float32) for _ in range(2)]

    def project(T):
        qkv = torch.from_numpy(rng.standard_normal((T, (Hq + 2 * Hkv) * d))).half().to(DEV)
        return [x.view(T, -1, d) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1)]

    class Step:
        """Plan, rotation and append of up to T new tokens."""

        def __init__(self, T):
            self.T, self.pos, self.slots, self.add = T, z(T), z(T), z(B)
            self.q, self.k, self.v = project(T)
            self.qo, self.ko = (torch.empty((T, h, d), dtype=torch.float16, device=DEV) for h in (Hq, Hkv))
            self.out, self.lse = torch.empty_like(self.qo), torch.empty((T, Hq), device=DEV)

        def run(self):
            F.page_plan(F.page_params(B, ps, P, mp, self.T), self.add, lens, table, free, count, lens, count, starts, self.pos, self.slots, refused)
            F.qk_norm_rope(F.qk_params(self.q, self.k, self.v, self.qo, None, k_out=self.ko), rope, self.q, self.k, self.v, None, None, self.pos,
                           None, self.qo, self.ko, None, None)
            F.paged8_append(F.append8_params(self.ko, self.v, pools[0], "head", pools[2]), self.ko, self.v, self.slots, *pools)

        def attend8(self):
            p = F.paged8_params(self.qo, self.out, pools[0], pools[2], "head", table, window=100, sinks=4)
            F.paged8_attend(p, *pools, table, lens, self.qo, self.out, self.lse, ws, positions=self.pos)

        def follow(self):
            """The same in the plain implementation; what each request has."""
            torch.cuda.synchronize()
            for x, c, s in ((self.ko, codes[0], scales[0]), (self.v, codes[1], scales[1])):
                V.append(_np(x), self.slots.tolist(), c, s, ps, block, fmt)
            for got, want in zip(pools, codes):
                assert np.array_equal(_codes(got, "head"), want)
            for got, want in zip(pools[2:], scales):
                assert np.array_equal(got.cpu().numpy(), want)

    # the prompts; the last one is refused
    first = Step(sum(prompts))
    first.add.copy_(_i32(prompts))
    first.run()
    got = _prompt(first.qo, first.ko, first.v, [0] + np.cumsum(prompts).tolist(), 100, 4, first.pos.tolist(), ws=ws)
    assert int(refused) == 1 and lens.tolist() == prompts[:3] + [0]
    _check_prompt(got, first.qo, first.ko, first.v, [0] + np.cumsum(prompts).tolist(), 100, 4, "f16", refused=(3,))
    first.follow()

    # decode steps: directly, then captured
    one = Step(B)
    one.add.copy_(_i32([1, 1, 1, 1]))
    graph = None
    for t in range(steps):
        for x, y in zip((one.q, one.k, one.v), project(B)):
            x.copy_(y * 1.3 ** t)
        if t < 2:
            one.run()
            one.attend8()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, capture_error_mode="relaxed"):
                    one.run()
                    one.attend8()
            graph.replay()
        one.follow()
        n = [p + t + 1 for p in prompts[:3]] + [t + 1]
        assert lens.tolist() == n
        want = V.attend(_np(one.qo), codes[0], codes[1], scales[0], scales[1], table.cpu().numpy(), n, 100, 4, d ** -0.5, fmt, one.pos.tolist())
        _check_attend((one.out, one.lse), want, max(n), d, torch.float16)

    # a chunk on top: kept in 8 bits, read back as pages of full vectors and answered by the prefill over those
    more = Step(sum(chunk))
    more.add.copy_(_i32(chunk))
    more.run()
    more.follow()
    n = lens.tolist()
    full = [torch.full((B * mp, Hkv, ps, d), float("nan"), dtype=torch.float16, device=DEV) for _ in range(2)]
    F.paged8_read(F.read8_params(pools[0], pools[2], full[0], table, "head"), *pools, table, lens, None, None, *full)
    own = torch.arange(B * mp, dtype=torch.int32, device=DEV).view(B, mp)
    p = F.paged_params(more.qo, more.out, full[0], "head", own, 100, 4)
    assert ws.numel() >= F.paged_prefill_workspace_bytes(p)
    F.paged_prefill(p, *full, own, lens, starts, more.qo, more.out, more.lse, ws, positions=more.pos)
    torch.cuda.synchronize()
    at = 0
    for b in (0, 2):
        k, _, ok = V.gather(codes[0], scales[0], table[b].cpu().numpy(), n[b], fmt)
        v, _, _ = V.gather(codes[1], scales[1], table[b].cpu().numpy(), n[b], fmt)
        k, v = (x.astype(np.float16).astype(np.float64) for x in (k, v))       # what is read back is rounded once
        rows = slice(at, at + chunk[b])
        want = U.attend_rows(_np(more.qo[rows]), k, v, ok, list(range(n[b] - chunk[b], n[b])), 100, 4, d ** -0.5)
        e_out, e_lse = U.bounds(*want, d, torch.finfo(torch.float16).eps, 1)
        assert (np.abs(_np(more.out[rows]) - want[0]) <= e_out).all() and (np.abs(_np(more.lse[rows]) - want[1]) <= e_lse).all()
        at += chunk[b]
