"""The paged-cache calls (page plans, head norms with rotation and append,
attention of single tokens and of chunks over the pages) against plain
implementations in 64 bits, through the C ABI (needs a GPU).

Whole numbers: equal.  Rotated vectors: half a step of the stored type plus
what 32-bit arithmetic allows (stated at the test).  Attention: the bounds of
paged_util.bounds, element by element.
"""
import math

import numpy as np
import pytest

from tests import paged_util as U

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


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


# --- page plans -------------------------------------------------------------

def _run_plan(add, lengths, table, free, count, ps, cap, in_place=False):
    from dictionary_sparse_kv_gb300 import fadkv as F
    B = len(add)
    p = F.page_params(B, ps, len(free), table.shape[1], cap)
    t, f, n, c = _i32(table), _i32(free), _i32(lengths), _i32([count])
    no, co = (n, c) if in_place else (torch.full_like(n, -7), torch.full_like(c, -7))
    starts, refused = torch.full((B + 1,), -7, dtype=torch.int32, device=DEV), _i32([-7])
    pos, slots = (torch.full((max(cap, 1),), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    F.page_plan(p, _i32(add), n, t, f, c, no, co, starts, pos, slots, refused)
    torch.cuda.synchronize()
    g = lambda x: x.cpu().numpy()
    return dict(table=g(t), free=g(f), lengths=g(no), count=g(co), starts=g(starts), positions=g(pos)[:cap],
                slots=g(slots)[:cap], refused=g(refused))


def _plan_state(rng, B, ps, mp, spare, longest):
    lens = rng.integers(0, min(longest, mp * ps) + 1, B)
    lens[rng.random(B) < 0.2] //= ps
    need = -(-lens // ps)
    P = int(need.sum()) + spare
    order = rng.permutation(P).astype(np.int32)
    table = np.full((B, mp), -1, np.int32)
    o = 0
    for b in range(B):
        table[b, :need[b]] = order[o:o + need[b]]
        o += need[b]
    free = np.full(P, -1, np.int32)
    free[:P - o] = order[o:]
    return lens, table, free, P - o


PLANS = [
    # B, ps, max_pages, spare pages, longest, most new tokens, share ending, rows kept
    (1, 16, 4, 4, 40, 1, 0.0, 1),
    (16, 16, 40, 16, 600, 1, 0.0, 16),
    (33, 8, 20, 30, 150, 40, 0.2, None),              # pages run out: later requests are refused
    (33, 8, 20, 500, 150, 40, 0.2, 300),              # rows run out
    (257, 64, 6, 400, 380, 70, 0.1, None),            # some would pass max_pages
    (1025, 16, 16, 3000, 200, 3, 0.05, None),         # more requests than threads
    (40, 16, 80, 2000, 900, 400, 0.1, None),          # rows over the whole grid (more than one block writes)
    (3, 1024, 3, 9, 2048, 1500, 0.3, 9000),
    (2500, 8, 3, 100, 24, 2, 0.5, 6000),
]


@pytest.mark.parametrize("B,ps,mp,spare,longest,most,ending,cap", PLANS)
@pytest.mark.parametrize("in_place", [False, True])
def test_page_plan(B, ps, mp, spare, longest, most, ending, cap, in_place):
    rng = np.random.default_rng(B * 31 + ps)
    lens, table, free, count = _plan_state(rng, B, ps, mp, spare, longest)
    add = rng.integers(0, most + 1, B)
    add[rng.random(B) < ending] = -1
    T = int(np.maximum(add, 0).sum())
    cap = T + 5 if cap is None else cap
    want = U.plan(add, lens, table, free, count, ps, cap)
    got = _run_plan(add, lens, table, free, count, ps, cap, in_place)
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def test_page_plan_edges():
    """No requests; lengths and counts outside their ranges are clamped; a bad page in the table gives no slot; the
    same inputs twice give the same plan."""
    empty = np.zeros((0, 3), np.int32)
    r = _run_plan([], [], empty, np.arange(4, dtype=np.int32), 3, 8, 5)
    assert r["starts"].tolist() == [0] and r["count"].tolist() == [3] and r["refused"].tolist() == [0]
    assert (r["positions"] == -1).all() and (r["slots"] == -1).all()
    table = np.array([[99, -1], [1, 2], [-5, 0]], np.int32)
    free = np.array([3, 4, 5, 6, 7, 0], np.int32)
    for add, lens, count in (([1, 1, 1], [3, 99, -4], 77), ([1, -1, 1], [3, 16, 2], -3), ([0, 0, 0], [1, 2, 3], 2),
                             ([2 ** 31 - 1] * 3, [1, 2, 3], 2)):
        want = U.plan(add, lens, table, free, count, 8, 6)
        for _ in range(2):
            got = _run_plan(add, lens, table, free, count, 8, 6)
            for k in want:
                assert np.array_equal(got[k], want[k]), (k, add)


# --- norm, rotation, append ---------------------------------------------------

def _pool(shape, layout, dtype, fill=0.0):
    pages, hkv, ps, d = shape
    t = torch.full((pages, hkv, ps, d) if layout == "head" else (pages, ps, hkv, d), fill, dtype=dtype, device=DEV)
    return t


ROPES = [
    # T, Hq, Hkv, d, type, q type, kv type, rotated, pairs, scaling, norms, ps, layout
    (1, 1, 1, 64, "f16", "f16", "f16", 64, False, "plain", "qk", 8, "head"),
    (1, 24, 8, 128, "f16", "f32", "f16", 128, False, "parts", "qk", 16, "head"),
    (19, 5, 5, 64, "f32", "f16", "bf16", 32, True, "stretch", "", 32, "token"),
    (37, 7, 1, 128, "bf16", "bf16", "bf16", 64, False, "linear", "q", 8, "token"),
    (130, 3, 3, 128, "bf16", "f32", "f32", 16, False, "plain", "k", 64, "head"),
    (67, 8, 2, 64, "f16", "bf16", "f32", 64, True, "parts", "qk", 16, "token"),
    (5, 2, 1, 128, "f32", "f32", "f32", 0, False, "plain", "qk", 16, "head"),        # no rotation
    (700, 32, 8, 128, "f16", "f16", "f16", 128, True, "linear", "qk", 16, "head"),  # warps that take several steps
    (2500, 9, 3, 64, "bf16", "bf16", "f16", 48, False, "plain", "qk", 16, "token"),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,dt,qt,kt,rd,pairs,scaling,norms,ps,layout", ROPES)
def test_qk_norm_rope(T, Hq, Hkv, d, dt, qt, kt, rd, pairs, scaling, norms, ps, layout):
    from dictionary_sparse_kv_gb300 import fadkv as F
    g = torch.Generator().manual_seed(T * 7 + d)
    kw = dict(base=500000.0, factor=8.0, scaling=scaling, original=8192.0, slow=1.0, fast=4.0)
    amp, eps = (1.25 if scaling == "parts" else 1.0), 1e-5
    fused = torch.randn((T, (Hq + 2 * Hkv) * d + 8), generator=g).to(TYPES[dt]).to(DEV)   # rows further apart than full
    q, k, v = (x.view(T, -1, d) for x in fused[:, :-8].split([Hq * d, Hkv * d, Hkv * d], 1))
    q[T // 2] *= 0                                            # a row of zeros: eps alone under the root
    w = (1 + 0.3 * torch.randn((2, d), generator=g)).to(TYPES[dt]).to(DEV)
    wq, wk = (w[0] if "q" in norms else None), (w[1] if "k" in norms else None)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1                                      # the largest position
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32)
    if T > 4:
        pos[1], slots[2], slots[3] = -1, -1, pages * ps       # an empty row; slots outside the pool
    posd, slotsd = pos.to(DEV), slots.to(DEV)
    kp, vp = (_pool((pages, Hkv, ps, d), layout, TYPES[kt], 3.0) for _ in range(2))
    qo = torch.full((T, Hq, d), 7.0, dtype=TYPES[qt], device=DEV)
    ko = torch.full((T, Hkv, d), 7.0, dtype=TYPES[kt], device=DEV)
    F.qk_norm_rope(F.qk_params(q, k, v, qo, kp, layout, eps), F.rope_init(d, rd, pairs, amplitude=amp, **kw), q, k, v, wq, wk,
                   posd, slotsd, qo, ko, kp, vp)
    torch.cuda.synchronize()
    f = U.frequencies(rd, **kw) if rd else np.zeros(0)
    p = pos.numpy().astype(np.int64)
    wn = lambda x: None if x is None else _np(x)
    for x, wt, out in ((q, wq, qo), (k, wk, ko)):
        y, mag = U.norm_rope(_np(x), wn(wt), eps, p, f, rd, pairs, amp)
        # 32-bit arithmetic: the mean of d squares and its root (d 2^-24 + 2^-22), products and sums (6 2^-24), cosine
        # and sine from an angle of 24 bits (pi 2^-24) to two steps (2^-23); then half a step of the stored type
        e = torch.finfo(out.dtype).eps
        tol = mag * (d * 2.0 ** -24 + 2.0 ** -22 + (6 + math.pi) * 2.0 ** -24 + 2.0 ** -22) + e / 2 * np.abs(y) * 1.001 + 2.0 ** -25
        assert (np.abs(_np(out) - y) <= tol).all(), np.abs(_np(out) - y).max()
    # the pools: exactly k_out and v where a slot asks for them, untouched elsewhere
    for pool, x in ((kp, ko), (vp, v.to(TYPES[kt]))):
        want = torch.full((pages * ps, Hkv, d), 3.0, dtype=TYPES[kt], device=DEV)
        live = (posd >= 0) & (slotsd >= 0) & (slotsd < pages * ps)
        want[slotsd[live].long()] = x[live]
        got = pool if layout == "token" else pool.transpose(1, 2)
        assert torch.equal(got.reshape(pages * ps, Hkv, d), want)


def test_qk_norm_rope_without_pool_or_keys_out():
    """No slots: queries and keys alone, equal to what the call with a pool gives; no k_out: the pools alone; T = 0."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    T, Hq, Hkv, d = 21, 6, 2, 128
    q, k, v = (torch.randn((T, h, d), device=DEV).half() for h in (Hq, Hkv, Hkv))
    pos, slots = _i32(np.arange(T)), _i32(np.arange(T))
    rope = F.rope_init(d, d)
    kp, vp = (_pool((3, Hkv, 8, d), "head", torch.float16) for _ in range(2))
    qo, q2 = (torch.empty((T, Hq, d), device=DEV) for _ in range(2))
    ko, k2 = torch.empty_like(k), torch.empty_like(k)
    F.qk_norm_rope(F.qk_params(q, k, v, qo, kp), rope, q, k, v, None, None, pos, slots, qo, ko, kp, vp)
    F.qk_norm_rope(F.qk_params(q, k, v, q2, None), rope, q, k, v, None, None, pos, None, q2, k2, None, None)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    F.qk_norm_rope(F.qk_params(q, k, v, q2, kp2), rope, q, k, v, None, None, pos, slots, q2, None, kp2, vp2)
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)
    e = lambda h: torch.empty((0, h, d), dtype=torch.float16, device=DEV)
    F.qk_norm_rope(F.qk_params(e(6), e(2), e(2), e(6), kp), rope, e(6), e(2), e(2), None, None, None, slots, e(6), None, kp, vp)
    torch.cuda.synchronize()


# --- attention --------------------------------------------------------------------

class Case:
    """Random pools and tables; unseen tokens hold NaN, so reading one shows."""

    def __init__(self, lens, Hq, Hkv, d, dt, ps, new=None, window=0, sinks=0, layout="head", scale=None, seed=0, qscale=2.0,
                 bad_pages=(), q_pad=0, spare_columns=1):
        g = torch.Generator().manual_seed(seed * 1000 + sum(lens) + Hq)
        B, self.dt = len(lens), TYPES[dt]
        self.lens, self.new = list(lens), [1] * B if new is None else list(new)
        need = [-(-max(l, 0) // ps) for l in lens]
        pages, mp = sum(need) + 3, max(max(need), 1) + spare_columns
        order = torch.randperm(pages, generator=g).tolist()
        self.table = np.full((B, mp), -1, np.int32)
        kp, vp = (torch.full((pages, Hkv, ps, d), math.nan) for _ in range(2))
        o = 0
        for b, l in enumerate(lens):
            for j in range(need[b]):
                self.table[b, j] = order[o]
                n = min(ps, l - j * ps)
                # tokens that no query of the chunk sees stay NaN
                first = l - self.new[b]
                t = np.arange(j * ps, j * ps + n)
                seen = np.ones(n, bool) if window == 0 else (t < sinks) | (t > first - window)
                rows = torch.from_numpy(np.nonzero(seen)[0])
                kp[order[o], :, rows] = torch.randn((Hkv, len(rows), d), generator=g)
                vp[order[o], :, rows] = torch.randn((Hkv, len(rows), d), generator=g)
                o += 1
        for b, j, page in bad_pages:
            self.table[b, j] = page
        if layout == "token":
            kp, vp = kp.transpose(1, 2).contiguous(), vp.transpose(1, 2).contiguous()
        self.k, self.v = kp.to(self.dt).to(DEV), vp.to(self.dt).to(DEV)
        T = sum(self.new)
        q = (qscale * torch.randn((T, Hq * d + q_pad), generator=g)).to(self.dt).to(DEV)
        self.q = q[:, :Hq * d].view(T, Hq, d)
        self.out = torch.full((T, Hq * d + q_pad), 9.0, dtype=self.dt, device=DEV)[:, :Hq * d].view(T, Hq, d)
        self.lse = torch.full((T, Hq), 9.0, device=DEV)
        self.d, self.ps, self.layout, self.window, self.sinks = d, ps, layout, window, sinks
        self.scale = d ** -0.5 if scale is None else scale
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.prefill = new is not None

    def run(self, workspace=None, **kw):
        from dictionary_sparse_kv_gb300 import fadkv as F
        t = _i32(self.table)
        p = F.paged_params(self.q, self.out, self.k, self.layout, t, self.window, self.sinks, self.scale)
        if workspace is None:
            ask = F.paged_prefill_workspace_bytes if self.prefill else F.paged_attend_workspace_bytes
            workspace = torch.zeros(max(ask(p), 1), dtype=torch.uint8, device=DEV)
        if self.prefill:
            F.paged_prefill(p, self.k, self.v, t, _i32(self.lens), _i32(self.starts), self.q, self.out, self.lse, workspace, **kw)
            self.ws = workspace
        else:
            F.paged_attend(p, self.k, self.v, t, _i32(self.lens), self.q, self.out, self.lse, workspace, **kw)
        return self

    def check(self):
        torch.cuda.synchronize()
        if self.prefill:
            assert int(self.ws[:16].max()) == 0           # no wait ran out; the counters are back at zero
        kp, vp, q = _np(self.k), _np(self.v), _np(self.q)
        got, lse = _np(self.out), _np(self.lse)
        eps = torch.finfo(self.dt).eps
        for b, l in enumerate(self.lens):
            l = max(l, 0)
            rows = slice(self.starts[b], self.starts[b + 1])
            k, ok = U.gather(kp, self.table[b], l, self.layout)
            v, _ = U.gather(vp, self.table[b], l, self.layout)
            pos = l - self.new[b] + np.arange(self.new[b])
            want = U.attend_rows(q[rows], k, v, ok, pos, self.window, self.sinks, self.scale)
            e_out, e_lse = U.bounds(*want, self.d, eps, 1 if self.prefill else 2)
            assert np.isfinite(got[rows]).all(), b
            err = np.abs(got[rows] - want[0])
            assert (err <= e_out).all(), (b, err.max(), (err / e_out).max())
            empty = ~np.isfinite(want[1])
            assert np.array_equal(np.isneginf(lse[rows]), empty), b
            assert (got[rows][empty] == 0).all()
            d = np.abs(lse[rows][~empty] - want[1][~empty])
            assert (d <= e_lse[~empty]).all(), (b, d.max())
        return self


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130]

DECODES = [
    dict(lens=EDGES, Hq=24, Hkv=8, d=128, dt="f16", ps=16),
    dict(lens=EDGES, Hq=4, Hkv=4, d=64, dt="bf16", ps=8, layout="token"),
    dict(lens=[5, 900, 33], Hq=8, Hkv=1, d=128, dt="bf16", ps=32),
    dict(lens=[77, 300], Hq=12, Hkv=1, d=128, dt="f16", ps=64),           # more than eight heads a KV head
    dict(lens=[77, 300], Hq=40, Hkv=2, d=64, dt="f16", ps=64),            # two pieces a KV head
    dict(lens=[40, 90, 3], Hq=35, Hkv=5, d=64, dt="f16", ps=128, layout="token"),
    dict(lens=[9000], Hq=2, Hkv=1, d=128, dt="f16", ps=16),               # one request over many CTAs
    dict(lens=[30000], Hq=1, Hkv=1, d=64, dt="bf16", ps=64),              # more pieces than are joined at once
    dict(lens=[20000, 3, 9000], Hq=3, Hkv=1, d=128, dt="f16", ps=256),    # the same, in uneven shares
    dict(lens=[5000, 1, 0, 3000, 64], Hq=6, Hkv=2, d=128, dt="bf16", ps=1024),
    dict(lens=[100] * 150, Hq=3, Hkv=3, d=64, dt="f16", ps=16),           # more requests than threads
    dict(lens=EDGES + [500], Hq=6, Hkv=2, d=128, dt="f16", ps=16, window=40, sinks=0),
    dict(lens=EDGES + [500], Hq=6, Hkv=2, d=64, dt="bf16", ps=16, window=20, sinks=5, layout="token"),
    dict(lens=[500, 70, 3], Hq=4, Hkv=2, d=128, dt="f16", ps=32, window=1, sinks=0),
    dict(lens=[500, 70, 3], Hq=4, Hkv=2, d=128, dt="f16", ps=32, window=64, sinks=1000),
    dict(lens=[500, 70], Hq=4, Hkv=2, d=128, dt="f16", ps=32, window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    dict(lens=[200, 50], Hq=4, Hkv=2, d=128, dt="f16", ps=16, scale=0.0),
    dict(lens=[200, 50], Hq=4, Hkv=2, d=128, dt="f16", ps=16, scale=-0.3),
    dict(lens=[200, 50], Hq=4, Hkv=2, d=128, dt="bf16", ps=16, qscale=100.0),   # one key takes it all
    dict(lens=[200, 50, 17], Hq=4, Hkv=2, d=128, dt="f16", ps=16, q_pad=64),
    # pages outside the pool: their tokens are not seen, all of a request's among them
    dict(lens=[100, 40, 16], Hq=4, Hkv=2, d=128, dt="f16", ps=16, bad_pages=[(0, 0, -1), (0, 3, 10 ** 6), (2, 0, -5)]),
]


@pytest.mark.parametrize("i", range(len(DECODES)))
def test_paged_attend(i):
    Case(**DECODES[i]).run().check()


def test_paged_attend_without_lse_and_lengths_outside():
    """lse may be left out; lengths below 0 and above the table's are clamped."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    c = Case([48, 32], 4, 2, 128, "f16", 16, spare_columns=0)
    c.run().check()
    want = c.out.clone()
    p = F.paged_params(c.q, c.out, c.k, "head", _i32(c.table))
    ws = torch.zeros(F.paged_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    F.paged_attend(p, c.k, c.v, _i32(c.table), _i32([10 ** 6, 32]), c.q, c.out, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)                    # 10^6 is clamped to the table's 48
    F.paged_attend(p, c.k, c.v, _i32(c.table), _i32([-3, 32]), c.q, c.out, None, ws)
    torch.cuda.synchronize()
    assert (c.out[0] == 0).all() and torch.equal(c.out[1], want[1])


def test_paged_attend_shares_one_workspace_and_repeats_bit_for_bit():
    """Calls of different shapes in turn on one workspace, each run again later: the same bits."""
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    cases = [Case(**DECODES[i]) for i in (0, 6, 4, 12, 9, 7, 8)]
    first = [(c.run(ws).check().out.clone(), c.lse.clone()) for c in cases]
    for _ in range(3):
        for c, (o, l) in zip(cases, first):
            c.out.fill_(5), c.lse.fill_(5)
            c.run(ws)
            torch.cuda.synchronize()
            assert torch.equal(c.out, o) and torch.equal(c.lse, l)


PREFILLS = [
    dict(lens=[1], new=[1], Hq=4, Hkv=2, d=128, dt="f16", ps=16),
    dict(lens=[150], new=[150], Hq=3, Hkv=1, d=128, dt="f16", ps=16),
    dict(lens=[300, 0, 40, 129], new=[70, 0, 40, 1], Hq=6, Hkv=2, d=128, dt="bf16", ps=32),
    dict(lens=[65, 64, 63, 200], new=[65, 64, 3, 17], Hq=4, Hkv=4, d=64, dt="f16", ps=8, layout="token"),
    dict(lens=[20, 5], new=[30, 7], Hq=4, Hkv=2, d=64, dt="bf16", ps=16),          # more rows than tokens: some see nothing
    dict(lens=[700], new=[260], Hq=5, Hkv=1, d=128, dt="f16", ps=64, window=100, sinks=0),
    dict(lens=[700, 90], new=[300, 90], Hq=4, Hkv=2, d=64, dt="bf16", ps=16, window=33, sinks=5, layout="token"),
    dict(lens=[400], new=[400], Hq=2, Hkv=2, d=128, dt="f16", ps=128, window=1, sinks=0),
    dict(lens=[400], new=[150], Hq=2, Hkv=1, d=128, dt="f16", ps=16, window=128, sinks=200),
    dict(lens=[300], new=[300], Hq=2, Hkv=1, d=64, dt="f16", ps=16, window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    dict(lens=[90], new=[33], Hq=80, Hkv=1, d=64, dt="f16", ps=16),                # a wide group
    dict(lens=[90], new=[33], Hq=140, Hkv=1, d=64, dt="f16", ps=16),               # wider than a tile's rows
    dict(lens=[200, 50], new=[40, 50], Hq=4, Hkv=2, d=128, dt="bf16", ps=16, qscale=100.0),
    dict(lens=[200, 50], new=[40, 50], Hq=4, Hkv=2, d=128, dt="f16", ps=1024, q_pad=64, scale=-0.2),
    dict(lens=[100, 40, 16], new=[60, 40, 16], Hq=4, Hkv=2, d=128, dt="f16", ps=16,
         bad_pages=[(0, 0, -1), (0, 3, 10 ** 6), (2, 0, -5)]),
    dict(lens=[30 + i for i in range(140)], new=[1 + i % 5 for i in range(140)], Hq=2, Hkv=1, d=64, dt="f16", ps=16),
    dict(lens=[1500], new=[600], Hq=2, Hkv=1, d=128, dt="bf16", ps=256),
    # few rows on many keys: cut along the keys
    dict(lens=[3000], new=[5], Hq=6, Hkv=2, d=128, dt="f16", ps=16),
    dict(lens=[3000, 100, 0, 2100], new=[40, 7, 0, 90], Hq=4, Hkv=2, d=64, dt="bf16", ps=32, layout="token"),
    dict(lens=[5000], new=[1], Hq=2, Hkv=2, d=128, dt="bf16", ps=64),
    dict(lens=[4000, 1100], new=[70, 33], Hq=3, Hkv=1, d=128, dt="f16", ps=16, window=2000, sinks=130),
    dict(lens=[2500], new=[17], Hq=140, Hkv=1, d=64, dt="f16", ps=128),
    dict(lens=[1200], new=[1300], Hq=1, Hkv=1, d=64, dt="f16", ps=16),
    dict(lens=[2048], new=[3], Hq=4, Hkv=2, d=128, dt="f16", ps=128, scale=-0.3, bad_pages=[(0, j, -1) for j in range(3, 12)]),
    dict(lens=[2048], new=[3], Hq=4, Hkv=2, d=128, dt="f16", ps=128, bad_pages=[(0, j, 10 ** 9) for j in range(16)]),
]


@pytest.mark.parametrize("i", range(len(PREFILLS)))
def test_paged_prefill(i):
    Case(**PREFILLS[i]).run().check()


# more tiles than multiprocessors and 2 to 96 requests: the tiles come by the keys that they see
TURNS = [
    dict(lens=[0, 900, 17, 300, 1000], new=[0, 400, 17, 350, 1], Hq=64, Hkv=1, d=64, dt="f16", ps=16),      # rows before token 0
    dict(lens=[300, 2000], new=[300, 350], Hq=64, Hkv=1, d=128, dt="bf16", ps=32),
    dict(lens=[700, 20, 1500], new=[300, 20, 400], Hq=64, Hkv=1, d=64, dt="f16", ps=16, window=200, sinks=7),
    dict(lens=[40 + 37 * i % 400 for i in range(40)], new=[1 + 29 * i % 40 for i in range(40)], Hq=40, Hkv=5, d=128, dt="f16", ps=16,
         window=100, sinks=3, layout="token"),
    dict(lens=[(i > 2) * (60 + 61 * i % 500) for i in range(64)], new=[0] * 3 + [1 + 13 * i % 60 for i in range(61)], Hq=24, Hkv=4, d=64,
         dt="bf16", ps=16, bad_pages=[(5, 0, -1), (60, 2, 10 ** 6)]),
    dict(lens=[1 + 11 * i % 250 for i in range(96)], new=[1 + 7 * i % 30 for i in range(96)], Hq=16, Hkv=4, d=64, dt="f16", ps=16),
    dict(lens=[0] * 33, new=[20] * 33, Hq=8, Hkv=8, d=64, dt="f16", ps=16),                                  # nothing is seen
]


@pytest.mark.parametrize("i", range(len(TURNS)))
def test_paged_prefill_of_several_requests(i):
    Case(**TURNS[i]).run().check()


def test_both_calls_share_one_workspace():
    """Single tokens and chunks, cut along their keys and not, in turn on one workspace: the same bits each time."""
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    cases = [Case(**DECODES[0]), Case(**PREFILLS[17]), Case(**DECODES[6]), Case(**PREFILLS[2]), Case(**DECODES[12]), Case(**PREFILLS[18]), Case(**DECODES[8])]
    first = [(c.run(ws).check().out.clone(), c.lse.clone()) for c in cases]
    for _ in range(2):
        for c, (o, l) in zip(cases, first):
            c.out.fill_(5), c.lse.fill_(5)
            c.run(ws)
            torch.cuda.synchronize()
            assert torch.equal(c.out, o) and torch.equal(c.lse, l)


def test_paged_prefill_leaves_other_rows_alone():
    """Rows of q past starts[B] are padding: neither their out nor their lse is written; T cuts rows off."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    c = Case([90, 60], 4, 2, 128, "f16", 16, new=[40, 30])
    c.run().check()
    want, wl = c.out.clone(), c.lse.clone()
    p = F.paged_params(c.q, c.out, c.k, "head", _i32(c.table))
    ws = torch.zeros(max(1, F.paged_prefill_workspace_bytes(p)), dtype=torch.uint8, device=DEV)
    c.out.fill_(5), c.lse.fill_(5)
    F.paged_prefill(p, c.k, c.v, _i32(c.table), _i32(c.lens), _i32([0, 40, 55]), c.q, c.out, c.lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(c.out[:40], want[:40]) and (c.out[55:] == 5).all() and (c.lse[55:] == 5).all()
    c.out.fill_(5), c.lse.fill_(5)
    p.T = 50
    F.paged_prefill(p, c.k, c.v, _i32(c.table), _i32(c.lens), _i32([0, 40, 70]), c.q, c.out, c.lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(c.out[:50], want[:50]) and torch.equal(c.lse[:50], wl[:50]) and (c.out[50:] == 5).all()


@pytest.mark.parametrize("d,ps", [(128, 64), (128, 8), (64, 16)])
def test_paged_prefill_full_grid_repeats_bit_for_bit(d, ps):
    """Every multiprocessor streaming its own pages (loads arrive in any order): no wait runs out, and the bits are
    the same every time."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    B, n, length, Hkv, grp = 25, 90, 4096, 8, 3
    g = torch.Generator(device=DEV).manual_seed(d + ps)
    pages = B * length // ps
    k, v = (torch.randn((pages, Hkv, ps, d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((B * n, Hkv * grp, d), generator=g, device=DEV, dtype=torch.bfloat16)
    table = torch.randperm(pages, generator=g, device=DEV).view(B, -1).to(torch.int32)
    lens, starts = _i32([length - 37 * (b % 5) for b in range(B)]), _i32(np.arange(B + 1) * n)
    out, lse = torch.empty_like(q), torch.empty((B * n, Hkv * grp), device=DEV)
    p = F.paged_params(q, out, k, "head", table)
    ws = torch.zeros(F.paged_prefill_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(20):
        out.fill_(7)
        F.paged_prefill(p, k, v, table, lens, starts, q, out, lse, ws)
        if first is None:
            first = out.clone()
        assert torch.equal(out, first)
        assert int(ws[:16].max()) == 0
    # one request against the plain form
    b = 7
    kb, vb = (x[table[b].long()].transpose(1, 2).reshape(length, Hkv, d)[:int(lens[b])] for x in (k, v))
    pos = int(lens[b]) - n + np.arange(n)
    rows = slice(b * n, (b + 1) * n)
    heads = slice(0, grp)
    want = U.attend_rows(_np(q[rows, heads]), _np(kb[:, :1]), _np(vb[:, :1]), np.ones(int(lens[b]), bool), pos, 0, 0, d ** -0.5)
    e_out, e_lse = U.bounds(*want, d, torch.finfo(torch.bfloat16).eps, 1)
    assert (np.abs(_np(out[rows, heads]) - want[0]) <= e_out).all()
    assert (np.abs(_np(lse[rows, heads]) - want[1]) <= e_lse).all()


def test_offsets_past_32_bits():
    """Pages more than 2^31 elements apart."""
    c = Case([40], 2, 1, 128, "f16", 16, new=[20])
    far = (1 << 31) // 2 + 1024                        # elements between pages: page 2 on lies past 2^31
    for name in ("k", "v"):
        small = getattr(c, name)
        n = small.shape[0]
        big = torch.empty(((n - 1) * far + 16 * 128,), dtype=c.dt, device=DEV).as_strided((n, 1, 16, 128), (far, 2048, 128, 1))
        big.copy_(small)
        setattr(c, name, big)
    c.run()
    torch.cuda.synchronize()
    out = c.out.clone()
    one = Case([40], 2, 1, 128, "f16", 16)
    one.k, one.v, one.table, one.q = c.k, c.v, c.table, c.q[-1:]
    one.run()
    torch.cuda.synchronize()
    c.k, c.v = c.k.contiguous(), c.v.contiguous()
    one.k, one.v = c.k, c.v
    one.check()
    c.check()
    assert torch.equal(c.run().out, out)


def test_on_another_stream():
    s = torch.cuda.Stream()
    for c in (Case(**DECODES[0]), Case(**PREFILLS[2])):
        c.run().check()
        want = c.out.clone()
        c.out.fill_(5)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            c.run()
        s.synchronize()
        assert torch.equal(c.out, want)


# --- together ------------------------------------------------------------------------

def _loop_state(B, Hq, Hkv, d, ps, mp, pages, cap):
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device=DEV)
    s = dict(table=torch.full((B, mp), -1, dtype=torch.int32, device=DEV), free=torch.arange(pages, dtype=torch.int32, device=DEV),
             count=_i32([pages]), lens=z(B), starts=z(B + 1), pos=z(cap), slots=z(cap), refused=z(1), add=z(B))
    s["kp"], s["vp"] = (torch.zeros((pages, Hkv, ps, d), dtype=torch.float16, device=DEV) for _ in range(2))
    return s


def _step(F, s, q, k, v, rope, ps, prefill):
    """One step of a serving loop: plan, norm + rotation + append, attention."""
    B, T = s["table"].shape[0], q.shape[0]
    F.page_plan(F.page_params(B, ps, s["kp"].shape[0], s["table"].shape[1], T), s["add"], s["lens"], s["table"], s["free"], s["count"],
                s["lens"], s["count"], s["starts"], s["pos"], s["slots"], s["refused"])
    qo, out = torch.empty_like(q), torch.empty_like(q)
    F.qk_norm_rope(F.qk_params(q, k, v, qo, s["kp"]), rope, q, k, v, None, None, s["pos"][:T], s["slots"][:T], qo, None, s["kp"], s["vp"])
    p = F.paged_params(qo, out, s["kp"], "head", s["table"], window=48, sinks=4)
    if prefill:
        F.paged_prefill(p, s["kp"], s["vp"], s["table"], s["lens"], s["starts"], qo, out, None, s["pws"])
    else:
        F.paged_attend(p, s["kp"], s["vp"], s["table"], s["lens"], qo, out, None, s["ws"])
    return out


def test_a_loop_of_steps_and_its_graph():
    """A prompt in two chunks, then decode steps, against attention over all rotated keys in 64 bits; the decode step
    captured once and replayed gives the same bits as run directly."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    B, Hq, Hkv, d, ps, mp, pages, steps = 3, 6, 2, 128, 16, 12, 40, 5
    g = torch.Generator(device=DEV).manual_seed(3)
    prompts, chunk = [61, 90, 17], [30, 45, 17]
    rope = F.rope_init(d, d)
    x = [torch.randn((h, B, 100, d), generator=g, device=DEV).half().transpose(0, 2) for h in (Hq, Hkv, Hkv)]   # [token][B][heads][d]
    two = []
    for _ in range(2):
        s = _loop_state(B, Hq, Hkv, d, ps, mp, pages, 128)
        s["ws"] = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
        s["pws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
        two.append(s)
    outs = []
    for s in two:
        got = {}
        for lo, hi in ((0, 0), (1, 0)):
            a = [(0, c) if lo == 0 else (c, n) for c, n in zip(chunk, prompts)]
            s["add"].copy_(_i32([n - m for m, n in a]))
            rows = [torch.cat([y[m:n, b] for b, (m, n) in enumerate(a)]).contiguous() for y in x]
            o = _step(F, s, *rows, rope, ps, True)
            at = 0
            for b, (m, n) in enumerate(a):
                for t in range(m, n):
                    got[b, t] = o[at]
                    at += 1
        outs.append(got)
    rows = [torch.empty((B, y.shape[2], d), dtype=torch.float16, device=DEV) for y in x]
    feed = lambda t: [r.copy_(torch.stack([y[prompts[b] + t, b] for b in range(B)])) for r, y in zip(rows, x)]
    for s in two:
        s["add"].fill_(1)
    direct, graphed = two
    feed(0)
    o = _step(F, direct, *rows, rope, ps, False)
    _step(F, graphed, *rows, rope, ps, False)
    dec = [o.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        og = _step(F, graphed, *rows, rope, ps, False)
    for t in range(1, steps):
        feed(t)
        o = _step(F, direct, *rows, rope, ps, False)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, og) and torch.equal(direct["kp"], graphed["kp"]) and torch.equal(direct["lens"], graphed["lens"])
        dec.append(o.clone())
    f = U.frequencies(d)
    for b in range(B):
        n = prompts[b] + steps
        pos = np.arange(n)
        # rotated and stored as the library stores them: rounded to binary16 (twice half a step with the queries')
        k, _ = U.norm_rope(_np(x[1][:n, b]), None, 0, pos, f, d, False, 1.0)
        q, _ = U.norm_rope(_np(x[0][:n, b]), None, 0, pos, f, d, False, 1.0)
        want = U.attend_rows(q, k, _np(x[2][:n, b]), np.ones(n, bool), pos, 48, 4, d ** -0.5)
        eps = torch.finfo(torch.float16).eps
        e_out, _ = U.bounds(*want, d, eps, 1)
        e_out += 2 * eps * want[3][..., None] * want[2] * 1.1          # scores of rounded q and k: off by eps times sum |q_i k_i|
        got = np.stack([_np(outs[0][b, t]) for t in range(prompts[b])] + [_np(dec[t][b]) for t in range(steps)])
        assert (np.abs(got - want[0]) <= e_out).all()
    assert int(direct["refused"]) == 0 and int(direct["count"]) == pages - sum(-(-(n + steps) // ps) for n in prompts)


def test_the_example_runs():
    """examples/paged_loop.py: prompts, decode steps and codes of one layer."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_loop.py")
    spec = importlib.util.spec_from_file_location("paged_loop", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(["--prompt", "20", "--steps", "3", "--requests", "3"])
    assert r["tokens"] == [23, 23, 23] and r["refused"] == 0 and r["pages left"] == 0
    # one token's output twice: rounded once each, and once more for the probabilities of the prefill; values are of the
    # order of one, so half a step is 2^-11 and |out| + sum p |v| at most 5 or so
    assert r["prefill and decode differ by"] < 2.0 ** -11 * 3 * 5
    assert all(math.isfinite(r[k + " against full"]) for k in ("window", "codes"))
