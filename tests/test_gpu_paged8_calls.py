"""Calls of the 8-bit paged cache and of prompts among one another: everything that a call writes is taken back before it is made
again, on another stream and from a graph, also with other inputs in the same buffers; and waits of prompts that do run out
(needs a GPU)."""
import numpy as np
import pytest

from tests.test_gpu_paged8 import DEV, TYPES, _attend_state, _i32, _prompt_state, _slots, _to_pool

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


class Step:
    """One step of all four calls on buffers of its own; `fill` puts a seed's inputs there and overwrites what they write."""

    def __init__(self, fmt, d, dt):
        from dictionary_sparse_kv_gb300 import fadkv as F
        self.F, self.fmt, self.d, self.dt, self.hkv, self.ps, self.block = F, fmt, d, dt, 2, 32, 32
        self.fixed = 4, 600, 40                        # requests, most tokens of one, new rows
        B, longest, T = self.fixed
        mp = -(-longest // self.ps)
        self.table, self.lens, self.slots = _i32(np.full((B, mp), -1)), _i32([0] * B), _i32([-1] * T)
        self.starts = _i32([0] * 3)
        P = B * mp
        self.pools = [_to_pool(np.zeros((P, self.ps, self.hkv, d), np.uint8), "head", fmt) for _ in range(2)] + [
            torch.zeros((P, self.hkv, self.ps // self.block), device=DEV) for _ in range(2)]
        self.q = torch.empty((B, 8, d), dtype=TYPES[dt], device=DEV)
        self.pq, self.pk = (torch.empty((300, h, d), dtype=TYPES[dt], device=DEV) for h in (6, self.hkv))
        self.pv = torch.empty_like(self.pk)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((B, 8), device=DEV)
        self.po, self.plse = torch.empty_like(self.pq), torch.empty((300, 6), device=DEV)
        self.full = [torch.empty((P, self.hkv, self.ps, d), dtype=torch.float16, device=DEV) for _ in range(2)]
        k, v = self.pk[:T], self.pv[:T]
        self.pa = F.append8_params(k, v, self.pools[0], "head", self.pools[2])
        self.pr = F.read8_params(self.pools[0], self.pools[2], self.full[0], self.table, "head")
        self.p8 = F.paged8_params(self.q, self.out, self.pools[0], self.pools[2], "head", self.table)
        self.pp = F.prompt_params(self.pq, self.pk, self.pv, self.po, 2)
        self.ws = torch.zeros(max(F.paged8_attend_workspace_bytes(self.p8), F.prompt_attend_workspace_bytes(self.pp)), dtype=torch.uint8,
                              device=DEV)

    def fill(self, seed):
        rng = np.random.default_rng(seed)
        B, longest, T = self.fixed
        lens = [int(n) for n in rng.integers(T // 2, longest + 1, B)]
        new = [20, 5, 1, 0]
        table, P, codes, scales = _attend_state(rng, lens, self.hkv, self.d, self.fmt, self.ps, self.block, "head")
        self.table.fill_(-1)
        self.table[:, :min(table.shape[1], self.table.shape[1])] = _i32(table[:, :self.table.shape[1]])
        slots = _slots(table, [a - b for a, b in zip(lens, new)], new, self.ps)
        self.slots.fill_(-1)
        self.slots[:len(slots)] = _i32(slots)
        self.lens.copy_(_i32(lens))
        for pool, c in zip(self.pools, codes):
            pool.view(torch.uint8).fill_(0)
            pool.view(torch.uint8)[:P] = _to_pool(c, "head", self.fmt).view(torch.uint8)[:pool.shape[0]]
        for pool, s in zip(self.pools[2:], scales):
            pool.fill_(1)
            pool[:P] = torch.from_numpy(s[:pool.shape[0]] / 64).to(DEV)        # (small: most of them grow)
        self.starts.copy_(_i32([0, int(rng.integers(1, 200)), int(rng.integers(200, 301))]))
        for x, y in zip((self.pq, self.pk, self.pv), _prompt_state(rng, 300, 6, self.hkv, self.d, self.dt)):
            x.copy_(y)
        self.q.copy_(torch.from_numpy(rng.standard_normal(self.q.shape)))
        for x in (*self.full, self.out, self.lse, self.po, self.plse):
            x.fill_(3)
        torch.cuda.synchronize()

    def run(self):
        F, k, v = self.F, self.pk[:self.fixed[2]], self.pv[:self.fixed[2]]
        F.paged8_append(self.pa, k, v, self.slots, *self.pools)
        F.paged8_read(self.pr, *self.pools, self.table, self.lens, None, None, *self.full)
        F.paged8_attend(self.p8, *self.pools, self.table, self.lens, self.q, self.out, self.lse, self.ws)
        F.prompt_attend(self.pp, self.pq, self.pk, self.pv, self.starts, self.po, self.plse, self.ws)

    def results(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (*[p.view(torch.uint8) for p in self.pools[:2]], *self.pools[2:], *self.full, self.out, self.lse,
                                    self.po, self.plse)]


@pytest.mark.parametrize("fmt,d,dt", [("i8", 128, "bf16"), ("e4m3", 64, "f16")])
def test_every_call_on_another_stream_and_replayed_with_other_inputs(fmt, d, dt):
    step = Step(fmt, d, dt)
    seeds, want = range(3), []
    for seed in seeds:
        step.fill(seed)
        before = step.results()
        step.run()
        want.append(step.results())
        # every output is written, and nothing of one input's is another's
        assert not any(torch.equal(a, b) for a, b in zip(before, want[-1]))
        assert seed == 0 or not any(torch.equal(a, b) for a, b in zip(want[-2], want[-1]))
    s = torch.cuda.Stream()
    for seed in seeds:
        step.fill(seed)
        with torch.cuda.stream(s):
            step.run()
        assert all(torch.equal(a, b) for a, b in zip(step.results(), want[seed])), seed
    step.fill(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    for seed in (1, 0, 2, 2, 1):
        step.fill(seed)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(step.results(), want[seed])), seed
    assert step.F.paged_status(step.ws) == 0


@pytest.mark.parametrize("d,dt", [(64, torch.float16), (128, torch.bfloat16)])
def test_waits_of_a_long_prompt_run_out(d, dt):
    """Waits of a nanosecond, for items of up to 4096 key tiles, several milliseconds each (a wait gives up after 256 looks at its
    barrier at least): they do run out, the status word says so, and the workspace is fit for the next call."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    T = 1 << 19
    gen = torch.Generator(device=DEV).manual_seed(d)
    q, k, v = (torch.randn((T, 1, d), generator=gen, device=DEV).to(dt) for _ in range(3))
    out, lse = torch.full_like(q, 9), torch.full((T, 1), 9.0, device=DEV)
    p = F.prompt_params(q, k, v, out, 1, lse=lse)
    ws = torch.zeros(F.prompt_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    starts = _i32([0, T])
    call = lambda: F.prompt_attend(p, q, k, v, starts, out, lse, ws)
    call()
    assert F.paged_status(ws) == 0
    want, wl = out.clone(), lse.clone()
    for row in (0, 1, 127, 128, 300, T // 2 + 77, T - 1):
        x = (k[:row + 1, 0].double() @ q[row, 0].double()) * d ** -0.5
        # one addition in 32 bits for each key tile, and the scores' and exponents' rounding
        assert abs(lse[row, 0].double() - torch.logsumexp(x, 0)) <= row / 128 * 2.0 ** -24 + 1e-4, row
    F.debug_paged_wait_limit(1)
    for _ in range(3):
        call()
    assert F.paged_status(ws, clear=False) == F.DEV_TIMEOUT
    assert F.paged_status(ws) == F.DEV_TIMEOUT and F.paged_status(ws) == 0
    F.debug_paged_wait_limit(0)
    out.fill_(5), lse.fill_(5)
    call()
    assert F.paged_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)
