"""The bounded waits of the prefill over pages, made to run out (needs a GPU).

The limit is set to one nanosecond, so that waits give up while copies and
products are in flight.  The kernel still waits for those (with the full
limit), gives its tensor memory back and leaves the workspace's counters at
zero: no CUDA error, the status word says what happened, and the next call on
the workspace is right.
"""
import math

import pytest

from tests.test_gpu_paged import DEV, PREFILLS, TURNS, Case, _i32

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


def _long(length, new, others, d, dt, ps=1024):
    """One request of `length` tokens (one page over and over) and `others` of one token: q, out, lse, pools, tables."""
    B, T, Hq = 1 + others, new + others, 2
    g = torch.Generator(device=DEV).manual_seed(d)
    k, v = (torch.randn((2, 1, ps, d), generator=g, device=DEV).to(dt) for _ in range(2))
    q = torch.randn((T, Hq, d), generator=g, device=DEV).to(dt)
    table = torch.ones((B, -(-length // ps)), dtype=torch.int32, device=DEV)
    lens, starts = _i32([length] + [1] * others), _i32([0] + [new + i for i in range(others + 1)])
    return q, torch.full_like(q, 9), torch.full((T, Hq), 9.0, device=DEV), k, v, table, lens, starts


@pytest.mark.parametrize("d,dt", [(128, torch.float16), (64, torch.bfloat16)])
@pytest.mark.parametrize("length,new,others", [(1 << 20, 300, 256), (1 << 25, 3, 0), (1 << 25, 90, 0)])
def test_waits_run_out_drain_and_the_workspace_recovers(length, new, others, d, dt):
    """More than 256 requests: items are walked whole; fewer: cut into 64 pieces and joined.  A wait gives up after 256
    looks at its barrier at least, so each item or piece is some thousand key tiles, several milliseconds, long."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    q, out, lse, k, v, table, lens, starts = _long(length, new, others, d, dt)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    p = F.paged_params(q, out, k, "head", table)
    call = lambda: F.paged_prefill(p, k, v, table, lens, starts, q, out, lse, ws)
    call()
    assert F.paged_status(ws) == 0
    want, wl = out.clone(), lse.clone()
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


def test_short_calls_with_waits_that_give_up():
    """Waits of these may or may not run out; either way nothing faults and the workspace stays fit."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    cases = [Case(**PREFILLS[i]) for i in (2, 3, 6, 10, 17, 18)] + [Case(**TURNS[i]) for i in (0, 3)]
    F.debug_paged_wait_limit(1)
    for c in cases:
        c.run(ws)
    assert F.paged_status(ws) in (0, F.DEV_TIMEOUT)
    F.debug_paged_wait_limit(0)
    for c in cases:
        c.out.fill_(5), c.lse.fill_(5)
        c.run(ws).check()


def test_an_item_may_take_longer_than_a_wait():
    """One token on 60 million cached (a page over and over) beside 256 requests of one: its item, which is walked whole,
    takes more than the 200 ms of a wait, and is no reason to give up."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    length, ps, d, dt = 60_000_000, 1024, 64, torch.float16
    length -= length % ps
    q, out, lse, k, v, table, lens, starts = _long(length, 1, 256, d, dt, ps)
    p = F.paged_params(q, out, k, "head", table)
    ws = torch.zeros(F.paged_prefill_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    F.paged_prefill(p, k, v, table, lens, starts, q, out, lse, ws)
    end.record()
    assert F.paged_status(ws) == 0
    assert begin.elapsed_time(end) > 200
    # every page holds the same tokens: the sum over one page times the pages.  The sum in 32 bits has one addition for each
    # key tile, off by half a step (2^-24) at most
    x = (q[0].double() @ k[1, 0].double().T) * d ** -0.5
    want = torch.logsumexp(x, -1) + math.log(length / ps)
    assert ((lse[0].double() - want).abs() <= length / 128 * 2.0 ** -24 + 1e-4).all()
    assert torch.equal(out[1:], v[1, 0, 0].expand_as(out[1:]))                # requests of one token: its value


def test_a_window_of_more_than_a_billion_tokens():
    """One token on 1.2 billion cached (a page over and over) with a window of 1.1 billion: every page in it counts."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    ps, d, dt = 1024, 64, torch.float16
    length, window = 1_200_000 * ps, 1_100_000 * ps
    q, out, lse, k, v, table, lens, starts = _long(length, 1, 0, d, dt, ps)
    p = F.paged_params(q, out, k, "head", table, window=window)
    ws = torch.zeros(F.paged_prefill_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    F.paged_prefill(p, k, v, table, lens, starts, q, out, lse, ws)
    assert F.paged_status(ws) == 0
    x = (q[0].double() @ k[1, 0].double().T) * d ** -0.5
    want = torch.logsumexp(x, -1) + math.log(window / ps)
    # 64 pieces, each with one addition in 32 bits a key tile; a window of 2^30 would be off by 0.047
    assert ((lse[0].double() - want).abs() <= window / 128 / 64 * 2.0 ** -24 + 1e-4).all()
