"""Paged attention where one key takes nearly all of the probability and very
many keys share the rest (needs a GPU): what thousands of small probabilities
add up to, and how exactly a single-token call multiplies them.

Scores are exact here: one product of two 16-bit numbers each, scale 1.  The
first token's value is 0, so that the output is made by the small
probabilities alone.
"""
import math

import numpy as np
import pytest

from tests import paged_range_util as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    B.build()


def _run(drops, length, new, d, dt, ps, layout="head"):
    """out, lse, and their values in 64 bits, of `new` query rows (None: one, by the single-token call) over `length`
    tokens; head h scores drops[h] with the first token and 0 with the others."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    n, T, H = length, new or 1, len(drops)
    v = torch.from_numpy(R.values(ps, d, H)).to(TYPES[dt])                   # pages 0 and 1; token 0 of page 0 is 0
    k = torch.zeros((2, 1, ps, d), dtype=TYPES[dt])
    k[0, 0, 0, :H] = 1
    kp, vp = k.to(DEV), v[:, None].contiguous().to(DEV)
    if layout == "token":
        kp, vp = (x.transpose(1, 2).contiguous() for x in (kp, vp))
    table = torch.ones((1, -(-n // ps)), dtype=torch.int32, device=DEV)      # page 1 over and over
    table[0, 0] = 0
    q = torch.zeros((T, H, d), dtype=TYPES[dt])
    for h, x in enumerate(drops):
        q[:, h, h] = x
        assert float(q[0, h, h]) == x
    q = q.to(DEV)
    out, lse = torch.empty_like(q), torch.empty((T, H), device=DEV)
    lens, starts = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([n], [0, T]))
    p = F.paged_params(q, out, kp, layout, table, scale=1.0)
    if new:
        ws = torch.zeros(max(1, F.paged_prefill_workspace_bytes(p)), dtype=torch.uint8, device=DEV)
        F.paged_prefill(p, kp, vp, table, lens, starts, q, out, lse, ws)
    else:
        ws = torch.zeros(F.paged_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
        F.paged_attend(p, kp, vp, table, lens, q, out, lse, ws)
    torch.cuda.synchronize()
    want = [R.expected(drops, n - T + i + 1, v.double().numpy()) for i in range(T)]
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), np.stack([w[0] for w in want]), np.stack([w[1] for w in want])


DECODE = [(131072, (12.125, 5.0, 0.0)), (32768, (15.25, 17.5, 14.875)), (1 << 20, (20.0, 24.0, 22.5))]


@pytest.mark.parametrize("dt,d,ps,layout", [("f16", 128, 64, "head"), ("f16", 64, 32, "token"), ("bf16", 128, 128, "head")])
@pytest.mark.parametrize("n,drops", DECODE)
def test_paged_attend_keeps_small_probabilities(n, drops, dt, d, ps, layout):
    out, lse, want, wl = _run(drops, n, None, d, dt, ps, layout)
    rel, e_lse = R.small_bounds(drops, n, R.STEPS_DECODE(n), 2 ** -40.0 if dt == "f16" else 0.0)
    e = torch.finfo(TYPES[dt]).eps
    tol = np.abs(want) * (e / 2 + rel[None, :, None]) + 2.0 ** -25
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) / tol).max()
    assert (np.abs(lse - wl) <= e_lse[None]).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [37, 700])
def test_paged_attend_multiplies_both_terms(dt, d, n):
    """Probabilities whose single rounding to the 16-bit type is off by a good part of half a step (the bound of the
    single-token call leaves a hundredth of that): losing the second term fails in every head."""
    drops = R.DROPS[dt]
    out, lse, want, wl = _run(drops, n, None, d, dt, 16)
    e = torch.finfo(TYPES[dt]).eps
    tol = R.two_term_bound(want, drops, n, e)
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) / tol).max()


PREFILL = [(131072, 3, (12.125, 5.0, 0.0)), (32768, 40, (15.25, 17.5, 14.875)), (1 << 20, 1, (16.5, 14.0, 15.0)),
           (32768, 12800, (15.25, 17.5, 13.125))]                           # the last one: items are not cut


@pytest.mark.parametrize("dt,d,ps,layout", [("f16", 128, 64, "head"), ("f16", 64, 32, "token"), ("bf16", 64, 128, "head")])
@pytest.mark.parametrize("n,new,drops", PREFILL)
def test_paged_prefill_keeps_small_probabilities(n, new, drops, dt, d, ps, layout):
    out, lse, want, wl = _run(drops, n, new, d, dt, ps, layout)
    steps = R.STEPS_PREFILL(n, new < 10000)
    rel, e_lse = R.small_bounds(drops, n, steps, 2 ** -32.0 if dt == "f16" else 0.0)
    e = torch.finfo(TYPES[dt]).eps
    tol = np.abs(want) * (e + rel[None, :, None]) + 2.0 ** -25               # one rounding of out, one of each probability
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) / tol).max()
    assert (np.abs(lse - wl) <= e_lse[None]).all()
