"""The bounds of tests/test_gpu_paged_range.py catch what they are for: on the CPU, 64-bit attention whose
probabilities are rounded as a kernel with a mistake would round them."""
import numpy as np
import pytest

from tests import paged_range_util as R

torch = pytest.importorskip("torch")
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _round(x, t):
    return torch.from_numpy(np.asarray(x, np.float64)).to(t).double().numpy()


def _out(drops, n, v, terms, up, t):
    """The output in type t, its probabilities entering as `terms` terms of it, multiplied by `up` before the rounding."""
    exact, _ = R.expected(drops, n, v)
    p = np.exp(-np.array(drops, np.float64)) * up
    used = _round(p, t)
    if terms == 2:
        used = used + _round(p - used, t)
    return _round(exact * (used / p)[:, None], t), exact


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n", [37, 700])
@pytest.mark.parametrize("d", [64, 128])
def test_two_term_bound(dt, n, d):
    t = TYPES[dt]
    v = torch.from_numpy(R.values(16, d, 4)).to(t).double().numpy()
    for terms, inside in ((2, True), (1, False)):
        out, exact = _out(R.DROPS[dt], n, v, terms, 1.0, t)
        tol = R.two_term_bound(exact[None], R.DROPS[dt], n, torch.finfo(t).eps)[0]
        for h in range(4):
            assert (np.abs(out - exact) <= tol)[h].all() == inside, (terms, h)


@pytest.mark.parametrize("n,drops", [(131072, (12.125,)), (32768, (15.25,)), (32768, (17.5,)), (1 << 20, (20.0,))])
def test_small_probability_bounds(n, drops):
    """Binary16 probabilities of at most 1 lose these; of at most 2^15 (single tokens) they do not."""
    t = torch.float16
    v = torch.from_numpy(R.values(64, 64, 1)).to(t).double().numpy()
    for up, inside in ((2.0 ** 15, True), (1.0, False)):
        out, exact = _out(drops, n, v, 2, up, t)
        rel, _ = R.small_bounds(drops, n, R.STEPS_DECODE(n), 2.0 ** -40)
        tol = np.abs(exact) * (2.0 ** -11 + rel[:, None]) + 2.0 ** -25
        assert (np.abs(out - exact) <= tol).all() == inside, up
