"""Values, keys and queries that are not finite, in single-token attention
over the pages (needs a GPU): what they touch and what they leave alone."""
import pytest

from tests.test_gpu_paged import DEV, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    B.build()


def _slot(c, b, token):
    return int(c.table[b, token // c.ps]), token % c.ps


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_value_that_is_not_finite_touches_its_element_alone(dt, value):
    """KV head 0 of request 1: element 17 of token 70; the other elements, heads and requests as without it."""
    lens, Hq, Hkv, d = [90, 200, 3], 6, 2, 128
    c = Case(lens, Hq, Hkv, d, dt, 16)
    c.run().check()
    want, wl = c.out.clone(), c.lse.clone()
    page, at = _slot(c, 1, 70)
    c.v[page, 0, at, 17] = value
    c.run()
    torch.cuda.synchronize()
    touched = torch.zeros_like(want, dtype=torch.bool)
    touched[1, :Hq // Hkv, 17] = True
    assert not torch.isfinite(c.out[touched]).any()
    assert torch.equal(c.out[~touched], want[~touched]) and torch.equal(c.lse, wl)
    if value != value:
        assert torch.isnan(c.out[touched]).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["key", "query"])
def test_scores_that_are_nan_touch_their_rows_alone(dt, what):
    lens, Hq, Hkv, d = [90, 200, 9000], 6, 2, 128
    c = Case(lens, Hq, Hkv, d, dt, 16)
    c.run().check()
    want, wl = c.out.clone(), c.lse.clone()
    rows = torch.zeros((3, Hq), dtype=torch.bool, device=DEV)
    if what == "key":
        for b, token in ((1, 70), (2, 8000)):                 # of the second one a piece among many
            page, at = _slot(c, b, token)
            c.k[page, 1, at, 5] = float("nan")
            rows[b, Hq // Hkv:] = True
    else:
        c.q[0, 2, 9] = float("nan")
        rows[0, 2] = True
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.out[rows]).all() and torch.isnan(c.lse[rows]).all()
    assert torch.equal(c.out[~rows], want[~rows]) and torch.equal(c.lse[~rows], wl[~rows])
