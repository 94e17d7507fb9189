"""Requests that a plan refuses, through the attention: their rows are no
tokens of the cache and see nothing, the other requests' are what they would
be alone (needs a GPU)."""
import numpy as np
import pytest

from tests import paged_util as U
from tests.test_gpu_paged import DEV, _i32, _np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    B.build()


def _planned_step(lens, add, spare, ps, Hq, Hkv, d, dt, seed):
    """Requests of `lens` cached tokens in pools of random values, a plan of `add` more with `spare` free pages, the new
    tokens rotated and appended."""
    from dictionary_sparse_kv_gb300 import fadkv as F
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, T = len(lens), sum(max(a, 0) for a in add)
    need = [-(-n // ps) for n in lens]
    pages, mp = sum(need) + spare, max(-(-(n + max(a, 0)) // ps) for n, a in zip(lens, add))
    table, o = np.full((B, mp), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(o, o + n)
        o += n
    s = dict(table=_i32(table), lens=_i32(lens), lens_out=_i32(lens), starts=_i32([0] * (B + 1)), refused=_i32([0]),
             pos=_i32([0] * T), slots=_i32([0] * T), count=_i32([spare]), count_out=_i32([0]))
    free = _i32(list(range(o, pages)) + [0] * o)
    s["k"], s["v"] = (torch.randn((pages, Hkv, ps, d), generator=g, device=DEV).to(dt) for _ in range(2))
    F.page_plan(F.page_params(B, ps, pages, mp, T), _i32(add), s["lens"], s["table"], free, s["count"], s["lens_out"], s["count_out"],
                s["starts"], s["pos"], s["slots"], s["refused"])
    q, k, v = (torch.randn((T, h, d), generator=g, device=DEV).to(dt) for h in (Hq, Hkv, Hkv))
    s["q"] = torch.empty_like(q)
    F.qk_norm_rope(F.qk_params(q, k, v, s["q"], s["k"]), F.rope_init(d, d), q, k, v, None, None, s["pos"], s["slots"], s["q"], None,
                   s["k"], s["v"])
    return s


def _check(s, add, out, lse, refused, p_terms, window, sinks, scale, dt):
    """Rows of the requests in `refused` are empty, the others as in 64 bits."""
    starts, lens, table = s["starts"].tolist(), s["lens_out"].tolist(), s["table"].cpu().numpy()
    kp, vp, q, out, lse = _np(s["k"]), _np(s["v"]), _np(s["q"]), _np(out), _np(lse)
    assert int(s["refused"]) == len(refused) > 0
    for b, n in enumerate(add):
        rows = slice(starts[b], starts[b + 1])
        if b in refused:
            assert (out[rows] == 0).all() and np.isneginf(lse[rows]).all(), b
        elif n > 0:
            k, ok = U.gather(kp, table[b], lens[b], "head")
            v, _ = U.gather(vp, table[b], lens[b], "head")
            want = U.attend_rows(q[rows], k, v, ok, lens[b] - n + np.arange(n), window, sinks, scale)
            e_out, e_lse = U.bounds(*want, q.shape[2], torch.finfo(dt).eps, p_terms)
            assert (np.abs(out[rows] - want[0]) <= e_out).all() and (np.abs(lse[rows] - want[1]) <= e_lse).all(), b


CHUNKS = [
    # cached, new, spare pages, window, refused: the second one's pages are too many, so the later ones that need pages are too
    ([40, 100, 17, 60], [20, 200, 20, 3], 4, 30, {1, 2}),
    ([40, 1000, 17], [2, 70, 1], 1, 0, {1}),                    # cut along the keys
    ([16 * i + 12 for i in range(70)], [1 + i % 9 + 150 * (i == 20) for i in range(70)], 12, 0, None),
]


@pytest.mark.parametrize("d,dt", [(128, torch.float16), (64, torch.bfloat16)])
@pytest.mark.parametrize("lens,add,spare,window,refused", CHUNKS)
def test_refused_chunks_see_nothing(lens, add, spare, window, refused, d, dt):
    from dictionary_sparse_kv_gb300 import fadkv as F
    s = _planned_step(lens, add, spare, 16, 6, 2, d, dt, len(lens))
    if refused is None:
        starts, pos = s["starts"].tolist(), s["pos"].tolist()
        refused = {b for b in range(len(add)) if add[b] > 0 and pos[starts[b]] < 0}
    sinks = 2 if window else 0
    out, lse = torch.full_like(s["q"], 9), torch.full(s["q"].shape[:2], 9.0, device=DEV)
    p = F.paged_params(s["q"], out, s["k"], "head", s["table"], window, sinks)
    ws = torch.zeros(max(1, F.paged_prefill_workspace_bytes(p)), dtype=torch.uint8, device=DEV)
    F.paged_prefill(p, s["k"], s["v"], s["table"], s["lens_out"], s["starts"], s["q"], out, lse, ws, positions=s["pos"])
    torch.cuda.synchronize()
    _check(s, add, out, lse, refused, 1, window, sinks, d ** -0.5, dt)


@pytest.mark.parametrize("B", [5, 50])
def test_refused_single_tokens_see_nothing(B):
    from dictionary_sparse_kv_gb300 import fadkv as F
    lens = [16 * (1 + b % 7) - (b % 3 == 0) for b in range(B)]                # two of three need a page
    s = _planned_step(lens, [1] * B, B // 3, 16, 6, 2, 128, torch.float16, B)
    refused = {b for b in range(B) if s["pos"][b] < 0}
    out, lse = torch.full_like(s["q"], 9), torch.full(s["q"].shape[:2], 9.0, device=DEV)
    p = F.paged_params(s["q"], out, s["k"], "head", s["table"])
    ws = torch.zeros(F.paged_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    F.paged_attend(p, s["k"], s["v"], s["table"], s["lens_out"], s["q"], out, lse, ws, positions=s["pos"])
    torch.cuda.synchronize()
    _check(s, [1] * B, out, lse, refused, 2, 0, 0, 128 ** -0.5, torch.float16)
