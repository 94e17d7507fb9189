"""Single-token attention with so many blocks of tokens that shares are worked
out in 64 bits (2^22 and more; needs a GPU).

The block tables repeat a handful of pages, so the cache is small and the
result is that over the distinct pages: the same weights, a log-sum-exp larger
by the log of the repeats.
"""
import pytest

from tests.test_gpu_paged import DECODES, DEV, TYPES, Case, _i32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dictionary_sparse_kv_gb300 import build as B
    B.build()


def _units(lens, Hkv):
    return sum(max(1, -(-n // 64)) for n in lens) * Hkv


# pages of 1024 tokens; lengths in pages
WIDE = [
    ("just below, many requests", [54] * 1000 + [96 + 31 * i for i in range(24)], 4, 64),
    ("above, many requests", [64] * 1000 + [1200 + 77 * i for i in range(24)], 4, 64),
    ("above, few requests", [9000 + 500 * i for i in range(9)] + [1], 6, 64),
    ("above, of one length", [16400] * 16, 1, 128),
    ("above, of one length, d = 64", [8200] * 32, 1, 64),
]


@pytest.mark.parametrize("name,pages,Hkv,d", WIDE, ids=[w[0] for w in WIDE])
def test_very_many_blocks(name, pages, Hkv, d):
    from dictionary_sparse_kv_gb300 import fadkv as F
    ps, distinct, dt = 1024, 3, "f16"
    g = torch.Generator().manual_seed(len(pages))
    kp, vp = (torch.randn((distinct, Hkv, ps, d), generator=g).to(TYPES[dt]).to(DEV) for _ in range(2))
    B = len(pages)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = (torch.arange(n) + b) % distinct
    q = torch.randn((B, Hkv, d), generator=g).to(TYPES[dt]).to(DEV)
    lens = [n * ps for n in pages]
    units = _units(lens, Hkv)
    assert (units < 1 << 22) == name.startswith("just below")
    out, lse = torch.full_like(q, 9), torch.full((B, Hkv), 9.0, device=DEV)
    p = F.paged_params(q, out, kp, "head", table.to(DEV))
    ws = torch.zeros(F.paged_attend_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    tb = table.to(DEV)
    for _ in range(2):                                        # the counters are back at zero after the first
        out.fill_(9), lse.fill_(9)
        F.paged_attend(p, kp, vp, tb, _i32(lens), q, out, lse, ws)
    torch.cuda.synchronize()
    c = Case(**DECODES[0])                                    # and a small call on the same workspace
    need = F.paged_attend_workspace_bytes(F.paged_params(c.q, c.out, c.k, c.layout, _i32(c.table)))
    c.run(ws if ws.numel() >= need else None).check()

    x = torch.einsum("bhd,phtd->bhpt", q.double(), kp.double()) * d ** -0.5
    repeats = torch.tensor([[(n - (s - b) % distinct + distinct - 1) // distinct for s in range(distinct)] for b, n in enumerate(pages)],
                           dtype=torch.float64, device=DEV).clamp(min=0)     # times page s is among the first n
    assert repeats.sum(1).tolist() == [float(n) for n in pages]
    x = x + repeats.log()[:, None, :, None]
    z = torch.logsumexp(x.flatten(2), -1)
    w = torch.exp(x - z[..., None, None])
    want, mass = torch.einsum("bhpt,phtd->bhd", w, vp.double()), torch.einsum("bhpt,phtd->bhd", w, vp.double().abs())
    # scores as in paged_util.bounds; sums: a chain of two products of 16 tokens a block of a CTA's share, 2^-23 each
    big = torch.einsum("bhd,phtd->bhpt", q.double().abs(), kp.double().abs()).amax((2, 3)) * d ** -0.5
    delta = (d + 8) * 2.0 ** -23 * big
    chain = 2 * (units / 304 + 1) * 2.0 ** -23 + 2.0 ** -18
    eps = torch.finfo(TYPES[dt]).eps
    tol = eps / 2 * want.abs() * 1.01 + 2 * (2 * delta[..., None] + chain) * mass + 2.0 ** -24
    assert ((out.double() - want).abs() <= tol).all(), ((out.double() - want).abs() / tol).max()
    assert ((lse.double() - z).abs() <= 2 * delta + chain + z.abs() * 2.0 ** -22).all()
