"""Measured cases of the paged-cache operators: page plans, head norms with the position rotation, attention of single new
tokens over the pages, and attention of chunks of new tokens over the pages.

``own = False`` computes each operator in its plain form (elementary torch operations); ``own = True`` makes the library's
calls.  Head shapes are those of this repository's decode workloads (24 query heads over 8 key/value heads of 128, 32 over 8)
and generic ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def _plan(B, ps, longest, add, ended=0, ragged=1):
    """B requests of up to `longest` cached tokens; every request but the ended ones gets up to `add` new tokens."""
    return {"op": "plan", "B": B, "ps": ps, "longest": longest, "add": add, "ended": ended, "ragged": ragged}


def _rope(T, Hq, Hkv, d, dtype, q_dtype, kv_dtype, rd, layout, scaling, norm, ps=16, pool="head", far=4096):
    return {"op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "q_dtype": q_dtype, "kv_dtype": kv_dtype,
            "rd": rd, "layout": layout, "scaling": scaling, "norm": norm, "ps": ps, "pool": pool, "far": far}


def _decode(B, longest, Hq, Hkv, d, dtype, ps, window=0, sinks=0, pool="head", ragged=1):
    return {"op": "decode", "B": B, "longest": longest, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "ps": ps,
            "window": window, "sinks": sinks, "pool": pool, "ragged": ragged}


def _prefill(B, new, cached, Hq, Hkv, d, dtype, ps, window=0, sinks=0, pool="head", ragged=1):
    """B requests of up to `new` query tokens each, on top of up to `cached` tokens that are in the pages already."""
    return {"op": "prefill", "B": B, "new": new, "cached": cached, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "ps": ps,
            "window": window, "sinks": sinks, "pool": pool, "ragged": ragged}


def listed():
    cases = [
        # one decode step of 16 sequences: a token each, a new page now and then; what every step of a serving loop starts with
        ("plan, 16 decoding", _plan(16, 16, 4096, 1)),
        # a busy server: prompts of very different lengths come in while other requests decode and some end
        ("plan, 1000 mixed", _plan(1000, 16, 8192, 257, ended=31)),
        # the decode step's keys and queries: 16 tokens, queries in 32 bits as the attention over codes takes them
        ("rotate, 16 tokens", _rope(16, 24, 8, 128, "f16", "f32", "f16", 128, "half", "parts", True, far=131072)),
        # a long prompt
        ("rotate, 16384 tokens", _rope(16384, 32, 8, 128, "bf16", "bf16", "bf16", 128, "half", "linear", True, far=131072)),
        # part of the head, neighbouring pairs, 32-bit activations, an odd number of tokens
        ("rotate, part of the head", _rope(3001, 12, 5, 64, "f32", "f16", "f16", 32, "pairs", "stretch", False, ps=32, pool="token")),
        # one sequence of a few hundred tokens: latency
        ("decode, 1 sequence", _decode(1, 777, 24, 8, 128, "f16", 16, ragged=0)),
        # the 16-sequence decode step over full vectors
        ("decode, 16 of 4096", _decode(16, 4096, 24, 8, 128, "f16", 16)),
        # a large batch with long contexts
        ("decode, 64 of 16384", _decode(64, 16384, 32, 8, 128, "bf16", 32)),
        # a recent window and a few first tokens, everything between left to the codes
        ("decode, window", _decode(113, 30000, 16, 2, 64, "bf16", 64, window=1024, sinks=4, pool="token")),
        # chunks of new tokens on top of cached ones
        ("chunks, 8 of 500", _prefill(8, 500, 4000, 24, 8, 128, "f16", 16)),
        # a prompt from its first token on
        ("prompt, 8192", _prefill(1, 8192, 0, 24, 8, 128, "bf16", 64, ragged=0)),
        # a long prompt with a window
        ("prompt, window", _prefill(2, 12001, 0, 8, 2, 64, "f16", 32, window=1024, sinks=4, pool="token")),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "decode", "decode", "prefill", "prefill"])
    ps = rng.choice([8, 16, 32, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    pool = rng.choice(["head", "token"])
    d = rng.choice([64, 128, 128])
    ragged = rng.randrange(1, 1000)
    if op == "plan":
        B = _log(rng, 1, 1000)
        return _plan(B, ps, _log(rng, 16, 8192), rng.choice([1, 1, _log(rng, 2, 257)]), ended=rng.randrange(0, 1 + B // 8), ragged=ragged)
    Hkv = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8] + ([16] if Hkv <= 2 else []))
    if op == "rope":
        rd = rng.choice([d, d, d // 2, d // 4])
        return _rope(_log(rng, 1, 16384), min(Hq, 32 // Hkv * Hkv), Hkv, d, rng.choice(["f16", "bf16", "f32"]), rng.choice(["f16", "bf16", "f32"]),
                     rng.choice(["f16", "bf16"]), rd, rng.choice(["half", "pairs"]), rng.choice(["plain", "linear", "stretch", "parts"]),
                     rng.random() < 0.6, ps=ps, pool=pool, far=_log(rng, 1000, 1000000))
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    sinks = rng.choice([0, 1, 4, 37]) if window else 0
    if op == "decode":
        longest = _log(rng, 1, 32768)
        most = 64 * 16384 * 8 * 128 // (longest * Hkv * d)
        return _decode(_log(rng, 1, max(1, min(256, most))), longest, Hq, Hkv, d, dtype, ps, window, sinks, pool, ragged)
    new = _log(rng, 1, 8192)
    cached = rng.choice([0, _log(rng, 1, 8192)])
    most = min(32, 8192 * 8192 * 24 * 128 // (new * (2 * cached + new) * Hq * d), 24 * 8192 * 8192 // (Hq * new * (new + cached)))
    while most < 1:  # as dear as the largest listed case at most
        new, cached = max(1, new // 2), cached // 2
        most = min(32, 8192 * 8192 * 24 * 128 // (new * (2 * cached + new) * Hq * d), 24 * 8192 * 8192 // (Hq * new * (new + cached)))
    return _prefill(_log(rng, 1, most), new, cached, Hq, Hkv, d, dtype, ps, window, sinks, pool, ragged)


def _spread(n, longest, ragged, least=1):
    """n lengths up to `longest`, at least one of them that long; all of them where ragged is 0."""
    if not ragged:
        return [longest] * n
    r = random.Random(ragged * 7919 + n)
    got = [r.randint(min(least, longest), longest) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _plan_lengths(c):
    r = random.Random(c["ragged"])
    lens = _spread(c["B"], c["longest"], c["ragged"], 0)
    add = [c["add"] if r.random() < 0.5 else r.randint(0 if c["add"] > 1 else 1, c["add"]) for _ in range(c["B"])]
    for b in r.sample(range(c["B"]), c["ended"]):
        add[b] = -1
    return lens, add


def _prefill_lengths(c):
    new = _spread(c["B"], c["new"], c["ragged"])
    old = _spread(c["B"], c["cached"], c["ragged"] and c["ragged"] + 1, 0)
    return new, [a + b for a, b in zip(new, old)]


def _visible(position, window, sinks):
    """Keys that a query at `position` sees."""
    if position < 0:
        return 0
    n = position + 1
    return n if not window or n <= window else window + min(sinks, n - window)


def work(c):
    op = c["op"]
    if op == "plan":
        lens, add = _plan_lengths(c)
        T = sum(max(a, 0) for a in add)
        pages = sum(-(-(l + a) // c["ps"]) - -(-l // c["ps"]) for l, a in zip(lens, add) if a > 0) + sum(-(-l // c["ps"]) for l, a in zip(lens, add) if a < 0)
        return {"bytes": 4 * (5 * c["B"] + 2 * T + 2 * pages), "flops": 0}
    if op == "rope":
        T, q, kv, s = c["T"], c["Hq"] * c["d"], c["Hkv"] * c["d"], SIZES[c["dtype"]]
        return {"bytes": T * ((q + 2 * kv) * s + q * SIZES[c["q_dtype"]] + 3 * kv * SIZES[c["kv_dtype"]] + 8), "flops": T * (q + kv) * 7}
    if op == "decode":
        seen = sum(_visible(l - 1, c["window"], c["sinks"]) for l in _spread(c["B"], c["longest"], c["ragged"]))
        rows = c["B"] * c["Hq"]
        return {"bytes": seen * c["Hkv"] * c["d"] * 4 + rows * (c["d"] * 4 + 4) + 4 * (seen // c["ps"] + 2 * c["B"]), "flops": 4 * seen * c["Hq"] * c["d"]}
    pairs = keys = 0
    new, total = _prefill_lengths(c)
    W, S = c["window"], c["sinks"]
    for n, l in zip(new, total):
        if W:
            pairs += sum(_visible(p, W, S) for p in range(l - n, l))
            keys += min(l, n + W - 1 + S)
        else:
            pairs += n * (l - n) + n * (n + 1) // 2
            keys += l
    rows = sum(new) * c["Hq"]
    return {"bytes": keys * c["Hkv"] * c["d"] * 4 + rows * (c["d"] * 4 + 4), "flops": 4 * pairs * c["Hq"] * c["d"]}


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pools(g, pages, Hkv, ps, d, dtype, layout, zero=False):
    """Key and value pools; a page is [Hkv][ps][d] ("head") or [ps][Hkv][d] ("token")."""
    shape = (pages, Hkv, ps, d) if layout == "head" else (pages, ps, Hkv, d)
    if zero:
        return [torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(2)]
    return [torch.randn(shape, generator=g, dtype=dtype, device=DEV) for _ in range(2)]


def _tables(g, lens, ps, spare=0):
    """Block tables over a pool whose pages are handed out in a random order; entries past a request's last page are -1.
    Page 0 stays out of use.  Also: the pages left over, and the number of pages of the pool."""
    need = [-(-l // ps) for l in lens]
    most = max(1, max(need))
    total = sum(need) + spare
    order = (torch.randperm(total, generator=g, device=DEV) + 1).to(torch.int32)
    n = _ints(need)[:, None]
    off = torch.cumsum(n, 0) - n
    col = torch.arange(most, device=DEV)[None]
    table = torch.where(col < n, order[(off + col).clamp(max=max(0, total - 1))] if total else -1, torch.full_like(n, -1)).to(torch.int32)
    return table.contiguous(), order[sum(need):].contiguous(), total + 1


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    dt = DTYPES.get(c.get("dtype"))
    if c["op"] == "plan":
        lens, add = _plan_lengths(c)
        ps = c["ps"]
        widest = -(-(c["longest"] + c["add"]) // ps)
        grown = sum(max(a, 0) // ps + 1 for a in add)
        table, free, pages = _tables(g, lens, ps, grown)
        rows = torch.full((c["B"], widest), -1, dtype=torch.int32, device=DEV)
        rows[:, :table.shape[1]] = table[:, :widest]
        pool = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        pool[:free.numel()] = free
        T = sum(max(a, 0) for a in add)
        cap = T + T // 16 + 1  # rows that a captured step keeps for more requests than it has now
        s |= {"lens": _ints(lens), "add": _ints(add), "table": rows, "free": pool, "count": _ints([free.numel()]), "cap": cap, "pages": pages}
        s["out"] = {k: torch.empty(n, dtype=torch.int32, device=DEV) for k, n in
                    (("lens", c["B"]), ("count", 1), ("starts", c["B"] + 1), ("positions", cap), ("slots", cap), ("refused", 1))}
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["plan"] = F.page_params(c["B"], ps, pages, widest, cap)
    elif c["op"] == "rope":
        T, Hq, Hkv, d, ps = c["T"], c["Hq"], c["Hkv"], c["d"], c["ps"]
        qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, dtype=dt, device=DEV)  # one projection's output, cut in three
        s["q"], s["k"], s["v"] = (x.view(T, -1, d) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=1))
        w = 1 + 0.1 * torch.randn((2, d), generator=g, dtype=torch.float32, device=DEV)
        s["wq"], s["wk"] = (w[0].to(dt), w[1].to(dt)) if c["norm"] else (None, None)
        pages = -(-T // ps) + 1
        s["slots"] = (torch.randperm((pages - 1) * ps, generator=g, device=DEV)[:T] + ps).to(torch.int32)
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        if T > 8:  # rows that hold no token of this step
            s["slots"][T - T // 16 - 1:] = -1
            s["positions"][T - T // 16 - 1:] = -1
        kv = DTYPES[c["kv_dtype"]]
        s["k_pages"], s["v_pages"] = _pools(g, pages, Hkv, ps, d, kv, c["pool"], zero=True)
        s["q_out"] = torch.empty((T, Hq, d), dtype=DTYPES[c["q_dtype"]], device=DEV)
        s["k_out"] = torch.empty((T, Hkv, d), dtype=kv, device=DEV)
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["rope"] = F.rope_init(d, c["rd"], interleaved=c["layout"] == "pairs", base=500000.0, scaling=c["scaling"], factor=8.0,
                                    original=8192.0, slow=1.0, fast=4.0, amplitude=1.2 if c["scaling"] == "parts" else 1.0)
            s["plan"] = F.qk_params(s["q"], s["k"], s["v"], s["q_out"], s["k_pages"], c["pool"], eps=1e-6)
    else:
        B, Hq, Hkv, d, ps = c["B"], c["Hq"], c["Hkv"], c["d"], c["ps"]
        new, lens = ([1] * B, _spread(B, c["longest"], c["ragged"])) if c["op"] == "decode" else _prefill_lengths(c)
        s["table"], _, pages = _tables(g, lens, ps)
        s["lens"], T = _ints(lens), sum(new)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        s["starts"], s["most"], s["longest"] = _ints(starts), max(new), max(lens)
        s["k_pages"], s["v_pages"] = _pools(g, pages, Hkv, ps, d, dt, c["pool"])
        s["q"] = 2 * torch.randn((T, Hq, d), generator=g, dtype=dt, device=DEV)
        s["out"] = torch.empty((T, Hq, d), dtype=dt, device=DEV)
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=DEV)
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["plan"] = F.paged_params(s["q"], s["out"], s["k_pages"], c["pool"], s["table"], window=c["window"], sinks=c["sinks"])
            ask = F.paged_attend_workspace_bytes if c["op"] == "decode" else F.paged_prefill_workspace_bytes
            s["workspace"] = torch.zeros(max(1, ask(s["plan"])), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "decode": _plain_decode, "prefill": _plain_prefill}[op](s)
    from dictionary_sparse_kv_gb300 import fadkv as F
    if op == "plan":
        o = s["out"]
        F.page_plan(s["plan"], s["add"], s["lens"], s["table"], s["free"], s["count"], o["lens"], o["count"], o["starts"], o["positions"],
                    o["slots"], o["refused"])
        return {"table": s["table"], "free": s["free"], **o}
    if op == "rope":
        F.qk_norm_rope(s["plan"], s["rope"], s["q"], s["k"], s["v"], s["wq"], s["wk"], s["positions"], s["slots"], s["q_out"], s["k_out"],
                       s["k_pages"], s["v_pages"])
        return {"q": s["q_out"], "k": s["k_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "decode":
        F.paged_attend(s["plan"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["q"], s["out"], s["lse"], s["workspace"])
    else:
        F.paged_prefill(s["plan"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["starts"], s["q"], s["out"], s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_plan(s):
    c, table, free, cap, P = s["case"], s["table"], s["free"], s["cap"], s["pages"]
    ps, mp = c["ps"], table.shape[1]
    lens, add = s["lens"].long(), s["add"].long()
    n, ended = add.clamp(min=0), add < 0
    have = (lens + ps - 1) // ps
    col = torch.arange(mp, device=DEV)[None]
    # pages of ended requests go to the end of the free list
    back = torch.where(ended, have, 0)
    upto = torch.cumsum(back, 0)
    at = s["count"].long() + (upto - back)[:, None] + col
    at = torch.where(ended[:, None] & (col < have[:, None]), at, P).clamp(max=P)
    free = torch.cat([free, free[:1]]).scatter(0, at.flatten(), table.flatten())[:P]
    F = (s["count"].long() + upto[-1:]).clamp(max=P)
    # requests are served in their order while pages last; a page is taken from the list's end
    starts = torch.cat([torch.zeros_like(n[:1]), torch.cumsum(n, 0)])
    grown = lens + n
    fits = (grown <= mp * ps) & (starts[1:] <= cap)
    need = torch.where((n > 0) & fits, (grown + ps - 1) // ps - have, 0)
    before = torch.cumsum(need, 0) - need
    served = fits & ((need == 0) | (before + need <= F)) & (n > 0)
    need = torch.where(served, need, 0)
    j = col - have[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    table = torch.where(fresh, free[(F - 1 - before[:, None] - j).clamp(0, P - 1)], table)
    s["table"].copy_(table)
    s["free"].copy_(free)
    t = torch.arange(cap, device=DEV)
    b = torch.searchsorted(starts, t, right=True).sub(1).clamp(max=c["B"] - 1)
    ok = (t < starts[-1]) & served[b]
    pos = lens[b] + t - starts[b]
    slot = table[b, (pos // ps).clamp(0, mp - 1)].long() * ps + pos % ps
    i32 = torch.int32
    return {"table": s["table"], "free": s["free"], "lens": torch.where(ended, 0, torch.where(served, grown, lens)).to(i32),
            "count": (F - need.sum()).to(i32), "starts": starts.to(i32), "positions": torch.where(ok, pos, -1).to(i32),
            "slots": torch.where(ok, slot, -1).to(i32), "refused": ((n > 0) & ~served).sum().to(i32).view(1)}


def _frequencies(c):
    """Radians a position, in 64 bits, of the rotated pairs; and what the rotated part is multiplied by."""
    rd = c["rd"]
    base, factor, original, slow, fast = 500000.0, 8.0, 8192.0, 1.0, 4.0
    if c["scaling"] == "stretch":
        base *= factor ** (rd / (rd - 2))
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=DEV) / rd)
    if c["scaling"] == "linear":
        f = f / factor
    if c["scaling"] == "parts":
        keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f, 1.2 if c["scaling"] == "parts" else 1.0


def _plain_rope(s):
    c = s["case"]
    rd, ps, Hkv, d = c["rd"], c["ps"], c["Hkv"], c["d"]
    f, amplitude = _frequencies(c)
    angle = s["positions"].double()[:, None] * f  # 64 bits: 32 lose the angle of a far position
    cos, sin = ((x * amplitude).float()[:, None] for x in (angle.cos(), angle.sin()))
    keep = (s["positions"] >= 0)[:, None, None]

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.float()
        r, rest = x[..., :rd], x[..., rd:]
        if c["layout"] == "half":
            a, b = r[..., :rd // 2], r[..., rd // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.where(keep, torch.cat([r, rest], -1), 0)

    q = turn(s["q"], s["wq"]).to(DTYPES[c["q_dtype"]])
    k = turn(s["k"], s["wk"]).to(DTYPES[c["kv_dtype"]])
    slot = s["slots"].long()
    page, at = slot.clamp(min=0) // ps, slot.clamp(min=0) % ps
    for pool, x in ((s["k_pages"], k), (s["v_pages"], s["v"])):
        rows = pool if c["pool"] == "token" else pool.transpose(1, 2)
        # rows without a slot write what is there at slot 0, which no token has
        rows[page, at] = torch.where((slot >= 0)[:, None, None], x.to(pool.dtype), rows[page, at])
    return {"q": q, "k": k, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _tokens(pool, table, layout):
    """[B][pages * ps][Hkv][d] of a pool through the block tables."""
    x = pool[table.clamp(min=0).long()]
    if layout == "head":
        x = x.transpose(2, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])


def _softmax_out(sc, mask, v):
    """out and log-sum-exp of masked scores [..., rows, keys] and values [..., keys, d], in 32 bits."""
    sc = sc.masked_fill_(~mask, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0, m)
    p = sc.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, 1)
    return out, (m + l.log()).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    lens = s["lens"].long()[:, None]
    ps, W, S = c["ps"], c["window"], c["sinks"]
    if W:  # only the first tokens and the window
        j = torch.arange(S + W, device=DEV)[None]
        at = torch.where(j < S, j, lens - W + j - S)
        mask = (at >= 0) & (at < lens) & ((j < S) | (at >= S))
        page = torch.gather(s["table"].long(), 1, (at.clamp(min=0) // ps).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
        k, v = ((p if c["pool"] == "token" else p.transpose(1, 2))[page, at.clamp(min=0) % ps] for p in (s["k_pages"], s["v_pages"]))
    else:
        k, v = (_tokens(p, s["table"], c["pool"]) for p in (s["k_pages"], s["v_pages"]))
        mask = torch.arange(k.shape[1], device=DEV)[None] < lens
    k, v = (x.transpose(1, 2).float() for x in (k, v))  # [B][Hkv][keys][d]
    q = s["q"].view(B, Hkv, Hq // Hkv, d).float()
    out, lse = _softmax_out(torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5, mask[:, None, None], v)
    return {"out": out.reshape(B, Hq, d).to(s["q"].dtype), "lse": lse.reshape(B, Hq)}


def _plain_prefill(s):
    c = s["case"]
    B, Hq, Hkv, d, W, S = c["B"], c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    L, N, T = s["longest"], s["most"], s["q"].shape[0]
    starts, lens = s["starts"].long(), s["lens"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(N, device=DEV)[None]
    row = (starts[:-1, None] + i).clamp(max=T - 1)  # [B][N]
    pos = (lens - n)[:, None] + i
    key = torch.arange(L, device=DEV)
    mask = (key <= pos[..., None]) & (i < n[:, None])[..., None]
    if W:
        mask &= (key > pos[..., None] - W) | (key < S)
    k, v = (_tokens(p, s["table"], c["pool"])[:, :L].transpose(1, 2).float() for p in (s["k_pages"], s["v_pages"]))
    q = s["q"][row].view(B, N, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d).float() * d ** -0.5
    sc = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, N, L)
    out, lse = _softmax_out(sc, mask[:, None, None], v[:, :, None])
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(starts, t, right=True).sub(1)
    at = t - starts[b]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, d)[b, at]
    lse = lse.permute(0, 3, 1, 2).reshape(B, N, Hq)[b, at]
    return {"out": out.to(s["q"].dtype), "lse": lse.contiguous()}


# ---------------------------------------------------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def exact(c, seed):
    if c["op"] == "plan":
        return None  # whole numbers alone
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    return _exact_attention(c, s)


def _exact_rope(c, s):
    rd, ps, d = c["rd"], c["ps"], c["d"]
    turns = []
    for i in range(rd // 2):
        base, f = 500000.0, 0.0
        if c["scaling"] == "stretch":
            base = base * 8.0 ** (rd / (rd - 2.0))
        f = math.exp(-2.0 * i / rd * math.log(base))
        if c["scaling"] == "linear":
            f /= 8.0
        elif c["scaling"] == "parts":
            share = min(1.0, max(0.0, (8192.0 * f / (2 * math.pi) - 1.0) / 3.0))
            f = share * f + (1 - share) * f / 8.0
        turns.append(f)
    wide = torch.complex128
    angle = s["positions"].double()[:, None] * torch.tensor(turns, dtype=torch.float64, device=DEV)
    unit = torch.polar(torch.full_like(angle, 1.2 if c["scaling"] == "parts" else 1.0), angle)[:, None]
    live = (s["positions"] >= 0).double()[:, None, None]

    def whole(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        head = x[..., :rd]
        z = torch.complex(head[..., :rd // 2], head[..., rd // 2:]) if c["layout"] == "half" else torch.complex(head[..., ::2], head[..., 1::2])
        z = z.to(wide) * unit
        y = x.clone()
        if c["layout"] == "half":
            y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
        else:
            y[..., 0:rd:2], y[..., 1:rd:2] = z.real, z.imag
        return y * live

    k, v = whole(s["k"], s["wk"]), s["v"].double()
    pools = []
    has = torch.nonzero(s["slots"] >= 0).flatten()
    slot = s["slots"][has].long()
    for x in (k, v):
        flat = torch.zeros((s["k_pages"].shape[0] * ps, c["Hkv"], d), dtype=torch.float64, device=DEV)
        flat[slot] = x[has]
        flat = flat.view(-1, ps, c["Hkv"], d)
        pools.append(flat if c["pool"] == "token" else flat.permute(0, 2, 1, 3).contiguous())
    return {"q": whole(s["q"], s["wq"]), "k": k, "k_pages": pools[0], "v_pages": pools[1]}


def _exact_attention(c, s):
    Hq, Hkv, d, ps, W, S = c["Hq"], c["Hkv"], c["d"], c["ps"], c["window"], c["sinks"]
    group = Hq // Hkv
    if work(c)["flops"] > 1e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for b in range(c["B"]):
        n, length = starts[b + 1] - starts[b], lens[b]
        pages = s["table"][b, :-(-length // ps)].long()
        for lo in range(0, n, 1024):  # query rows lo .. hi of the request
            hi = min(n, lo + 1024)
            first, last = length - n + lo, length - n + hi - 1
            keys = torch.arange(last + 1, device=DEV)
            if W:
                keys = keys[(keys < S) | (keys > first - W)]
            at = torch.arange(first, last + 1, device=DEV)[:, None]
            seen = keys[None] <= at
            if W:
                seen &= (keys[None] < S) | (keys[None] > at - W)
            kv = []
            for pool in (s["k_pages"], s["v_pages"]):
                pg, off = pages[keys // ps], keys % ps
                kv.append(pool[pg, off].double() if c["pool"] == "token" else pool[pg, :, off].double())
            rows = slice(starts[b] + lo, starts[b] + hi)
            for h in range(Hkv):
                heads = slice(h * group, (h + 1) * group)
                x = torch.einsum("thd,kd->htk", s["q"][rows, heads].double(), kv[0][:, h]) / math.sqrt(d)
                x = torch.where(seen, x, -math.inf)
                z = torch.logsumexp(x, -1)
                out[rows, heads] = torch.einsum("htk,kd->thd", torch.exp(x - z[..., None]), kv[1][:, h])
                lse[rows, heads] = z.T
    return {"out": out, "lse": lse}
