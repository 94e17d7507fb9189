"""Measured cases of the operators around the 8-bit paged cache: keys and values quantised as they are written, read back,
attention of single new tokens over the 8-bit pages, and attention of packed prompts over their own keys and values.

``own = False`` computes each operator in its plain form (elementary torch operations); ``own = True`` makes the library's
calls.  Head shapes are those of this repository's decode workloads (24 query heads over 8 key/value heads of 128, 32 over 8)
and generic ones.

An 8-bit pool holds codes (``e4m3`` numbers or whole numbers -127 .. 127); a token's value is its code times the scale of its
block of tokens and head.  A block's scale is a power of two: the least t >= 2^-126 whose largest code reaches the block's
largest value.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"f16": 2, "bf16": 2, "f32": 4}
HELD = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
LARGEST = {"e4m3": 448, "i8": 127}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def _append(B, new, cached, Hkv, d, k_dtype, v_dtype, held, ps, block, pool="head", ragged=1):
    """B requests of up to `new` new tokens each, on top of up to `cached` tokens that are in the pages already."""
    return {"op": "append", "B": B, "new": new, "cached": cached, "Hkv": Hkv, "d": d, "k_dtype": k_dtype, "v_dtype": v_dtype,
            "held": held, "ps": ps, "block": block, "pool": pool, "ragged": ragged}


def _read(B, longest, Hkv, d, dtype, held, ps, block, last=0, pool="head", ragged=1):
    """The tokens of B requests (their last ones with `last`) as pages of full vectors."""
    return {"op": "read", "B": B, "longest": longest, "Hkv": Hkv, "d": d, "dtype": dtype, "held": held, "ps": ps, "block": block,
            "last": last, "pool": pool, "ragged": ragged}


def _attend(B, longest, Hq, Hkv, d, dtype, held, ps, block, window=0, sinks=0, pool="head", ragged=1):
    return {"op": "attend", "B": B, "longest": longest, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "held": held, "ps": ps,
            "block": block, "window": window, "sinks": sinks, "pool": pool, "ragged": ragged}


def _prompt(B, longest, Hq, Hkv, d, dtype, window=0, sinks=0, ragged=1):
    return {"op": "prompt", "B": B, "longest": longest, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "window": window, "sinks": sinks,
            "ragged": ragged}


def listed():
    cases = [
        # the decode step of 16 sequences: a token each, in blocks that began earlier; now and then a scale grows
        ("append, 16 decoding", _append(16, 1, 4096, 8, 128, "f16", "f16", "e4m3", 16, 16)),
        # long prompts
        ("append, prompts", _append(3, 8000, 0, 8, 128, "bf16", "bf16", "i8", 64, 32)),
        # chunks on top of cached tokens: 16-bit keys as the rotation gives them, 32-bit values, blocks that are half full
        ("append, chunks", _append(37, 200, 3000, 5, 64, "f16", "f32", "e4m3", 32, 32, pool="token")),
        # a chunk's cached tokens, before the attention of the chunk over full vectors
        ("read, 8 of 4096", _read(8, 4096, 8, 128, "f16", "e4m3", 16, 16)),
        # the recent tokens of many requests, on their way to an encode
        ("read, the last 1024", _read(113, 30000, 2, 64, "f16", "i8", 64, 64, last=1024, pool="token")),
        # one sequence of a few hundred tokens: latency
        ("single, 1 sequence", _attend(1, 777, 24, 8, 128, "f16", "e4m3", 16, 16, ragged=0)),
        # the 16-sequence decode step
        ("single, 16 of 4096", _attend(16, 4096, 24, 8, 128, "f16", "i8", 64, 64)),
        # a large batch with long contexts
        ("single, 64 of 16384", _attend(64, 16384, 32, 8, 128, "bf16", "e4m3", 32, 32)),
        # a recent window and a few first tokens, everything between left to the codes
        ("single, window", _attend(113, 30000, 16, 2, 64, "bf16", "e4m3", 64, 16, window=1024, sinks=4, pool="token")),
        # a few short prompts
        ("prompts, 7 of 300", _prompt(7, 300, 24, 8, 128, "f16")),
        # prompts of very different lengths in one call
        ("prompts, 4 of 6000", _prompt(4, 6000, 32, 8, 128, "bf16")),
        # long prompts with a window
        ("prompts, window", _prompt(3, 9001, 8, 2, 64, "f16", window=1024, sinks=4)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "prompt", "prompt"])
    ps = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= ps])
    held, pool = rng.choice(["e4m3", "i8"]), rng.choice(["head", "token"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["f16", "bf16"])
    ragged = rng.randrange(1, 1000)
    Hkv = rng.choice([1, 2, 4, 5, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8] + ([16] if Hkv <= 2 else []))
    if op == "append":
        new = rng.choice([1, _log(rng, 1, 8000)])
        cached = rng.choice([0, _log(rng, 1, 8000)])
        most = max(1, min(256, 24000 // new, 300000 // (new + cached)))
        return _append(_log(rng, 1, most), new, cached, Hkv, d, rng.choice(["f16", "bf16", "f32"]), rng.choice(["f16", "bf16", "f32"]), held,
                       ps, block, pool, ragged)
    longest = _log(rng, 1, 32768)
    if op == "read":
        last = rng.choice([0, 0, _log(rng, 1, 2000)])
        most = 300000 // longest
        return _read(_log(rng, 1, max(1, min(256, most))), longest, Hkv, d, rng.choice(["f16", "bf16", "f32"]), held, ps, block, last, pool, ragged)
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    sinks = rng.choice([0, 1, 4, 37]) if window else 0
    if op == "attend":
        most = 64 * 16384 * 8 * 128 // (longest * Hkv * d)
        return _attend(_log(rng, 1, max(1, min(256, most))), longest, Hq, Hkv, d, dtype, held, ps, block, window, sinks, pool, ragged)
    longest = _log(rng, 1, 9001)
    most = 4 * 6000 * 6000 * 32 // (longest * longest * Hq)
    while most < 1:  # as dear as the largest listed case at most
        longest = max(1, longest // 2)
        most = 4 * 6000 * 6000 * 32 // (longest * longest * Hq)
    return _prompt(_log(rng, 1, min(32, most)), longest, Hq, Hkv, d, dtype, window, sinks, ragged)


def _spread(n, longest, ragged, least=1):
    """n lengths up to `longest`, at least one of them that long; all of them where ragged is 0."""
    if not ragged:
        return [longest] * n
    r = random.Random(ragged * 7919 + n)
    got = [r.randint(min(least, longest), longest) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _lengths(c):
    """New tokens, and tokens in all, of each request."""
    if c["op"] == "append":
        new = _spread(c["B"], c["new"], c["ragged"])
        return new, [a + b for a, b in zip(new, _spread(c["B"], c["cached"], c["ragged"] and c["ragged"] + 1, 0))]
    lens = _spread(c["B"], c["longest"], c["ragged"])
    return lens if c["op"] == "prompt" else [1] * c["B"], lens


def _visible(position, window, sinks):
    """Keys that a query at `position` sees."""
    n = position + 1
    return n if not window or n <= window else window + min(sinks, n - window)


def work(c):
    new, lens = _lengths(c)
    Hkv, d = c["Hkv"], c["d"]
    if c["op"] == "append":
        blocks = sum(-(-l // c["block"]) - (l - n) // c["block"] for n, l in zip(new, lens))
        T = sum(new)
        return {"bytes": T * (Hkv * d * (SIZES[c["k_dtype"]] + SIZES[c["v_dtype"]] + 2) + 4) + blocks * Hkv * 8, "flops": T * Hkv * d * 4}
    if c["op"] == "read":
        n = sum(min(l, c["last"] or l) for l in lens)
        return {"bytes": n * Hkv * d * 2 * (1 + SIZES[c["dtype"]]) + n // c["block"] * Hkv * 8, "flops": n * Hkv * d * 2}
    W, S = c["window"], c["sinks"]
    if c["op"] == "attend":
        seen = sum(_visible(l - 1, W, S) for l in lens)
        rows = c["B"] * c["Hq"]
        return {"bytes": seen * Hkv * d * 2 + rows * (d * 4 + 4) + seen // c["block"] * Hkv * 8 + 4 * (seen // c["ps"] + 2 * c["B"]),
                "flops": 4 * seen * c["Hq"] * d}
    pairs = sum(sum(_visible(p, W, S) for p in range(n)) if W else n * (n + 1) // 2 for n in new)
    T = sum(new)
    return {"bytes": T * d * (4 * c["Hq"] + 4 * Hkv) + T * c["Hq"] * 4, "flops": 4 * pairs * c["Hq"] * d}


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _two_to(e):
    """2^e in 32 bits, e whole and at least -126."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _codes(g, shape, held):
    """Codes of normal values; those of a pool that has been in use for a while."""
    x = torch.randn(shape, generator=g, dtype=torch.float16, device=DEV)
    return (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn) if held == "e4m3" else (x * 30).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, pages, c):
    """Powers of two that give values of about one, some blocks smaller and some larger."""
    step = -7 if c["held"] == "e4m3" else -5
    e = torch.randint(step - 1, step + 2, (pages, c["Hkv"], c["ps"] // c["block"]), generator=g, device=DEV)
    return _two_to(e)


def _tables(g, lens, ps):
    """Block tables over a pool whose pages are handed out in a random order; entries past a request's last page are -1.
    Page 0 stays out of use.  Also the number of pages of the pool."""
    need = [-(-l // ps) for l in lens]
    most, total = max(1, max(need)), sum(need)
    order = (torch.randperm(total, generator=g, device=DEV) + 1).to(torch.int32)
    n = _ints(need)[:, None]
    off = torch.cumsum(n, 0) - n
    col = torch.arange(most, device=DEV)[None]
    table = torch.where(col < n, order[(off + col).clamp(max=max(0, total - 1))] if total else -1, torch.full_like(n, -1)).to(torch.int32)
    return table.contiguous(), total + 1


def _starts(new):
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    return at


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    new, lens = _lengths(c)
    B, Hkv, d, T = c["B"], c["Hkv"], c["d"], sum(new)
    if c["op"] == "prompt":
        dt, Hq = DTYPES[c["dtype"]], c["Hq"]
        s["q"] = 2 * torch.randn((T, Hq, d), generator=g, dtype=dt, device=DEV)
        s["k"] = torch.randn((T, Hkv, d), generator=g, dtype=dt, device=DEV)
        # the values as a projection leaves them: one part of its output's rows
        s["v"] = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, dtype=dt, device=DEV)[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        s["starts"], s["most"] = _ints(_starts(new)), max(new)
        s["out"] = torch.empty((T, Hq, d), dtype=dt, device=DEV)
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=DEV)
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["plan"] = F.prompt_params(s["q"], s["k"], s["v"], s["out"], B, window=c["window"], sinks=c["sinks"])
            s["workspace"] = torch.zeros(max(1, F.prompt_attend_workspace_bytes(s["plan"])), dtype=torch.uint8, device=DEV)
        return s
    ps, held = c["ps"], c["held"]
    s["table"], pages = _tables(g, lens, ps)
    s["lens"] = _ints(lens)
    shape = (pages, Hkv, ps, d) if c["pool"] == "head" else (pages, ps, Hkv, d)
    s["k_pages"], s["v_pages"] = _codes(g, shape, held), _codes(g, shape, held)
    s["k_scales"], s["v_scales"] = _scales(g, pages, c), _scales(g, pages, c)
    if c["op"] == "append":
        row = torch.arange(T, device=DEV)
        b = torch.repeat_interleave(torch.arange(B, device=DEV), _ints(new).long())
        pos = row - _ints(_starts(new))[b] + (_ints(lens) - _ints(new))[b]
        s["slots"] = (s["table"][b, pos // ps] * ps + pos % ps).to(torch.int32)
        wide = torch.exp(0.3 * torch.randn((T, 1, 1), generator=g, device=DEV))  # tokens differ in size
        s["k"] = (torch.randn((T, Hkv, d), generator=g, device=DEV) * wide).to(DTYPES[c["k_dtype"]])
        qkv = torch.randn((T, 5 * Hkv * d), generator=g, dtype=DTYPES[c["v_dtype"]], device=DEV)
        s["v"] = qkv[:, 4 * Hkv * d:].view(T, Hkv, d)
        s["blocks"] = sum(-(-l // c["block"]) - (l - n) // c["block"] for n, l in zip(new, lens))  # that get tokens
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["plan"] = F.append8_params(s["k"], s["v"], s["k_pages"], c["pool"], s["k_scales"])
    elif c["op"] == "read":
        dt = DTYPES[c["dtype"]]
        columns = s["table"].shape[1]
        s["first"] = _ints([max(0, l - c["last"]) if c["last"] else 0 for l in lens])
        # the full vectors' pages of their own: each request's pages one after the other, those before the first token left out
        need = [-(-l // ps) - (max(0, l - c["last"]) if c["last"] else 0) // ps for l in lens]
        skip = s["first"][:, None] // ps
        col = torch.arange(columns, device=DEV)[None]
        to = _ints(_starts(need))[:-1, None] + col - skip
        s["out_table"] = torch.where((col >= skip) & (col < (s["lens"][:, None] + ps - 1) // ps), to, -1).to(torch.int32).contiguous()
        shape = (sum(need), *shape[1:])
        s["k_out"], s["v_out"] = torch.zeros(shape, dtype=dt, device=DEV), torch.zeros(shape, dtype=dt, device=DEV)
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["plan"] = F.read8_params(s["k_pages"], s["k_scales"], s["k_out"], s["table"], c["pool"])
    else:
        dt, Hq = DTYPES[c["dtype"]], c["Hq"]
        s["q"] = 2 * torch.randn((B, Hq, d), generator=g, dtype=dt, device=DEV)
        s["out"] = torch.empty((B, Hq, d), dtype=dt, device=DEV)
        s["lse"] = torch.empty((B, Hq), dtype=torch.float32, device=DEV)
        if own:
            from dictionary_sparse_kv_gb300 import fadkv as F
            s["plan"] = F.paged8_params(s["q"], s["out"], s["k_pages"], s["k_scales"], c["pool"], s["table"], window=c["window"],
                                        sinks=c["sinks"])
            s["workspace"] = torch.zeros(max(1, F.paged8_attend_workspace_bytes(s["plan"])), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend, "prompt": _plain_prompt}[op](s)
    from dictionary_sparse_kv_gb300 import fadkv as F
    pools = [s.get(k) for k in ("k_pages", "v_pages", "k_scales", "v_scales")]
    if op == "append":
        F.paged8_append(s["plan"], s["k"], s["v"], s["slots"], *pools)
        return dict(zip(("k", "v", "ks", "vs"), pools))
    if op == "read":
        F.paged8_read(s["plan"], *pools, s["table"], s["lens"], s["first"], s["out_table"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attend":
        F.paged8_attend(s["plan"], *pools, s["table"], s["lens"], s["q"], s["out"], s["lse"], s["workspace"])
    else:
        F.prompt_attend(s["plan"], s["q"], s["k"], s["v"], s["starts"], s["out"], s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _by_token(pool, layout):
    """A view [pages][tokens][Hkv][...] of a pool."""
    return pool if layout == "token" else pool.transpose(1, 2)


def _bytes(pool):
    return pool.view(torch.uint8) if pool.dtype != torch.int8 else pool


def _plain_append(s):
    c = s["case"]
    block, ps, Hkv, T = c["block"], c["ps"], c["Hkv"], s["k"].shape[0]
    slot = s["slots"].long()
    blk = slot // block
    # the blocks that get tokens, one after the other, and each row's among them
    lead = torch.cat([torch.ones_like(blk[:1], dtype=torch.bool), blk[1:] != blk[:-1]])
    nth = torch.cumsum(lead, 0) - 1
    mine = torch.zeros(s["blocks"], dtype=torch.long, device=DEV).scatter(0, nth, blk)
    first = torch.full((s["blocks"],), block, device=DEV).scatter_reduce(0, nth, slot % block, "amin")
    page, part = mine // (ps // block), mine % (ps // block)
    at = part[:, None] * block + torch.arange(block, device=DEV)[None]  # its tokens' places in the page
    held = HELD[c["held"]]
    for x, pool, scales in ((s["k"], s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
        x = x.float()
        top = torch.zeros((s["blocks"], Hkv), device=DEV).scatter_reduce(0, nth[:, None].expand(T, Hkv), x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)
        if c["held"] == "e4m3":
            e = torch.where(m > 0.875, e - 8, e - 9)
        else:
            e = torch.where(m > 0.9921875, e - 6, e - 7)
        fresh = _two_to(torch.where(top > 0, e, -126).clamp(min=-126))
        old = scales[page, :, part]
        scale = torch.where(first[:, None] == 0, fresh, torch.maximum(fresh, old))
        tokens = _bytes(_by_token(pool, c["pool"]))
        was = tokens[page[:, None], at]  # [blocks][block][Hkv][d]
        known = was.view(held).float() * (old / scale)[:, None, :, None]
        keep = torch.arange(block, device=DEV)[None] < first[:, None]
        tokens[page[:, None], at] = torch.where(keep[..., None, None], _bytes(_round(known, held)), was)
        tokens[slot // ps, slot % ps] = _bytes(_round(x / scale[nth][..., None], held))
        scales[page, :, part] = scale
    return {"k": s["k_pages"], "v": s["v_pages"], "ks": s["k_scales"], "vs": s["v_scales"]}


def _round(x, held):
    return x.to(held) if held != torch.int8 else x.round().clamp(-127, 127).to(held)


def _values(pool, scales, table, c, dtype=torch.float32):
    """[B][pages * ps][Hkv][d] of a pool through block tables."""
    page = table.clamp(min=0).long()
    x = _by_token(_bytes(pool), c["pool"])[page].view(HELD[c["held"]]).to(dtype)  # [B][pages][ps][Hkv][d]
    f = scales[page].to(dtype).transpose(2, 3).repeat_interleave(c["block"], 2)  # [B][pages][ps][Hkv]
    x = x * f[..., None]
    return x.reshape(x.shape[0], -1, *x.shape[3:])


def _plain_read(s):
    c = s["case"]
    ps, columns = c["ps"], s["table"].shape[1]
    at = torch.arange(columns * ps, device=DEV)[None]
    if c["last"]:  # only the last tokens
        at = (s["lens"].long()[:, None] - c["last"]).clamp(min=0) + torch.arange(c["last"], device=DEV)[None]
    live = at < s["lens"].long()[:, None]
    at = at.clamp(max=columns * ps - 1).expand(c["B"], -1)
    page = torch.gather(s["table"].long(), 1, at // ps).clamp(min=0)
    to = torch.gather(s["out_table"].long(), 1, at // ps)
    for pool, scales, out in ((s["k_pages"], s["k_scales"], s["k_out"]), (s["v_pages"], s["v_scales"], s["v_out"])):
        x = _by_token(_bytes(pool), c["pool"])[page, at % ps].view(HELD[c["held"]]).float()  # [B][n][Hkv][d]
        x = x * scales.transpose(1, 2)[page, at % ps // c["block"]][..., None]
        rows = _by_token(out, c["pool"])
        # rows past a request's end go nowhere: to the place of its first token, with that one's value
        first = torch.where(live, at, at[:, :1])
        target = torch.where(live, to, to[:, :1])
        rows[target, first % ps] = torch.where(live[..., None, None], x, x[:, :1]).to(out.dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _softmax_out(sc, mask, v):
    """out and log-sum-exp of masked scores [..., rows, keys] and values [..., keys, d], in 32 bits."""
    sc = sc.masked_fill_(~mask, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0, m)
    p = sc.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(l > 0, l, 1)
    return out, (m + l.log()).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    lens = s["lens"].long()[:, None]
    ps, W, S = c["ps"], c["window"], c["sinks"]
    if W:  # only the first tokens and the window
        j = torch.arange(S + W, device=DEV)[None]
        at = torch.where(j < S, j, lens - W + j - S)
        mask = (at >= 0) & (at < lens) & ((j < S) | (at >= S))
        at = at.clamp(min=0)
        page = torch.gather(s["table"].long(), 1, (at // ps).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
        k, v = (_by_token(_bytes(p), c["pool"])[page, at % ps].view(HELD[c["held"]]).float() *
                f.transpose(1, 2)[page, at % ps // c["block"]][..., None]
                for p, f in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
    else:
        k, v = (_values(p, f, s["table"], c) for p, f in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
        mask = torch.arange(k.shape[1], device=DEV)[None] < lens
    k, v = (x.transpose(1, 2) for x in (k, v))  # [B][Hkv][keys][d]
    q = s["q"].view(B, Hkv, Hq // Hkv, d).float()
    out, lse = _softmax_out(torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5, mask[:, None, None], v)
    return {"out": out.reshape(B, Hq, d).to(s["q"].dtype), "lse": lse.reshape(B, Hq)}


def _plain_prompt(s):
    c = s["case"]
    B, Hq, Hkv, d, W, S = c["B"], c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    N, T = s["most"], s["q"].shape[0]
    starts = s["starts"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(N, device=DEV)
    row = (starts[:-1, None] + i[None]).clamp(max=T - 1)  # [B][N]
    mask = i[None] <= i[:, None]
    if W:
        mask = mask & ((i[None] > i[:, None] - W) | (i[None] < S))
    mask = mask[None] & (i[None] < n[:, None])[:, :, None]
    q = s["q"][row].view(B, N, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).float() * d ** -0.5
    k, v = (s[x][row].transpose(1, 2).float()[:, :, None] for x in ("k", "v"))
    out, lse = _softmax_out(torch.matmul(q, k.transpose(-1, -2)), mask[:, None, None], v)
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
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "read":
        return _exact_read(c, s)
    return _exact_attention(c, s)


def _power(e):
    """2^e in 64 bits, e whole."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _nearest(x, held):
    """The code nearest to x, ties to even, as a number."""
    if held == "i8":
        return torch.round(x).clamp(-127, 127)
    size = x.abs()
    step = _power(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(size / step) * step).clamp(max=448) * torch.sign(x)


def _exact_append(c, s):
    ps, block, held = c["ps"], c["block"], c["held"]
    new, lens = _lengths(c)
    table = s["table"].tolist()
    got = {}
    for name, x, pool, scales in (("k", s["k"], s["k_pages"], s["k_scales"]), ("v", s["v"], s["v_pages"], s["v_scales"])):
        codes, sizes = pool.to(torch.float32).double(), scales.double()
        x = x.double()
        row = 0
        for n, l, pages in zip(new, lens, table):
            at = l - n
            while at < l:  # a block at a time
                end = min(l, at // block * block + block)
                page, lo, hi, o = pages[at // ps], at // block * block % ps, at % ps, at % ps // block
                y = x[row:row + end - at].transpose(0, 1)  # [Hkv][tokens][d]
                top = y.abs().amax((1, 2)).clamp(min=2.0 ** -126)
                scale = _power(torch.ceil(torch.log2(top / LARGEST[held])))
                # (the logarithm may be off by a rounding: the least power of two that reaches)
                scale = torch.where(scale / 2 * LARGEST[held] >= top, scale / 2, scale)
                scale = torch.where(scale * LARGEST[held] < top, scale * 2, scale).clamp(min=2.0 ** -126)
                target = codes[page] if c["pool"] == "head" else codes[page].transpose(0, 1)
                if at % block:
                    scale = torch.maximum(scale, sizes[page, :, o])
                    before = target[:, lo:hi]
                    target[:, lo:hi] = _nearest(before * (sizes[page, :, o] / scale)[:, None, None], held)
                target[:, hi:hi + end - at] = _nearest(y / scale[:, None, None], held)
                sizes[page, :, o] = scale
                row += end - at
                at = end
        got[name], got[name + "s"] = codes if held == "e4m3" else None, sizes
    return got


def _exact_read(c, s):
    ps, block = c["ps"], c["block"]
    got = {}
    for name, pool, scales, out in (("k", s["k_pages"], s["k_scales"], s["k_out"]), ("v", s["v_pages"], s["v_scales"], s["v_out"])):
        y = torch.zeros(out.shape, dtype=torch.float64, device=DEV)
        for b, l in enumerate(s["lens"].tolist()):
            first = int(s["first"][b])
            j = torch.arange(first, l, device=DEV)
            page, to, o = s["table"][b].long()[j // ps], s["out_table"][b].long()[j // ps], j % ps
            f = scales.double()[page, :, o // block][..., None]
            if c["pool"] == "head":
                y[to, :, o] = _bytes(pool)[page, :, o].view(pool.dtype).to(torch.float32).double() * f
            else:
                y[to, o] = _bytes(pool)[page, o].view(pool.dtype).to(torch.float32).double() * f
        got[name] = y
    return got


def _exact_attention(c, s):
    Hq, Hkv, d, W, S = c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    group = Hq // Hkv
    if work(c)["flops"] > 1e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    new, lens = _lengths(c)
    starts = _starts(new)
    for b, (n, length) in enumerate(zip(new, lens)):
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
            if c["op"] == "prompt":
                kv = [s[x][starts[b]:starts[b + 1]][keys].double() for x in ("k", "v")]
            else:
                pg, o = s["table"][b].long()[keys // c["ps"]], keys % c["ps"]
                kv = []
                for pool, scales in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])):
                    x = _bytes(pool)[pg, :, o] if c["pool"] == "head" else _bytes(pool)[pg, o]
                    kv.append(x.contiguous().view(pool.dtype).to(torch.float32).double() * scales.double()[pg, :, o // c["block"]][..., None])
            rows = slice(starts[b] + lo, starts[b] + hi)
            for h in range(Hkv):
                heads = slice(h * group, (h + 1) * group)
                x = torch.einsum("thd,kd->htk", s["q"][rows, heads].double(), kv[0][:, h]) / math.sqrt(d)
                x = torch.where(seen, x, -math.inf)
                z = torch.logsumexp(x, -1)
                out[rows, heads] = torch.einsum("htk,kd->thd", torch.exp(x - z[..., None]), kv[1][:, h])
                lse[rows, heads] = z.T
    return {"out": out, "lse": lse}
