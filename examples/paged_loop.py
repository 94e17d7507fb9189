"""One attention layer of a serving loop: full vectors in pages, codes beside them.

Prompts of several requests are planned into pages, their queries and keys
normalised, rotated and appended, and attended in one call; then decode steps
follow, one token a request.  Every step's keys and values are also encoded
into the layer's dictionaries and stored as packed codes, so the same query is
answered three ways: over all full vectors, over a recent window and the first
tokens of them, and over the codes.

    python examples/paged_loop.py [--steps 16] [--prompt 48]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dictionary_sparse_kv_gb300 import build as B
from dictionary_sparse_kv_gb300 import fadkv as F
from dictionary_sparse_kv_gb300 import synthetic as S

HQ, HKV, D, PAGE, N_ATOMS, POOL, TERMS = 24, 8, 128, 16, 4096, 256, 8


class Layer:
    """Pools, tables and codes of one layer for R requests of up to `longest` tokens."""

    def __init__(self, R, longest, dev="cuda", seed=0):
        i32 = dict(dtype=torch.int32, device=dev)
        self.R, self.dev, self.longest = R, dev, longest
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        columns = -(-longest // PAGE)
        pages = R * columns
        self.k_pages, self.v_pages = (torch.zeros((pages, HKV, PAGE, D), dtype=torch.float16, device=dev) for _ in range(2))
        self.table = torch.full((R, columns), -1, **i32)
        self.free, self.free_count = torch.arange(pages, **i32), torch.tensor([pages], **i32)
        self.lengths, self.starts, self.refused = torch.zeros(R, **i32), torch.zeros(R + 1, **i32), torch.zeros(1, **i32)
        self.rope = F.rope_init(D, D, base=500000.0, scaling="parts", factor=32.0, original=8192.0, slow=1.0, fast=4.0)
        self.wq, self.wk = (1 + 0.1 * torch.randn((2, D), generator=self.gen, device=dev)).half()
        self.workspaces = {}
        # codes: a key and a value dictionary, random unit-norm atoms, all in use
        atoms = torch.stack([torch.from_numpy(S.make_dictionary(N_ATOMS, D, "float16", seed, i)) for i in range(2)])
        self.dict = F.Dictionary(atoms.to(dev), torch.ones((2, N_ATOMS), **i32), [0.50, 0.70], POOL, TERMS, R * HKV)
        self.cache = torch.zeros((2, R, HKV, longest, TERMS + 1), **i32)

    def workspace(self, kind, nbytes):
        """One zero-filled workspace per kind of call, kept (and grown) over the steps."""
        w = self.workspaces.get(kind)
        if w is None or w.numel() < nbytes:
            w = self.workspaces[kind] = torch.zeros(nbytes, dtype=torch.uint8, device=self.dev)
        return w

    def project(self, T):
        """Stands in for the layer's projections of T tokens: queries, keys and values side by side."""
        qkv = torch.randn((T, (HQ + 2 * HKV) * D), generator=self.gen, device=self.dev).half()
        return [x.view(T, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1)]

    def append(self, add):
        """Plans `add` new tokens a request and puts their keys and values into the pages; queries, keys, values."""
        T = int(add.clamp(min=0).sum())
        plan = F.page_params(self.R, PAGE, self.k_pages.shape[0], self.table.shape[1], T)
        self.positions, self.slots = (torch.empty(T, dtype=torch.int32, device=self.dev) for _ in range(2))
        F.page_plan(plan, add, self.lengths, self.table, self.free, self.free_count, self.lengths, self.free_count, self.starts,
                    self.positions, self.slots, self.refused)
        q, k, v = self.project(T)
        q_out, k_out = torch.empty((T, HQ, D), dtype=torch.float16, device=self.dev), torch.empty((T, HKV, D), dtype=torch.float16, device=self.dev)
        F.qk_norm_rope(F.qk_params(q, k, v, q_out, self.k_pages, k_out=k_out, v_pages=self.v_pages, wq=self.wq, wk=self.wk), self.rope, q, k, v, self.wq, self.wk, self.positions, self.slots,
                       q_out, k_out, self.k_pages, self.v_pages)
        return q_out, k_out, v

    def code(self, k, v, pos):
        """Encodes one token a request (k, v [R][HKV][D]), adapts the dictionaries and stores the packed codes."""
        x = torch.stack([k.reshape(-1, D), v.reshape(-1, D)]).contiguous()
        c = self.dict.new_codes(x.shape[1])
        self.dict.step(x, c)
        F.store_codes(2, self.R, HKV, TERMS, N_ATOMS, c.idx, c.coef, c.repl_id, c.repl_coef, pos, self.cache, self.longest)

    def attend(self, q, window=0, sinks=0, positions=None):
        """One query token a request over the pages; with the step's positions, requests that its plan refused see nothing."""
        out = torch.empty_like(q)
        p = F.paged_params(q, out, self.k_pages, "head", self.table, window, sinks, v_pages=self.v_pages)
        ws = self.workspace("decode", F.paged_attend_workspace_bytes(p))
        F.paged_attend(p, self.k_pages, self.v_pages, self.table, self.lengths, q, out, None, ws, positions=positions)
        return out

    def prefill(self, q, window=0, sinks=0):
        """The new tokens' queries (rows starts[b] .. starts[b + 1]) over the pages."""
        out = torch.empty_like(q)
        p = F.paged_params(q, out, self.k_pages, "head", self.table, window, sinks, v_pages=self.v_pages)
        ws = self.workspace("prefill", F.paged_prefill_workspace_bytes(p))
        F.paged_prefill(p, self.k_pages, self.v_pages, self.table, self.lengths, self.starts, q, out, None, ws,
                        positions=self.positions)
        return out

    def attend_codes(self, q):
        """The same queries over the codes."""
        q32 = q.float().contiguous()[None]
        out = torch.empty_like(q32)
        p = F.AttnParams(1, self.R, HQ, HKV, D, N_ATOMS, TERMS, self.longest, F.F16, D ** -0.5, 2 * N_ATOMS * D, self.cache.numel())
        F.attend(p, self.dict.atoms[0], self.dict.atoms[1], self.cache[0], self.cache[1], self.lengths, q32, out)
        return out[0]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=48)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--window", type=int, default=32)
    ap.add_argument("--sinks", type=int, default=4)
    a = ap.parse_args(argv)
    B.build()
    layer = Layer(a.requests, a.prompt + a.steps)
    i32 = dict(dtype=torch.int32, device=layer.dev)

    # the prompts: all of them in one call, a request's tokens together
    q, k, v = layer.append(torch.full((a.requests,), a.prompt, **i32))
    out = layer.prefill(q)
    by_token = lambda x: x.view(a.requests, a.prompt, -1, D).transpose(0, 1)
    for t in range(a.prompt):
        layer.code(by_token(k)[t], by_token(v)[t], torch.full((a.requests,), t, **i32))
    last = out.view(a.requests, a.prompt, HQ, D)[:, -1]
    same = (layer.attend(q.view(a.requests, a.prompt, HQ, D)[:, -1].contiguous()) - last).abs().max().item()

    diff = {}
    one = torch.ones(a.requests, **i32)
    for _ in range(a.steps):
        q, k, v = layer.append(one)
        layer.code(k, v, layer.lengths - 1)
        full = layer.attend(q, positions=layer.positions).float()
        recent = layer.attend(q, a.window, a.sinks, layer.positions).float()
        for name, other in (("window", recent), ("codes", layer.attend_codes(q))):
            diff.setdefault(name, []).append(((other - full).norm() / full.norm()).item())
    torch.cuda.synchronize()
    result = {"tokens": layer.lengths.tolist(), "refused": int(layer.refused), "pages left": int(layer.free_count),
              "prefill and decode differ by": same, **{n + " against full": sum(d) / len(d) for n, d in diff.items()}}
    for n, x in result.items():
        print(f"{n}: {x}")
    return result


if __name__ == "__main__":
    main()
