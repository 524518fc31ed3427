"""One transformer layer served token by token: coded weights, a 4-bit key/value cache, attention over it.

    python examples/cached_decode.py [--prompt 100] [--steps 8] [--batch 2] [--pages 4]

The projections and the SwiGLU MLP are entropy-coded 4-bit matrices (lw_gemv); queries and keys are turned by their
positions (lw_rope), keys and values quantised into a paged cache as they are made (lw_kv_append) and attended over
(lw_kv_attend), first the prompt in pieces of at most 16 tokens, then one new token a step.  With --pages a step attends
over that many pages of each sequence, chosen for each kv head by the bounds of their keys (lw_kv_bounds, lw_kv_select,
lw_kv_attend_selected).  A step is a fixed sequence of launches over buffers that stay in place, so it is
captured once and replayed; between steps the program moves the lengths on.  At the end the cache is read back
(lw_kv_read) and the last step is compared with attention in fp64 over what it holds.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import decode_gemv_amd as dg

HIDDEN, HEADS, KV, DIM, MLP, PAGE = 1024, 16, 4, 64, 2816, 32


def coded(rng, rows, cols):
    """A random coded matrix of 4-bit codes whose product keeps the size of its input."""
    codes = np.clip(np.rint(rng.normal(7.5, 1.8, (rows, cols))), 0, 15).astype(np.uint8)
    d = np.full((rows, cols // 256), np.float16(cols ** -0.5 / 1.8), np.float16).view(np.uint16)
    m = (d.view(np.float16) * np.float16(7.5)).view(np.uint16)
    return dg.upload(dg.lw_bundle_build_q(dg.LW_Q4_PAIR, codes, d, m))


class Layer:
    def __init__(self, batch, longest, chosen=0, seed=1):
        rng = np.random.default_rng(seed)
        self.qkv = coded(rng, (HEADS + 2 * KV) * DIM, HIDDEN)
        self.o = coded(rng, HIDDEN, HEADS * DIM)
        self.gate, self.up, self.down = coded(rng, MLP, HIDDEN), coded(rng, MLP, HIDDEN), coded(rng, HIDDEN, MLP)
        self.n_seqs, per = batch, -(-longest // PAGE)
        size = dg.lw_kv_page_bytes(KV, DIM, PAGE)
        pages = torch.empty(batch * per * size, dtype=torch.uint8, device="cuda")
        self.cache = dg.KvCache(pages, KV, DIM, PAGE)
        order = torch.from_numpy(rng.permutation(batch * per).astype(np.int32)).cuda()
        self.table = order.view(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.longest = longest
        self.rope = dg.lw_rope_make(DIM // 2)
        self.chosen = chosen                                 # pages that a new token attends over (0: all)
        self.bounds = torch.empty(batch * per * dg.lw_kv_bounds_bytes(KV, DIM), dtype=torch.uint8, device="cuda")

    def batch(self, new):
        """Every sequence has `new` tokens, packed one sequence after the other."""
        start = torch.arange(0, (self.n_seqs + 1) * new, new, dtype=torch.int32, device="cuda")
        return dg.KvBatch(start, self.lens, self.table, max_len=self.longest)

    def attend(self, q, out, kv, keep, get, chosen):
        n = q.shape[0]
        if not chosen:
            need = dg.lw_kv_attend_scratch_bytes(self.cache, kv, n, HEADS)
            dg.lw_kv_attend(self.cache, kv, q, out, work=get("work", need, dtype=torch.uint8) if need else None)
            return
        whole = dict(dtype=torch.int32)
        sel = keep["chosen"] = dg.KvSelection(get("sel start", n + 1, **whole), get("sel lens", n, **whole),
                                              get("sel table", n, KV, self.chosen, **whole))
        need = dg.lw_kv_select_scratch_bytes(self.cache, kv, n, HEADS)
        dg.lw_kv_select(self.cache, kv, q, self.bounds, sel, first=min(1, self.chosen - 1), last=0,
                        work=get("sel work", need, dtype=torch.uint8) if need else None)
        need = dg.lw_kv_attend_selected_scratch_bytes(self.cache, sel, HEADS)
        dg.lw_kv_attend_selected(self.cache, sel, q, out, work=get("work", need, dtype=torch.uint8) if need else None)

    def forward(self, x, kv, keep, step=False):
        """x [n][HIDDEN] fp16; lens already count these tokens.  keep: the buffers.  step: new tokens, which attend over the
        chosen pages; a piece of the prompt, also of one token a sequence, does over all."""
        n, chosen = x.shape[0], step and self.chosen > 0
        get = lambda name, *shape, dtype=torch.float32: keep.setdefault(
            (name, n, chosen), torch.empty(shape, dtype=dtype, device="cuda"))
        y = get("qkv", n, (HEADS + 2 * KV) * DIM)
        dg.lw_gemv(self.qkv, x, y, n)
        y = y.view(n, HEADS + 2 * KV, DIM)
        q, k, v = get("q", n, HEADS, DIM, dtype=torch.float16), y[:, HEADS:HEADS + KV], y[:, HEADS + KV:]
        dg.lw_rope(self.rope, y[:, :HEADS], q, batch=kv)
        dg.lw_rope(self.rope, k, k, batch=kv)
        dg.lw_kv_append(self.cache, kv, k, v)
        if self.chosen:
            dg.lw_kv_bounds(self.cache, kv, n, self.bounds)
        a = get("attended", n, HEADS, DIM, dtype=torch.float16)
        self.attend(q, a, kv, keep, get, chosen)
        keep["q"], keep["a"] = q, a
        z = get("o", n, HIDDEN)
        dg.lw_gemv(self.o, a, z, n)
        h = (x.float() + z).half()
        g, u, m, out = get("g", n, MLP), get("u", n, MLP), get("m", n, MLP, dtype=torch.float16), get("out", n, HIDDEN)
        dg.lw_gemv(self.gate, h, g, n)
        dg.lw_gemv(self.up, h, u, n)
        dg.lw_swiglu(g, u, m)
        dg.lw_gemv(self.down, m, out, n)
        r = h.float() + out
        return (r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6)).half()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--pages", type=int, default=0, help="pages that a new token attends over (0: all)")
    a = ap.parse_args(argv)
    if not 1 <= a.batch <= 16 or a.prompt < 1 or a.steps < 1 or not 0 <= a.pages <= 32768:
        ap.error("--batch must be in 1..16, --prompt and --steps at least 1, --pages in 0..32768")
    torch.manual_seed(0)
    layer, keep = Layer(a.batch, a.prompt + a.steps, a.pages), {}
    prompt = torch.randn((a.batch, a.prompt, HIDDEN), device="cuda").half()
    done, piece = 0, 16 // a.batch                          # lw_gemv takes up to 16 rows
    while done < a.prompt:
        n = min(piece, a.prompt - done)
        layer.lens.add_(n)
        y = layer.forward(prompt[:, done:done + n].reshape(-1, HIDDEN).contiguous(), layer.batch(n), keep)
        done += n
    x = y.view(a.batch, n, HIDDEN)[:, -1].contiguous()
    one, y = layer.batch(1), torch.empty_like(x)

    def step():
        y.copy_(layer.forward(x, one, keep, step=True))

    layer.lens.add_(1)
    step()                                                   # (its buffers, and the kernels' first use)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(a.steps):
        if i:
            x.copy_(y)
            layer.lens.add_(1)
        graph.replay()
    torch.cuda.synchronize()

    # the last step against fp64 attention over the cache as it reads back (the chosen pages of it)
    total = a.prompt + a.steps
    k, v = (torch.empty((a.batch * total, KV, DIM), device="cuda") for _ in range(2))
    dg.lw_kv_read(layer.cache, layer.batch(total), k, v)
    k, v = (t.view(a.batch, total, KV, DIM).double().repeat_interleave(HEADS // KV, 2) for t in (k, v))
    scores = (keep["q"].double()[:, None] * k).sum(-1) * DIM ** -0.5
    if a.pages:
        mine = layer.table.repeat_interleave(PAGE, 1)[:, :total]             # each token's page
        seen = (mine[:, :, None, None] == keep["chosen"].table[:, None]).any(-1)
        scores = scores.masked_fill(~seen.repeat_interleave(HEADS // KV, 2), -torch.inf)
    p = torch.softmax(scores, 1)
    want = (p[..., None] * v).sum(1)
    err = float((keep["a"].double() - want).norm() / want.norm())
    held = layer.cache.pages.numel()
    print(f"{a.batch} sequences, {total} tokens each: attention within {err:.1e} of fp64 over the cache; "
          f"{held} bytes hold what takes {layer.cache.n_pages * PAGE * 2 * KV * DIM * 2} in 16 bits", flush=True)
    return err


if __name__ == "__main__":
    sys.exit(0 if main() < 1e-3 else 1)
