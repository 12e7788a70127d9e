#!/usr/bin/env python3
"""Attention layers of a decoder on ternary weights, from prompt to forked continuations.

Two layers share one page table.  Each step of a layer is

    x -> q8_1_quantize_acts -> tq1_mmv_ws (q, k and v at once)
      -> tq1_rope_append (rotated q; k and v into the cache's pages)
      -> tq1_paged_attn (fp32) -> q8_1_quantize_acts -> tq1_mmv_ws (+ x)

and the cache's pages are kept by tq1_pages_resize, _fork and _compact: prompts of three requests in one ragged
batch, decode steps, a request that ends, one that is forked into two continuations, and a compaction in between.

    python examples/decoder_layer.py        # prints the largest difference from a plain fp64 computation
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_gemv_tq1_gb300 as tq  # noqa: E402
from bit_quantized_gemv_tq1_gb300 import _lib as lib  # noqa: E402

HIDDEN, N_Q, N_KV, D, PAGE, LAYERS = 2048, 16, 4, 128, 32, 2
N_SEQS, MAX_PAGES, N_PAGES = 6, 32, 96


class Decoder:
    """The layers' weights, their caches and the sequences' pages."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.weights = []
        for _ in range(LAYERS):
            layer = []
            for n, k in (((N_Q + 2 * N_KV) * D, HIDDEN), (HIDDEN, N_Q * D)):
                trits = torch.randint(-1, 2, (n, k), generator=g).float()
                w = (trits * 0.02).half().float().to(device)  # one scale: quantising loses nothing
                blocks = torch.empty(tq.tq1_blocks_bytes(n, k), dtype=torch.uint8, device=device)
                tq.tq1_quantize_rows(w, blocks, n, k)
                layer.append((blocks, w, n, k))
            self.weights.append(layer)
        self.kv = torch.zeros(LAYERS, 2, N_PAGES, N_KV, PAGE, D, dtype=torch.float16, device=device)
        self.table = torch.full((N_SEQS, MAX_PAGES), -1, dtype=torch.int32, device=device)
        self.len = torch.zeros(N_SEQS, dtype=torch.int32, device=device)
        self.refs = torch.zeros(N_PAGES, dtype=torch.int32, device=device)
        self.pool = tq.tq1_page_pool(self.kv.flatten(0, 1), self.table, self.len, self.refs, PAGE)
        self.pages_ws = torch.empty(tq.tq1_pages_workspace_size(self.pool), dtype=torch.uint8, device=device)
        self.caches = [tq.tq1_kv_cache(self.kv[i, 0], self.kv[i, 1]) for i in range(LAYERS)]
        self.inv_freq = torch.empty(D // 2, device=device)
        tq.tq1_rope_freqs(self.inv_freq, D, base=10000.0, factor=4.0, orig_len=256.0, low=1.0, high=8.0)

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.len.device)

    def resize(self, lens):
        """Sequences' lengths, {sequence: length}; 0 frees one."""
        tq.tq1_pages_resize(self.pool, self.ints(list(lens)), self.ints(list(lens.values())), self.pages_ws)

    def fork(self, parent, child):
        tq.tq1_pages_fork(self.pool, self.ints([parent]), self.ints([child]), self.pages_ws)

    def compact(self):
        tq.tq1_pages_compact(self.pool, self.pages_ws)

    def product(self, x, weight, res=None):
        blocks, _, n, k = weight
        t = x.shape[0]
        q8 = torch.empty(tq.tq1_q8_1_bytes(t, k), dtype=torch.uint8, device=x.device)
        tq.q8_1_quantize_acts(x, q8, t, k)
        y = torch.empty(t, n, device=x.device)
        need = lib.tq1_mmv_workspace_size(n, k, t)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        lib.tq1_mmv_ws(blocks, q8, y, n, k, t, ws, res=res)
        return y

    def step(self, x, new):
        """x [t][HIDDEN]: the next new[s] tokens of every sequence s, whose slots resize() has made room for."""
        t = x.shape[0]
        starts = [0]
        for s in range(N_SEQS):
            starts.append(starts[-1] + new.get(s, 0))
        batch = tq.tq1_kv_batch(self.table, self.ints(starts), self.len)
        for (w_qkv, w_out), cache in zip(self.weights, self.caches):
            qkv = self.product(x, w_qkv).unflatten(1, (-1, D))
            q = torch.empty(t, N_Q, D, dtype=torch.float16, device=x.device)
            tq.tq1_rope_append(cache, batch, qkv[:, :N_Q], qkv[:, N_Q:N_Q + N_KV], qkv[:, N_Q + N_KV:], q, self.inv_freq, D)
            out = torch.empty(t, N_Q, D, device=x.device)
            ws = torch.empty(tq.tq1_paged_attn_workspace_size(cache, t, N_Q, N_SEQS), dtype=torch.uint8, device=x.device)
            tq.tq1_paged_attn(cache, batch, q, out, 1 / math.sqrt(D), ws=ws)
            x = self.product(out.flatten(1), w_out, res=x)
        return x


def plain(dec, xs):
    """The layers over whole sequences xs [len][HIDDEN], fp64, without a cache; the activations' 8-bit rounding included."""
    def round8(x):
        d = x.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).float() / 127
        q = torch.where(d > 0, x.unflatten(-1, (-1, 32)) / d.double(), 0.0)
        q = torch.sign(q) * torch.floor(q.abs() + 0.5)
        return (q * d.half().double()).flatten(-2)

    x = xs.double()
    angle = torch.arange(x.shape[0], device=x.device).double()[:, None, None] * dec.inv_freq.double()
    for (_, w_qkv, _, _), (_, w_out, _, _) in dec.weights:
        qkv = (round8(x) @ w_qkv.double().T).unflatten(1, (-1, D))
        a, b = qkv[:, :N_Q + N_KV, :D // 2], qkv[:, :N_Q + N_KV, D // 2:]
        turned = torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1).half().double()
        q, k = turned[:, :N_Q], turned[:, N_Q:].repeat_interleave(N_Q // N_KV, 1)
        v = qkv[:, N_Q + N_KV:].half().double().repeat_interleave(N_Q // N_KV, 1)
        scores = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
        scores.masked_fill_(torch.ones_like(scores[0], dtype=torch.bool).triu(1), -math.inf)
        out = torch.einsum("hij,jhd->ihd", scores.softmax(-1), v).flatten(1)
        x = x + round8(out) @ w_out.double().T
    return x


def run(seed=0):
    """The story of the module's first lines; returns {sequence: (outputs, plain outputs)} of every token."""
    dec = Decoder(seed)
    g = torch.Generator().manual_seed(seed + 1)
    inputs, outputs = {}, {}

    def step(new):
        xs = {s: torch.randn(n, HIDDEN, generator=g) for s, n in sorted(new.items())}
        for s, x in xs.items():
            inputs[s] = torch.cat([inputs[s], x]) if s in inputs else x
        dec.resize({s: inputs[s].shape[0] for s in new})
        y = dec.step(torch.cat(list(xs.values())).cuda(), new)
        for (s, n), part in zip(sorted(new.items()), y.split([n for _, n in sorted(new.items())])):
            outputs[s] = torch.cat([outputs[s], part]) if s in outputs else part

    step({0: 200, 1: 37, 3: 1})             # prompts
    for _ in range(3):
        step({0: 1, 1: 1, 3: 1})            # decode steps
    dec.resize({0: 0})                      # the first request is done
    done = {0: (inputs.pop(0), outputs.pop(0))}
    dec.fork(1, 4)                          # the second goes on in two ways
    inputs[4], outputs[4] = inputs[1], outputs[1]
    dec.compact()
    step({1: 1, 3: 70, 4: 1, 5: 300})       # a chunk and a new prompt beside the steps
    step({1: 2, 3: 1, 4: 1, 5: 1})
    status = tq.tq1_sync_status()
    if status:
        raise tq.Tq1Error(status, "decoder_layer")
    for s in inputs:
        done[s] = (inputs[s], outputs[s])
    return {s: (y.double(), plain(dec, x.cuda())) for s, (x, y) in done.items()}


def main():
    for s, (got, want) in sorted(run().items()):
        print(f"sequence {s}: {got.shape[0]} tokens, |x| {want.norm(dim=1).mean():.2f}, "
              f"largest relative difference of a token {((got - want).norm(dim=1) / want.norm(dim=1)).max():.2e}")


if __name__ == "__main__":
    main()
