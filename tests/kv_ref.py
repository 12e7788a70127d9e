"""Plain references of the paged-cache operators, in 64 bits on the host, and
the small batches the tests run them on."""
import math

import numpy as np
import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half an ulp, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -130}  # half the spacing of the smallest numbers


def up(a, b):
    return -(-a // b)


class Batch:
    """Sequences with new[i] new tokens and len[i] in all, their pages in random order in a pool with spare
    pages; slots that no token owns hold `junk`."""

    def __init__(self, new, length, page, n_kv, d, dtype, seed=0, spare=3, layout="hsd", junk=0.0, extra_tokens=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.len, self.page, self.n_kv, self.d, self.dtype = list(new), list(length), page, n_kv, d, dtype
        held = [up(v, page) for v in self.len]
        self.n_pages, width = sum(held) + spare, max(held + [1]) + 2
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(new), width), -1, dtype=torch.int32)
        at = 0
        for i, h in enumerate(held):
            self.table[i, :h] = order[at:at + h]
            at += h
        starts = np.concatenate([[0], np.cumsum(self.new)])
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.kv_len = torch.tensor(self.len, dtype=torch.int32)
        self.t = int(starts[-1]) + extra_tokens
        kv = torch.randn(2, self.n_pages, n_kv, page, d, generator=g)
        kv[0, ..., :: d // 4] *= 3
        owned = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for i, v in enumerate(self.len):
            for j in range(v):
                owned[self.table[i, j // page], j % page] = True
        kv[:, ~owned[:, None, :].expand(-1, n_kv, -1)] = junk
        self.kv = kv.to(dtype)
        self.layout = layout
        self.g = g

    def to_gpu(self, L):
        kv = self.kv.cuda()
        if self.layout == "shd":  # pages of [page_size][n_kv][head_dim]
            kv = kv.transpose(2, 3).contiguous().transpose(2, 3)
        elif self.layout == "joint":  # keys and values of a page side by side, padded heads
            wide = torch.zeros(self.n_pages, 2, self.n_kv, self.page, self.d + 8, dtype=self.dtype, device="cuda")
            wide[..., :self.d] = kv.transpose(0, 1)
            kv = wide[..., :self.d].transpose(0, 1)
        self.gkv = kv
        self.gtable, self.gq, self.glen = self.table.cuda(), self.q_start.cuda(), self.kv_len.cuda()
        self.cache = L.tq1_kv_cache(kv[0], kv[1])
        self.batch = L.tq1_kv_batch(self.gtable, self.gq, self.glen)
        return self

    def sequence(self, i, which):
        """fp64 [len][n_kv][d] keys (0) or values (1) of sequence i."""
        pages = self.table[i, :up(self.len[i], self.page)].long()
        return self.kv[which][pages].double().transpose(1, 2).reshape(-1, self.n_kv, self.d)[:self.len[i]]


def attention(b, q, scale, causal, window):
    """(out, tol) fp64 [t][n_q][d].  tol bounds what fp32 accumulation and 16-bit weights may change, from the
    magnitudes of the terms (before the rounding of the output):
      scores     d products and sums of fp32: |dx| <= d 2^-24 scale sum |q k|, and 2^-22 |x| for their scaling
      weights    exp to 2^-21 relative, rounded to 16 bits (u, at least `tiny` when they underflow)
      sums       n terms of fp32"""
    t, n_q, d = q.shape
    group, u, tiny = n_q // b.n_kv, UNIT[b.dtype], TINY[b.dtype]
    where = "cuda" if torch.cuda.is_available() else "cpu"  # fp64 either way
    out, tol = (torch.zeros(t, n_q, d, dtype=torch.float64, device=where) for _ in range(2))
    q = q.to(where)
    at = 0
    for i, (n, ln) in enumerate(zip(b.new, b.len)):
        if n and ln:
            k, v = b.sequence(i, 0).to(where), b.sequence(i, 1).to(where)
            pos = torch.arange(ln - n, ln, device=where)[:, None]
            j = torch.arange(ln, device=where)[None, :]
            seen = torch.ones(n, ln, dtype=torch.bool, device=where)
            if causal:
                seen &= j <= pos
            if window:
                seen &= j > pos - window
            for h in range(n_q):
                x = (q[at:at + n, h].double() @ k[:, h // group].T) * scale
                ax = (q[at:at + n, h].double().abs() @ k[:, h // group].abs().T) * scale
                x = x.masked_fill(~seen, -math.inf)
                dx = (d * 2.0 ** -24 * ax + 2.0 ** -22 * ax).masked_fill(~seen, 0).amax(1, keepdim=True)
                m = x.amax(1, keepdim=True)
                e = torch.exp(x - torch.where(m.isinf(), torch.zeros_like(m), m))
                l = e.sum(1, keepdim=True)
                l = torch.where(l == 0, torch.ones_like(l), l)
                o = e @ v[:, h // group] / l
                a = e @ v[:, h // group].abs() / l
                out[at:at + n, h] = o
                tol[at:at + n, h] = ((u + 4 * dx + 2.0 ** -20 + 2 * ln * 2.0 ** -24) * a
                                     + ln * tiny * v[:, h // group].abs().amax() / l)
        at += n
    return out.cpu(), tol.cpu()


def rounded(tol, ref, dtype):
    """tol plus the rounding of the result itself to dtype."""
    if dtype == torch.float32:
        return tol + 2.0 ** -23 * ref.abs()
    return tol * (1 + 2.0 ** -7) + UNIT[dtype] * ref.abs() + TINY[dtype]


def rotate(x, angle, mscale, rot, interleaved):
    """(y, size): fp64 x [..., d] turned by angle [..., rot/2], and the magnitude of the terms of each result."""
    y, size = x.clone(), x.abs()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    c, s = angle.cos() * mscale, angle.sin() * mscale
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    both = (x[..., a].abs() + x[..., b].abs()) * abs(mscale)
    size[..., a], size[..., b] = both, both
    return y, size


class Pages:
    """The page bookkeeping as plain Python: tables, counts, lengths and which page copies which."""

    def __init__(self, table, kv_len, refs, pools, page):
        self.table, self.len, self.refs = table.tolist(), kv_len.tolist(), refs.tolist()
        self.pools, self.page = pools.clone(), page
        self.lacking = False

    def _up(self, v):
        return up(v, self.page)

    def _deal(self, wants):
        """Page ids for each want, lowest free first; None from the first that does not fit on."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        got, at = [], 0
        for w in wants:
            got.append(free[at:at + w] if at + w <= len(free) else None)
            if got[-1] is None:
                self.lacking = True
            at += w
        return got

    def _copy(self, pairs):
        old = self.pools.clone()
        for a, b in pairs:
            self.pools[:, b] = old[:, a]

    def resize(self, seqs, lens):
        for s, n in zip(seqs, lens):
            if 0 <= n <= self.len[s]:
                for j in range(self._up(n), self._up(self.len[s])):
                    self.refs[self.table[s][j]] -= 1
                    self.table[s][j] = -1
                self.len[s] = n
        grow = []
        for s, n in zip(seqs, lens):
            if n < 0 or self._up(n) > len(self.table[s]):
                self.lacking = True
            elif n > self.len[s]:
                had = self._up(self.len[s])
                own = self.len[s] % self.page != 0 and self.refs[self.table[s][had - 1]] > 1
                grow.append((s, n, had - own, own))
        got = self._deal([self._up(n) - first for _, n, first, _ in grow])
        pairs, left = [], []
        for (s, n, first, own), ids in zip(grow, got):
            if ids is None:
                continue
            if own:
                pairs.append((self.table[s][first], ids[0]))
                left.append(self.table[s][first])
            for k, p in enumerate(ids):
                self.table[s][first + k] = p
                self.refs[p] = 1
            self.len[s] = n
        for p in left:
            self.refs[p] -= 1
        self._copy(pairs)

    def fork(self, parents, children):
        wants = [1 if self.len[a] % self.page else 0 for a in parents]
        pairs = []
        for a, c, ids in zip(parents, children, self._deal(wants)):
            if ids is None:
                continue
            full = self.len[a] // self.page
            for j in range(full):
                self.table[c][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            if ids:
                pairs.append((self.table[a][full], ids[0]))
                self.table[c][full] = ids[0]
                self.refs[ids[0]] = 1
            self.len[c] = self.len[a]
        self._copy(pairs)

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in live if p >= n]
        to = dict(zip(movers, holes))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self._copy(list(to.items()))
