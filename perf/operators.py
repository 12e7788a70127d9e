"""The decoder-layer operators between the projections, as cases that can be timed and compared.

Three families, in the order a serving step runs them:

  rope    tq1_rope_append: rotary positions on the projections' fp32 q and k, the rotated keys and the values
          written into the sequences' cache pages
  attn    tq1_paged_attn: attention of each sequence's newest tokens over its pages (one token: decode;
          many: a prefill chunk)
  pages   tq1_pages_resize / tq1_pages_fork / tq1_pages_compact: the cache's page bookkeeping and page copies

With `own` false, run() computes the same in plain torch operations in 32 bits; with `own` true it makes the
library's calls.  The lengths of a case's sequences come from the case itself (its "shape" number), the
values from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # One decode step of one conversation: latency only.
        dict(name="rope_step_1", op="rope", shape=1, seqs=1, ctx_min=776, ctx_max=776, new_min=1, new_max=1,
             n_q=32, n_kv=8, d=128, rot=128, interleaved=False, factor=1.0, page=16, dtype="f16"),
        # A decode step of a batch; interleaved pairs over half of each head, an odd query group of five.
        dict(name="rope_step_64", op="rope", shape=2, seqs=64, ctx_min=40, ctx_max=16000, new_min=1, new_max=1,
             n_q=40, n_kv=8, d=128, rot=64, interleaved=True, factor=1.0, page=64, dtype="bf16"),
        # Ragged prompt chunks of several requests, positions scaled for a long context.
        dict(name="rope_chunk", op="rope", shape=3, seqs=7, ctx_min=1, ctx_max=9000, new_min=300, new_max=4000,
             n_q=40, n_kv=8, d=128, rot=128, interleaved=False, factor=8.0, page=32, dtype="bf16"),
        # The attention of that one conversation's decode step.
        dict(name="attn_step_1", op="attn", shape=1, seqs=1, ctx_min=776, ctx_max=776, new_min=1, new_max=1,
             n_q=32, n_kv=8, d=128, window=0, page=16, dtype="f16"),
        # A decode step of a batch with very different lengths: the cache is streamed once.
        dict(name="attn_step_64", op="attn", shape=2, seqs=64, ctx_min=40, ctx_max=16000, new_min=1, new_max=1,
             n_q=40, n_kv=8, d=128, window=0, page=64, dtype="bf16"),
        # One very long conversation: one row per head, a long axis to split.
        dict(name="attn_step_long", op="attn", shape=4, seqs=1, ctx_min=131070, ctx_max=131070, new_min=1, new_max=1,
             n_q=32, n_kv=4, d=128, window=0, page=16, dtype="f16"),
        # Prompt chunks mixed with short continuations, sliding window, small heads in groups of three.
        dict(name="attn_mixed", op="attn", shape=10, seqs=8, ctx_min=100, ctx_max=5000, new_min=1, new_max=1500,
             n_q=24, n_kv=8, d=64, window=1024, page=32, dtype="f16"),
        # A large chunk of a long prompt: bound by the matrix products.
        dict(name="attn_chunk", op="attn", shape=6, seqs=1, ctx_min=8192, ctx_max=8192, new_min=4096, new_max=4096,
             n_q=40, n_kv=8, d=128, window=0, page=64, dtype="bf16"),
        # A speculative decode step's bookkeeping: room for drafted tokens, then back to the accepted ones.
        dict(name="pages_draft", op="draft", shape=7, seqs=64, ctx_min=40, ctx_max=4000, draft=8,
             pools=16, n_kv=8, d=128, page=16, spare=500),
        # A beam-search round: the beams that lost are freed, the survivors forked into their places.
        dict(name="pages_beams", op="beams", shape=8, seqs=6, ctx_min=300, ctx_max=3000, beams=4,
             pools=64, n_kv=8, d=128, page=16, spare=100),
        # Turnover: finished sequences leave, the cache is compacted, others are admitted.
        dict(name="pages_turnover", op="turnover", shape=9, seqs=7, ctx_min=100, ctx_max=1500,
             pools=64, n_kv=8, d=128, page=16, spare=77),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = _draw_one(rng)
        if _cost(c) <= top and _plain_values(c) < 2.2e9:
            return c


def _draw_one(rng):
    op = rng.choice(["rope", "rope", "attn", "attn", "attn", "draft", "beams", "turnover"])
    shape = rng.randrange(1 << 20)
    n_kv, d, page = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op in ("rope", "attn"):
        group, dtype = rng.choice([1, 2, 3, 4, 5, 7, 8]), rng.choice(["f16", "bf16"])
        step = rng.random() < 0.5
        seqs = _log(rng, 1, 100) if step else _log(rng, 1, 12)
        ctx = _log(rng, 40, 130000) if seqs == 1 else _log(rng, 40, 16000)
        new = 1 if step else _log(rng, 2, 4096)
        c = dict(op=op, shape=shape, seqs=seqs, ctx_min=ctx if seqs == 1 else max(1, ctx // 50), ctx_max=ctx,
                 new_min=new if seqs == 1 else max(1, new // 40), new_max=new, n_q=n_kv * group, n_kv=n_kv, d=d,
                 page=page, dtype=dtype)
        if op == "rope":
            c |= dict(rot=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.5,
                      factor=rng.choice([1.0, 1.0, 4.0, 8.0]))
        else:
            c |= dict(window=rng.choice([0, 0, 0, _log(rng, 16, 5000)]))
        return c
    c = dict(op=op, shape=shape, seqs=_log(rng, 1, 9), ctx_min=20, ctx_max=_log(rng, 40, 3000), pools=_log(rng, 2, 64),
             n_kv=n_kv, d=d, page=page, spare=_log(rng, 50, 1000))
    if op == "draft":
        c |= dict(seqs=_log(rng, 1, 200), draft=rng.randint(1, 20))
    if op == "beams":
        c |= dict(beams=rng.randint(2, 8))
    return c


def _lengths(case):
    """Tokens before the call and new tokens of each sequence; one sequence has the largest of both."""
    rng = random.Random(case["shape"])
    n = case["seqs"]
    ctx = [_log(rng, case["ctx_min"], case["ctx_max"]) for _ in range(n)]
    new = [_log(rng, case.get("new_min", 1), case.get("new_max", 1)) for _ in range(n)]
    if n == 1:
        ctx, new = [case["ctx_max"]], [case.get("new_max", 1)]
    return ctx, new


def _up(a, b):
    return -(-a // b)


def _page_bytes(case):
    return case["n_kv"] * case["page"] * case["d"] * 2


def _visible(ctx, new, window):
    """Visible (row, key) pairs of one head, and the cache slots that any row sees."""
    w = window or ctx + new
    pairs = sum(min(ctx + i + 1, w) for i in range(new))
    return pairs, ctx + new - max(0, ctx + 1 - w)


def work(case):
    ctx, new = _lengths(case)
    op = case["op"]
    if op == "rope":
        t, vals = sum(new), case["d"] * (case["n_q"] + 2 * case["n_kv"])
        rotated = case["rot"] * (case["n_q"] + case["n_kv"])
        return {"bytes": t * vals * (4 + 2) + 4 * (case["rot"] // 2 + t + 2 * case["seqs"]), "flops": 3.0 * t * rotated}
    if op == "attn":
        seen = [_visible(c, n, case["window"]) for c, n in zip(ctx, new)]
        kv = 2 * 2 * case["n_kv"] * case["d"] * sum(s for _, s in seen)
        ids = 4 * sum(_up(s, case["page"]) for _, s in seen)
        return {"bytes": 2 * 2 * sum(new) * case["n_q"] * case["d"] + kv + ids + 8 * case["seqs"],
                "flops": 4.0 * case["n_q"] * case["d"] * sum(p for p, _ in seen)}
    ps, ints, copied = case["page"], 0, 0
    if op == "draft":  # each sequence's length and the entries that come and go; no page is copied
        ints = sum(4 + 2 * 2 * (_up(c + case["draft"], ps) - _up(c, ps)) for c in ctx)
    elif op == "beams":  # the last page of each fork, and its table row twice
        copied = sum(1 for c in ctx if c % ps) * (case["beams"] - 1)
        ints = sum(4 + 6 * _up(c, ps) for c in ctx) * (case["beams"] - 1)
    else:  # two rounds, in each of which a third of the pages moves
        held = sum(_up(c, ps) for c in ctx)
        copied, ints = 2 * held, 2 * (4 * 3 * held + 2 * 3 * held)
    return {"bytes": 2 * copied * case["pools"] * _page_bytes(case) + 4 * ints, "flops": 0.0}


def _cost(case):
    """Seconds that a case cannot do without, at rates of this class of machine; for the size of drawn cases only."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _plain_values(case):
    if case["op"] != "attn":
        return case["pools"] * _page_bytes(case) * 12 * case["seqs"] if "pools" in case else 0
    ctx, new = _lengths(case)
    return case["seqs"] * case["n_q"] * max(new) * max(c + n for c, n in zip(ctx, new))


# ----------------------------------------------------------------- states --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(lens, ps, spare, seed, rows=None):
    """A table of pages for sequences of these lengths, the pages in any order, `spare` pages in use by nobody."""
    held = [_up(v, ps) for v in lens]
    n_pages, width = sum(held) + spare, max(held) + 2
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((rows or len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    return table.cuda(), n_pages


def _cache(case, n_pages, g):
    shape = (2, n_pages, case["n_kv"], case["page"], case["d"])
    kv = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")
    for i in range(2):  # in pieces: a long cache's fp32 draw would not be small
        for p in range(0, n_pages, 4096):
            kv[i, p:p + 4096].normal_(generator=g)
    # A few channels of the keys are larger than the others, as in trained models.
    kv[0, ..., :: max(1, case["d"] // 4)] *= 3
    return kv


def prepare(case, seed):
    case = dict(case)
    op, g = case["op"], _gen(seed)
    ctx, new = _lengths(case)
    if op in ("rope", "attn"):
        lens, starts = [c + n for c, n in zip(ctx, new)], [0]
        for n in new:
            starts.append(starts[-1] + n)
        t, n_q, n_kv, d = starts[-1], case["n_q"], case["n_kv"], case["d"]
        table, n_pages = _tables(lens, case["page"], 5, seed)
        s = dict(case=case, t=t, max_len=max(lens), max_new=max(new), table=table, q_start=_ints(starts), kv_len=_ints(lens))
        if op == "rope":
            # One fused projection's output: q, k and v are column ranges of its rows.
            qkv = torch.empty(t, (n_q + 2 * n_kv) * d, device="cuda").normal_(generator=g)
            q, k, v = (qkv[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in ((0, n_q), (n_q, n_q + n_kv), (n_q + n_kv, n_q + 2 * n_kv)))
            s |= dict(q=q, k=k, v=v, mscale=1.0 if case["factor"] == 1 else 0.1 * math.log(case["factor"]) + 1,
                      kv=_cache(case, n_pages, g), q_out=torch.empty(t, n_q, d, dtype=DTYPES[case["dtype"]], device="cuda"),
                      inv_freq=_frequencies(case))
        else:
            s |= dict(kv=_cache(case, n_pages, g), scale=1 / math.sqrt(d),
                      q=torch.empty(t, n_q, d, device="cuda").normal_(generator=g).to(DTYPES[case["dtype"]]),
                      out=torch.empty(t, n_q, d, dtype=DTYPES[case["dtype"]], device="cuda"))
        if own:
            import bit_quantized_gemv_tq1_gb300 as tq
            s["tq"], s["cache"], s["batch"] = tq, tq.tq1_kv_cache(s["kv"][0], s["kv"][1]), tq.tq1_kv_batch(table, s["q_start"], s["kv_len"])
            if op == "attn":
                s["ws"] = torch.empty(max(16, tq.tq1_paged_attn_workspace_size(s["cache"], t, n_q, len(new))), dtype=torch.uint8, device="cuda")
        return s
    ps = case["page"]
    if op == "draft":
        rng = random.Random(case["shape"])
        kept = [c + rng.randint(0, case["draft"]) for c in ctx]
        lens, rows = kept, len(kept)
        spare, more = case["spare"] + len(ctx) * _up(case["draft"], ps), case["draft"]
    elif op == "beams":
        lens, rows, more = ctx, len(ctx) * case["beams"], 0
        spare = case["spare"] + rows
    else:
        lens, rows, spare, more = ctx * 3, 3 * len(ctx), case["spare"], 0
    table, n_pages = _tables([v + more for v in lens], ps, spare, seed, rows)
    held = torch.tensor([_up(v, ps) for v in lens] + [0] * (rows - len(lens)), device="cuda")
    if op == "turnover":  # the three groups lie behind one another, each in an order of its own
        per = sum(_up(c, ps) for c in ctx)
        order = torch.cat([torch.randperm(per, generator=torch.Generator().manual_seed(seed + i)) + i * per for i in range(3)])
        mask = torch.arange(table.shape[1], device="cuda") < held[:, None]
        table[mask] = order.to(torch.int32).cuda()
    table[torch.arange(table.shape[1], device="cuda") >= held[:, None]] = -1
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    pools = torch.randint(-(1 << 15), 1 << 15, (case["pools"], n_pages, case["n_kv"], ps, case["d"]), dtype=torch.int16,
                          device="cuda", generator=g)
    s = dict(case=case, table=table, refs=refs, pools=pools, kv_len=_ints(lens + [0] * (rows - len(lens))), ps=ps)
    n = len(ctx)
    if op == "draft":
        s |= dict(all=_ints(list(range(n))), longer=_ints([c + case["draft"] for c in ctx]), kept=_ints(kept))
    elif op == "beams":
        children = list(range(n, rows))
        s |= dict(children=_ints(children), parents=_ints([i % n for i in range(len(children))]), none=_ints([0] * len(children)))
    else:
        s |= dict(a=_ints(list(range(n))), c=_ints(list(range(2 * n, 3 * n))), lens=_ints(ctx), none=_ints([0] * n))
    if own:
        import bit_quantized_gemv_tq1_gb300 as tq
        s["tq"], s["pool"] = tq, tq.tq1_page_pool(pools, table, s["kv_len"], refs, ps)
        s["ws"] = torch.empty(tq.tq1_pages_workspace_size(s["pool"]), dtype=torch.uint8, device="cuda")
    return s


def _frequencies(case):
    """Inverse frequencies of the rotated pairs, low ones divided by the factor and those between blended."""
    rot = case["rot"]
    f = 10000.0 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if case["factor"] != 1:
        keep = ((8192 * f / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        f = f * ((1 - keep) / case["factor"] + keep)
    return f.to(torch.float32).cuda()


# -------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if op == "rope":
        if own:
            s["tq"].tq1_rope_append(s["cache"], s["batch"], s["q"], s["k"], s["v"], s["q_out"], s["inv_freq"], s["case"]["rot"],
                                    interleaved=s["case"]["interleaved"], mscale=s["mscale"])
            q = s["q_out"]
        else:
            q = _plain_rope(s)
        return {"q": q, "k_pages": s["kv"][0], "v_pages": s["kv"][1]}
    if op == "attn":
        if own:
            s["tq"].tq1_paged_attn(s["cache"], s["batch"], s["q"], s["out"], s["scale"], window=s["case"]["window"], ws=s["ws"])
            return s["out"]
        return _plain_attn(s)
    if own:
        tq, pool, ws = s["tq"], s["pool"], s["ws"]
        resize = lambda seqs, lens: tq.tq1_pages_resize(pool, seqs, lens, ws)  # noqa: E731
        fork, compact = (lambda a, b: tq.tq1_pages_fork(pool, a, b, ws)), (lambda: tq.tq1_pages_compact(pool, ws))
    else:
        resize = lambda seqs, lens: _plain_resize(s, seqs, lens)  # noqa: E731
        fork, compact = (lambda a, b: _plain_fork(s, a, b)), (lambda: _plain_compact(s))
    if op == "draft":
        resize(s["all"], s["longer"])
        resize(s["all"], s["kept"])
    elif op == "beams":
        resize(s["children"], s["none"])
        fork(s["parents"], s["children"])
    else:
        resize(s["a"], s["none"])
        compact()
        resize(s["a"], s["lens"])
        resize(s["c"], s["none"])
        compact()
        resize(s["c"], s["lens"])
    return {"table": s["table"], "kv_len": s["kv_len"], "refs": s["refs"], "pools": s["pools"]}


def _owner(s):
    """The sequence and the position of each new token."""
    tok = torch.arange(s["t"], device="cuda")
    seq = (s["q_start"][1:, None] <= tok).sum(0)
    return seq, s["kv_len"].long()[seq] - s["q_start"].long()[seq + 1] + tok


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1 if interleaved else -2).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rope(s):
    c, dtype = s["case"], s["q_out"].dtype
    seq, pos = _owner(s)
    angle = (pos.float()[:, None] * s["inv_freq"])[:, None, :]
    cos, sin = angle.cos() * s["mscale"], angle.sin() * s["mscale"]
    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    s["kv"][0][page, :, slot] = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]).to(dtype)
    s["kv"][1][page, :, slot] = s["v"].to(dtype)
    return _rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).to(dtype)


def _plain_attn(s):
    c, n, L, M = s["case"], s["case"]["seqs"], s["max_len"], s["max_new"]
    H, d, G = c["n_kv"], c["d"], c["n_q"] // c["n_kv"]
    pages = s["table"][:, :_up(L, c["page"])].clamp(min=0).long()
    K, V = (x[pages].transpose(1, 2).reshape(n, H, -1, d)[:, :, :L].float() for x in (s["kv"][0], s["kv"][1]))
    ln, start = s["kv_len"].long(), s["q_start"].long()
    new = start[1:] - start[:-1]
    i, j = torch.arange(M, device="cuda"), torch.arange(L, device="cuda")
    there = i < new[:, None]
    at = torch.where(there, start[:-1, None] + i, s["t"])
    q = s["q"][at.clamp(max=s["t"] - 1)].float().unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).reshape(n, H, G * M, d)
    pos = (ln - new)[:, None] + i
    seen = (j <= pos[..., None]) & (j < ln[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    V = torch.where((j < ln[:, None])[:, None, :, None], V, 0.0)
    e = (q @ K.transpose(2, 3)).mul_(s["scale"]).view(n, H, G, M, L)
    e.masked_fill_(~seen[:, None, None], -math.inf)
    e.sub_(e.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = e.sum(-1).clamp(min=1e-37)
    o = (e.view(n, H, G * M, L) @ V).view(n, H, G, M, d) / total[..., None]
    out = torch.zeros(s["t"] + 1, c["n_q"], d, dtype=s["q"].dtype, device="cuda")
    out[at] = o.permute(0, 3, 1, 2, 4).reshape(n, M, c["n_q"], d).to(out.dtype)
    return out[:-1]


def _give(s, seqs, first, need, copied, sources, upto):
    """Deals the lowest free pages: `copied` first (a copy of `sources`), then the table's places first .. upto."""
    free = (s["refs"] == 0).nonzero()[:, 0]
    before = need.cumsum(0) - need
    fits = before + need <= free.numel()
    src, dst = sources[copied & fits], free[before[copied & fits]]
    s["pools"][:, dst] = s["pools"][:, src]
    idx = torch.arange(s["table"].shape[1], device="cuda")
    put = (idx >= first[:, None]) & (idx < upto[:, None]) & fits[:, None]
    ids = free[(before[:, None] + idx - first[:, None])[put]]
    rows = s["table"][seqs]
    rows[put] = ids.to(torch.int32)
    s["table"][seqs] = rows
    s["refs"].index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    return fits


def _plain_resize(s, seqs, lens):
    seqs, lens, ps = seqs.long(), lens.long(), s["ps"]
    old = s["kv_len"][seqs].long()
    had, gets = (old + ps - 1) // ps, (lens + ps - 1) // ps
    idx = torch.arange(s["table"].shape[1], device="cuda")
    rows = s["table"][seqs]
    drop = (idx >= gets[:, None]) & (idx < had[:, None])
    s["refs"].index_add_(0, rows[drop].long(), -torch.ones_like(rows[drop]))
    rows[drop] = -1
    s["table"][seqs] = rows
    last = rows.gather(1, (had - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0).long()
    shared = (lens > old) & (old % ps != 0) & (s["refs"][last] > 1)
    first = had - shared.long()
    fits = _give(s, seqs, first, (gets - first).clamp(min=0), shared, last, gets)
    left = last[shared & fits]
    s["refs"].index_add_(0, left, -torch.ones_like(left, dtype=torch.int32))
    s["kv_len"][seqs] = torch.where(fits, lens, old).to(torch.int32)


def _plain_fork(s, parents, children):
    parents, children, ps = parents.long(), children.long(), s["ps"]
    ln = s["kv_len"][parents].long()
    full = ln // ps
    rows = s["table"][parents]
    shared = torch.arange(rows.shape[1], device="cuda") < full[:, None]
    s["table"][children] = torch.where(shared, rows, -1)
    last = rows.gather(1, full.clamp(max=rows.shape[1] - 1)[:, None])[:, 0].clamp(min=0).long()
    part = (ln % ps) != 0
    s["refs"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    _give(s, children, full, part.long(), part, last, full + part.long())
    s["kv_len"][children] = ln.to(torch.int32)


def _plain_compact(s):
    live = s["refs"] > 0
    n = int(live.sum())
    holes, movers = (~live[:n]).nonzero()[:, 0], live[n:].nonzero()[:, 0] + n
    s["pools"][:, holes] = s["pools"][:, movers]
    to = torch.arange(live.numel(), dtype=torch.int32, device="cuda")
    to[movers] = holes.to(torch.int32)
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], s["table"]))
    s["refs"][holes] = s["refs"][movers]
    s["refs"][movers] = 0


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time; page bookkeeping computes no numbers."""
    if case["op"] not in ("rope", "attn"):
        return None
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    k, v = s["kv"][0].double(), s["kv"][1].double()
    q, at, ps = s["q"].double(), 0, case["page"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for i, (c, n) in enumerate(zip(ctx, new)):
        pages = s["table"][i, :_up(c + n, ps)].long()
        if case["op"] == "rope":
            pos = torch.arange(c, c + n, device="cuda")
            z = torch.polar(torch.full((n, case["rot"] // 2), s["mscale"], dtype=torch.float64, device="cuda"),
                            pos.double()[:, None] * s["inv_freq"].double())[:, None]
            for x, put in ((q[at:at + n], None), (s["k"][at:at + n].double(), k), (s["v"][at:at + n].double(), v)):
                y = x.clone()
                if put is not v:
                    r = case["rot"]
                    first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
                    turned = torch.complex(x[..., first], x[..., second]) * z
                    y[..., first], y[..., second] = turned.real, turned.imag
                if put is None:
                    out[at:at + n] = y
                else:
                    put[pages[pos // ps], :, pos % ps] = y
        else:
            rows, cols = torch.arange(c, c + n, device="cuda")[:, None], torch.arange(c + n, device="cuda")
            hidden = cols > rows
            if case["window"]:
                hidden |= cols <= rows - case["window"]
            group = case["n_q"] // case["n_kv"]
            for h in range(case["n_q"]):
                keys, values = (x[pages, h // group].flatten(0, 1)[:c + n] for x in (k, v))
                scores = (q[at:at + n, h] @ keys.T / math.sqrt(case["d"])).masked_fill_(hidden, -math.inf)
                out[at:at + n, h] = scores.softmax(-1) @ values
        at += n
    return {"q": out, "k_pages": k, "v_pages": v} if case["op"] == "rope" else out
