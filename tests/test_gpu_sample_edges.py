"""tq1_sample where many logits are +inf (more than one list holds)."""
import math
from fractions import Fraction

import pytest
import torch

from tests.test_gpu_sample import INF, NAN, TYPES, f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from bit_quantized_gemv_tq1_gb300 import build
    build.build()
    import bit_quantized_gemv_tq1_gb300 as tq
    return tq


def choose(tq, x, u, **kw):
    t = x.shape[0]
    ids, probs = torch.full((t,), -9, dtype=torch.int32, device="cuda"), torch.full((t,), NAN, device="cuda")
    kw = {k: torch.full((t,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in kw.items()}
    tq.tq1_sample(x, f32(u), ids, probs=probs, **kw)
    assert tq.tq1_sync_status() == 0
    return ids.tolist(), probs.tolist()


def even(n, u, top_k=0, top_p=1.0, min_p=0.0, temperature=1.0):
    """The place among n equal tokens, and how many are kept: in whole numbers, nothing is rounded."""
    u, top_p = float(f32([u])[0]), float(f32([top_p])[0])
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        n = max(1, math.ceil(Fraction(top_p) * n))
    return math.floor(Fraction(u) * n), n


FILTERS = [dict(), dict(top_k=7), dict(top_k=1024), dict(top_k=1025), dict(top_k=1500), dict(top_p=0.3), dict(top_p=0.9), dict(min_p=0.1),
           dict(min_p=1.0), dict(temperature=0.3), dict(temperature=INF), dict(top_k=1300, top_p=0.9, min_p=0.5)]


# A row in one block of either size (many rows), and in several (few rows).
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,v,n", [(3, 4000, 1023), (3, 4000, 1024), (3, 4000, 1025), (2, 4000, 1100), (4, 4000, 3000), (310, 4001, 1200),
                                   (1, 20001, 1025), (2, 70001, 1200), (1, 131072, 5000), (1, 200000, 70001), (2, 5000, 5000)])
def test_many_infinities(tq, dtype, t, v, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = 3 * torch.randn(t, v, device="cuda", generator=g)
    x[:, 1::5] = NAN
    x[:, 2::7] = -INF
    x[:, 3::11] = torch.finfo(TYPES[dtype]).max
    at = []
    for i in range(t):  # the first token among the masked ones, unless all are +inf
        p = torch.arange(v, device="cuda") if n == v else 1 + torch.randperm(v - 1, device="cuda", generator=g)[:n]
        x[i, 0] = -INF
        x[i, p] = INF
        at.append(p.sort().values.tolist())
    x = x.to(TYPES[dtype])
    if n != v:
        x[:, 0] = 0
    for kw in FILTERS if t < 100 else FILTERS[::3]:
        for us in ([0.0, 0.37, 0.5, 1 - 2.0 ** -24], [0.999, 0.1, 1e-3, 0.75]):
            u = [us[i % 4] for i in range(t)]
            ids, probs = choose(tq, x, u, **kw)
            for i in range(t):
                place, kept = even(n, u[i], **kw)
                assert ids[i] == at[i][place], (kw, i, u[i], ids[i], at[i][place])
                assert abs(probs[i] - 1 / kept) <= 2.0 ** -23 / kept


def by_logit(row):
    return sorted(range(len(row)), key=lambda i: (-row[i], i))


@pytest.mark.parametrize("v", [700, 5000, 70001])
def test_subnormal_logits(tq, v):
    """Logits of a few steps of 2^-149: halves of odd ones are rounded, and all weigh 1."""
    x = torch.zeros(5, v)
    steps = {0: {11: 5, 30: 4, 77: 4, 600: 3}, 1: {11: -5, 30: 4, 77: 1, 600: 3}}
    for i in steps:
        for at, n in steps[i].items():
            x[i, at] = n * 2.0 ** -149
    g = torch.Generator().manual_seed(v)
    x[2] = torch.randint(0, 7, (v,), generator=g) * 2.0 ** -149
    x[3] = torch.randint(-9, 0, (v,), generator=g) * 2.0 ** -149
    x[4] = 3 * 2.0 ** -149
    order = [by_logit(row) for row in x.tolist()]
    dev = x.cuda()
    for kw in (dict(top_k=2), dict(top_k=3), dict(top_k=40), dict(top_k=600), dict(), dict(top_p=0.5), dict(min_p=0.5)):
        for u in (0.0, 0.37, 1 - 2.0 ** -24):
            ids, probs = choose(tq, dev, [u] * 5, **kw)
            for i in range(5):
                place, kept = even(v, u, **kw)
                assert ids[i] == order[i][place], (kw, i, u, order[i].index(ids[i]) if ids[i] >= 0 else -1, place)
                assert abs(probs[i] - 1 / kept) <= 2.0 ** -23 / kept
