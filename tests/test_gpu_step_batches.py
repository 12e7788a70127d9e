"""A row or token alone and in batches of other sizes, which other kernels or divisions of the work compute."""
import pytest
import torch

from tests.test_gpu_moe_layer import Layer
from tests.test_gpu_norm import TYPES, gen, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from bit_quantized_gemv_tq1_gb300 import build
    build.build()
    import bit_quantized_gemv_tq1_gb300 as tq
    return tq


@pytest.mark.parametrize("k,delta", [(2080, "f32"), (5120, "bf16"), (8192, "f16"), (6144, "")])
def test_a_norms_rows(tq, k, delta):
    """One, two and four groups a thread, and rows copied ahead: each sum is within its bound of the exact one, so two are within two."""
    g = gen(k)
    x = torch.randn(1400, k, device="cuda", generator=g)
    d = torch.randn(1400, k, device="cuda", generator=g).to(TYPES[delta]) if delta else None
    many = torch.empty_like(x)
    tq.tq1_rms_norm(x, None, 1e-6, y=many, delta=d)
    for t in (1, 48, 400, 1000):
        y, again = torch.empty(t, k, device="cuda"), torch.empty(t, k, device="cuda")
        for out in (y, again):
            tq.tq1_rms_norm(x[:t], None, 1e-6, y=out, delta=None if d is None else d[:t])
        assert torch.equal(y, again)
        assert ((y.double() - many[:t].double()).abs() <= 2 * ops(k) * many[:t].abs().double()).all()


# A few tokens go pair by pair, many share their experts' expansions; a pair's sums have one order in both.
@pytest.mark.parametrize("fmt", ["tq1", "tq2"])
@pytest.mark.parametrize("k,f,experts,top_k,t", [(2048, 768, 16, 4, 64), (4096, 2816, 8, 2, 24), (512, 512, 9, 4, 400), (1024, 1536, 4, 1, 200)])
def test_an_expert_layers_tokens(tq, fmt, k, f, experts, top_k, t):
    layer = Layer(tq, fmt, experts, k, f, seed=k)
    q8, logits = layer.acts(t), layer.logits(t)
    logits[2, 1:] = float("-inf")
    logits[3] = float("nan")
    res = torch.randn(t, k, device="cuda", generator=layer.g)
    many, ids, weights = torch.empty(t, k, device="cuda"), torch.empty(t, top_k, dtype=torch.int32, device="cuda"), torch.empty(t, top_k, device="cuda")
    layer.call(q8, logits, top_k, many, res=res, ids=ids, weights=weights, renormalize=False)
    for at, n in ((0, 1), (2, 2), (1, 4), (t - 1, 1), (t // 2, 7)):
        s = slice(at, at + n)
        out, few, own = torch.empty(n, k, device="cuda"), torch.empty(n, top_k, dtype=torch.int32, device="cuda"), torch.empty(n, top_k, device="cuda")
        layer.call(q8[s].clone(), logits[s].clone(), top_k, out, res=res[s].clone(), ids=few, weights=own, renormalize=False)
        assert torch.equal(out, many[s]) and torch.equal(few, ids[s]) and torch.equal(own, weights[s])
