"""tq1_moe / tq2_moe on rows that only one of its two forms has room for, whatever the batch."""
import pytest
import torch

from tests.test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from bit_quantized_gemv_tq1_gb300 import build
    build.build()
    import bit_quantized_gemv_tq1_gb300 as tq
    return tq


# One token has too little work to share; of 200 tokens of two experts many share an expansion.
@pytest.mark.parametrize("fmt", ["tq1", "tq2"])
@pytest.mark.parametrize("k,f,t,experts,top_k", [(14336, 512, 1, 3, 2), (14336, 512, 200, 2, 1), (14336, 256, 5, 130, 3), (16384, 256, 1, 2, 1),
                                                 (10752, 256, 2, 2, 2), (11008, 256, 2, 2, 2), (12800, 256, 2, 2, 2), (13056, 256, 2, 2, 2)])
def test_rows_longer_than_a_pair_has_room_for(tq, fmt, k, f, t, experts, top_k):
    Layer(tq, fmt, experts, k, f, seed=t).check(t, top_k)


@pytest.mark.parametrize("fmt", ["tq1", "tq2"])
def test_a_token_alone_and_in_a_batch_on_long_rows(tq, fmt):
    k, f, t = 14336, 256, 70
    layer = Layer(tq, fmt, 3, k, f, seed=3)
    q8, logits = layer.acts(t), layer.logits(t)
    many, one = torch.empty(t, k, device="cuda"), torch.empty(1, k, device="cuda")
    layer.call(q8, logits, 2, many)
    for i in (0, 33, 69):
        layer.call(q8[i:i + 1].clone(), logits[i:i + 1].clone(), 2, one)
        assert torch.equal(one[0], many[i])


@pytest.mark.parametrize("fmt,k,f,t,experts", [("tq2", 16384, 49152, 2, 1), ("tq1", 16384, 49152, 1, 1), ("tq1", 22528, 256, 2, 2), ("tq2", 256, 55040, 30, 1),
                                               ("tq2", 16384, 256, 40, 1024)])
def test_the_longest_rows_that_are_taken(tq, fmt, k, f, t, experts):
    Layer(tq, fmt, experts, k, f, seed=5).check(t, 1)
    torch.cuda.empty_cache()
