"""The paged cache's kernels begin before the kernel ahead of them has ended, so
they read what it may be writing: through ordinary loads only."""
import os
import re

import pytest

from bit_quantized_gemv_tq1_gb300 import build as B


@pytest.mark.parametrize("name", ["kv.cuh", "rope.cu", "attn.cu", "attn_tile.cu", "pages.cu"])
def test_no_read_only_loads(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(B.CSRC, name)).read())
    assert "pdl_wait" in text or name == "kv.cuh"
    # A pointer that is const and __restrict__ lets the compiler choose such loads by itself.
    assert re.findall(r"__ldg|ld\.global\.nc|ld\.nc|__restrict__", text) == []


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(B.CSRC) if f.endswith((".cu", ".cuh"))))
def test_read_only_loads_are_of_weights(name):
    # The other kernels begin early too: activations, routing ids, scales and
    # row ids come through ordinary loads; what no call writes, the weights'
    # bytes outside whole 16-byte pieces, may come through read-only ones.
    text = re.sub(r"//[^\n]*", "", open(os.path.join(B.CSRC, name)).read())
    weights = {"mmv.cu": 1, "mmv_mma.cu": 1, "mmv_small.cu": 1, "moe_small.cu": 2}
    assert len(re.findall(r"__ldg|ld\.global\.nc|ld\.nc", text)) == weights.get(name, 0)
    assert "__restrict__" not in text
