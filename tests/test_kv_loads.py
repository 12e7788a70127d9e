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
