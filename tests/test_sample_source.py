"""What one thread of the sampling kernel decides is read by the others between two barriers."""
import os
import re

from bit_quantized_gemv_tq1_gb300 import build as B


def test_decisions_are_read_before_the_next_barrier():
    # Behind the barrier that ends a turn, the first thread goes on to decide() and writes these again while
    # slower warps are still at the end of the turn.
    text = re.sub(r"//[^\n]*", "", open(os.path.join(B.CSRC, "sample.cu")).read())
    loop = text[text.index("act = decide()"):]
    turn = loop[loop.index("__syncthreads();") + len("__syncthreads();"):loop.index("a.ids[r] = sh.state.token")]
    told = re.compile(r"\b(?:s|sh\.state)\.(act|leave|last)\b")
    first = re.search(r"__syncthreads|dismiss\(|if \(act", turn).start()
    assert {m.group(1) for m in told.finditer(turn[:first])} == {"act", "leave", "last"}
    assert told.search(turn, first) is None


def test_every_list_is_looked_at_for_its_length():
    # Gathered tokens beyond the list's room are dropped: no list is used before that is ruled out.
    text = re.sub(r"//[^\n]*", "", open(os.path.join(B.CSRC, "sample.cu")).read())
    asked = re.findall(r"TQ1_DO\(ask\([^;]*kGather[^;]*;\s*(\S[^;{]*)", text)
    assert len(asked) == 4
    for then in asked:
        assert re.match(r"if \(sh\.sum\.n (<=|>) kList\)", then), then
