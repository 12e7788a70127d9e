"""The decoder-layer operators together: examples/decoder_layer.py against its
plain fp64 computation."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_two_layers_from_prompt_to_forks():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    results = example.run()
    assert sorted(results) == [0, 1, 3, 4, 5]
    assert [results[s][0].shape[0] for s in (0, 1, 3, 4, 5)] == [203, 43, 75, 42, 301]
    for got, want in results.values():
        # The attention's output and the second layer's input are rounded to 8
        # bits per 32 values (half a step of 1/127 of their largest): a value
        # that falls on the other side of a step, from a difference of 2^-11 or
        # less before, moves by a whole one.  1/254 of the norm per rounding,
        # three of them behind a difference, bounds what that can come to.
        rel = (got - want).norm(dim=1) / want.norm(dim=1)
        assert (rel < 3 / 254).all(), float(rel.max())
