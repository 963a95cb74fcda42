"""The example layer (quantised products, rotary positions, cache, tree attention) against its float64 form.

The reference has exact keys and values, the layer those of the cache: uniform rounding on a grid of maxq steps over a
row's range of about 6 standard deviations is an error of 6 / (maxq sqrt(12)) of one, 0.7% at 8 bits and 12% at 4, in
keys and in values, about averaged over the positions seen; three times their joint size is allowed, and 1% for the
bf16 queries, attention results and operands."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,allowed", [(8, 0.01 + 3 * 1.5 * 0.007), (4, 0.01 + 3 * 1.5 * 0.12)])
def test_draft_step(bits, allowed):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    err = m.main(bits)
    print("error %.3e" % err, flush=True)
    assert 0 < err <= allowed
