"""examples/output_layer.py: the loss falls, and the 4-bit layer answers like
the trained one.  The centres of V classes in D dimensions lie sqrt(2 D) apart
and the noise has 0.5 in each direction, so a trained layer separates them by
tens of its logits' own errors; before the first step all logits are 0 and the
loss is log V."""
import importlib.util
import math
import os

import pytest

from gpu_helpers import device, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens,features,classes", [(48, 256, 12), (1500, 200, 201)])
def test_output_layer_example(tokens, features, classes):
    device()
    say("output layer", tokens, features, classes)
    spec = importlib.util.spec_from_file_location("output_layer", os.path.join(ROOT, "examples", "output_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.main(tokens, features, classes, steps=6)
    assert abs(r["loss"][0] - math.log(classes)) < 1e-3
    assert r["loss"][-1] < 0.5 * r["loss"][0]
    assert r["accuracy"] > 0.95 and r["accuracy_4bit"] > 0.95
