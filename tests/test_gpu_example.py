"""The mixture-of-experts example learns its text and draws what the text allows."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


def test_the_example_learns():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixture_of_experts.py")
    spec = importlib.util.spec_from_file_location("mixture_of_experts", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last, allowed = example.main(steps=120, quiet=True)
    assert first > 0.8 * math.log(example.VOCAB)
    assert last < 1.5 * math.log(3)  # the text's own entropy is ln 3
    assert allowed > 0.9
