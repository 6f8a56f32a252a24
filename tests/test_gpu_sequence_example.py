"""The sequence operators together with the embedding stage, as the example uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_ranking_example_learns():
    spec = importlib.util.spec_from_file_location("sequence_ranking",
                                                  os.path.join(ROOT, "examples", "sequence_ranking.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    loss, right, repeat = example.main(steps=150, quiet=True)
    assert loss < 0.45 and right > 0.8 and repeat > 0.8, (loss, right, repeat)
