"""The example runs: its loss falls, and the mixed batch agrees with each user's own call (both
outputs are rounded once to bf16 from sums of the same terms: two roundings of the largest apart)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_train_and_serve():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_and_serve.py")
    spec = importlib.util.spec_from_file_location("train_and_serve", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, worst = mod.main(25, quiet=True)
    assert losses[-1] < 0.5 * losses[0]
    assert worst <= 2 * 2.0 ** -8
