"""The policy-step example's decoding: tokens of the vocabulary, the same for the same seed."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decoding_runs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import policy_step as ex

    model = ex.TokenModel(1009, 72)
    tokens = ex.decode(model, 5, 6, seed=1)
    assert len(tokens) == 6 and all(0 <= t < 1009 for t in tokens) and tokens == ex.decode(model, 5, 6, seed=1)
