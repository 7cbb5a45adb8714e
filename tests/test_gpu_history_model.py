"""The example that trains and serves a model over user histories."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_history_model_learns_and_serves():
    import history_model

    losses, error = history_model.main(users=40, steps=25, verbose=False)
    assert losses[-1] < 0.9 * losses[0], losses
    # weights and results of two kernels, each rounded to bf16 (2^-8), of
    # values up to about 4
    assert error <= 4 * 4 * 2.0 ** -8
