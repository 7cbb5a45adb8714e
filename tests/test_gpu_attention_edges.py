"""Attention at the edges of its contract: biases that hide keys or are of
large magnitude, streams and workspaces of the caller's choice, single caches
without pages.  References in 64 bits; helpers of the operators' main tests."""

import numpy as np
import pytest
import torch

import attention_reference as ref
import recommender_sparse_embeddings_gb300 as tbe
from test_gpu_attention import DTYPES, Batch, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("starts", [[0, 1, 30], [0, 5, 4000]])
@pytest.mark.parametrize("heads,kv_heads,histories", [(6, 3, 200), (8, 2, 5)])
def test_lowest_bias_in_some_heads(dim, starts, heads, kv_heads, histories):
    """The type's lowest value in the last bucket of every other head hides its
    keys there (every row has others), whatever the heads beside it hold: in
    batches whose tiles are taken in turn, and under query heads that share a
    key-value head."""
    g = np.random.default_rng(dim + histories)
    lengths = g.integers(1, 400, histories)
    lengths[0] = 4500 if starts[-1] > 400 else 700
    b = Batch(torch.bfloat16, heads, kv_heads, dim, lengths.tolist(), 0, 0, starts, seed=40)
    b.bias[-1, ::2] = -float("inf")
    want = b.run()
    b.bias[-1, ::2] = torch.finfo(torch.bfloat16).min
    for _ in range(3):
        got = b.run()
        for x in want:
            assert torch.equal(got[x], want[x]), x
    assert tbe.tbe_attention_get_error(b.handle) == tbe.TBE_OK
