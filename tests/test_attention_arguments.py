"""Arguments of tbe_attention_create that the binding refuses by itself."""

import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe


@pytest.mark.parametrize("kw", [dict(window=2 ** 32), dict(window=2 ** 32 + 5), dict(window=-2 ** 31 - 1),
                                dict(sinks=2 ** 32), dict(heads=2 ** 32 + 4), dict(kv_heads=2 ** 32 + 2),
                                dict(head_dim=2 ** 32 + 64), dict(bucket_starts=[0, 2 ** 32 + 1])])
def test_numbers_outside_int32_are_refused(kw, monkeypatch):
    """The library takes 32-bit fields: a window of 2^32 + 5 would become 5."""
    monkeypatch.setattr(tbe, "load_library", lambda: pytest.fail("reached the library"))
    args = dict(heads=4, kv_heads=2, head_dim=64, dtype=torch.bfloat16)
    args.update(kw)
    with pytest.raises(ValueError):
        tbe.tbe_attention_create(**args)
