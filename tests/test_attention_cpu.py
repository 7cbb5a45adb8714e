"""Host-side checks of the attention operators that need no GPU."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_reference as ref
import recommender_sparse_embeddings_gb300 as tbe

built = pytest.mark.skipif(not os.path.exists(tbe.library_path()),
                           reason="library not built (run __graft_entry__.build())")


@pytest.mark.parametrize("window,sinks,group,starts", [(0, 0, 1, None), (3, 2, 2, [0, 1, 2, 5]), (1, 0, 1, [0]),
                                                       (4, 6, 3, [0, 3])])
def test_reference_gradients_match_differences(window, sinks, group, starts):
    """The 64-bit reference's gradients against central differences of its
    forward (step 1e-5: truncation about 1e-10, rounding about 1e-11)."""
    g = np.random.default_rng(window + 10 * sinks)
    off, hk, d = [0, 5, 5, 6, 15], 2, 3
    x = {"q": g.standard_normal((15, hk * group, d)), "k": g.standard_normal((15, hk, d)),
         "v": g.standard_normal((15, hk, d))}
    if starts:
        x["bias"] = g.standard_normal((len(starts), hk * group))
    up = g.standard_normal(x["q"].shape)

    def loss(y):
        r, _ = ref.attention(y["q"], y["k"], y["v"], off, window, sinks, 0.7, starts, y.get("bias"))
        return float((r["out"] * up).sum())

    r, _ = ref.attention(x["q"], x["k"], x["v"], off, window, sinks, 0.7, starts, x.get("bias"), up)
    for name in x:
        step = g.standard_normal(x[name].shape)
        want = (loss({**x, name: x[name] + 1e-5 * step}) - loss({**x, name: x[name] - 1e-5 * step})) / 2e-5
        assert abs(want - float((r["grad_" + name] * step).sum())) < 1e-7, name


def test_relative_buckets():
    for n, most in ((1, 1), (2, 5), (8, 50), (31, 200), (32, 128), (32, 32), (64, 2000), (256, 65535)):
        s = tbe.tbe_relative_buckets(n, most)
        assert len(s) == n and s[0] == 0 and all(a < b for a, b in zip(s, s[1:]))
        assert s[:max(1, n // 2)] == list(range(max(1, n // 2)))
        if n > 1:
            assert s[-1] == most
    with pytest.raises(ValueError):
        tbe.tbe_relative_buckets(8, 5)
    with pytest.raises(ValueError):
        tbe.tbe_relative_buckets(0, 5)


def _create(**kw):
    lib = tbe.load_library()
    starts = kw.pop("starts", None)
    arr = (ctypes.c_int32 * max(1, len(starts or ())))(*(starts or ()))
    base = dict(dtype=2, heads=4, kv_heads=2, head_dim=64, window=0, sinks=0, scale=1.0,
                num_buckets=len(starts or ()))
    base.update(kw)
    cfg = tbe._AttentionConfig(*[base[n] for n in ("dtype", "heads", "kv_heads", "head_dim", "window", "sinks",
                                                   "scale", "num_buckets")], arr)
    out = ctypes.c_void_p(7)
    rc = lib.tbe_attention_create(ctypes.byref(cfg), ctypes.byref(out))
    return rc, out.value


@built
@pytest.mark.parametrize("kw", [dict(dtype=3), dict(heads=0), dict(kv_heads=0), dict(heads=5), dict(head_dim=0),
                                dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(num_buckets=-1), dict(starts=[1, 2]),
                                dict(starts=[0, 2, 2]), dict(starts=[0, 3, 1])])
def test_create_refuses_bad_arguments_without_cuda(kw):
    rc, out = _create(**kw)
    assert rc == tbe.TBE_ERR_INVALID_ARG and out is None


@built
@pytest.mark.parametrize("kw", [dict(head_dim=257), dict(sinks=129), dict(heads=2048, kv_heads=1),
                                dict(starts=list(range(257))), dict(starts=[0, 65536])])
def test_create_refuses_what_is_outside_the_limits(kw):
    rc, out = _create(**kw)
    assert rc == tbe.TBE_ERR_UNSUPPORTED and out is None


@built
def test_calls_refuse_null_handles():
    lib = tbe.load_library()
    assert lib.tbe_attention_create(None, None) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_attention_workspace_bytes(None, 1, 1, 0) == 0
    assert lib.tbe_attention_decode_workspace_bytes(None, 1, 1) == 0
    z = [None] * 16
    assert lib.tbe_attention_forward(None, *z[:5], 0, 1, 1, *z[:3], 0, None) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_attention_get_error(None, None) == tbe.TBE_ERR_INVALID_ARG
    lib.tbe_attention_destroy(None)
