"""Host-side checks of layer norm and the softmax loss that need no GPU."""

import ctypes
import os

import numpy as np
import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe
import rows_reference as ref

built = pytest.mark.skipif(not os.path.exists(tbe.library_path()),
                           reason="library not built (run __graft_entry__.build())")


@pytest.mark.parametrize("affine", [True, False])
def test_norm_reference_gradients_match_differences(affine):
    """Central differences of step 1e-5: truncation about 1e-10, rounding about 1e-10."""
    g = np.random.default_rng(3)
    t, up, on = g.standard_normal((4, 7)), g.standard_normal((4, 7)), g.standard_normal((4, 7))
    p = {"w": g.standard_normal(7), "b": g.standard_normal(7)} if affine else {}

    def value(t, p):
        return float((ref.norm(t, 1e-3, p.get("w"), p.get("b"))[0]["out"] * up).sum() + (t * on).sum())

    r, _ = ref.norm(t, 1e-3, p.get("w"), p.get("b"), up, on)
    step = g.standard_normal(t.shape) * 1e-5
    assert abs((value(t + step, p) - value(t - step, p)) / 2 - (r["grad_x"] * step).sum()) < 1e-13
    for key, name in (("w", "grad_weight"), ("b", "grad_bias")) if affine else ():
        step = g.standard_normal(7) * 1e-5
        diff = value(t, {**p, key: p[key] + step}) - value(t, {**p, key: p[key] - step})
        assert abs(diff / 2 - (r[name] * step).sum()) < 1e-13


def test_loss_reference_gradients_match_differences():
    g = np.random.default_rng(4)
    x, w, up = g.standard_normal((6, 5)), g.standard_normal((9, 5)), g.standard_normal(6)
    targets = np.array([0, 8, -1, 3, 3, -100])

    def value(x, w):
        return float((ref.loss(x, w, targets, 1.7)[0]["loss"] * up).sum())

    r, _ = ref.loss(x, w, targets, 1.7, up)
    dx, dw = g.standard_normal(x.shape) * 1e-5, g.standard_normal(w.shape) * 1e-5
    assert abs((value(x + dx, w) - value(x - dx, w)) / 2 - (r["grad_x"] * dx).sum()) < 1e-13
    assert abs((value(x, w + dw) - value(x, w - dw)) / 2 - (r["grad_table"] * dw).sum()) < 1e-13


def _create_norm(**kw):
    base = dict(dtype=2, dim=64, eps=1e-5, has_weight=1, has_bias=1)
    base.update(kw)
    out = ctypes.c_void_p(7)
    rc = tbe.load_library().tbe_layer_norm_create(ctypes.byref(tbe._LayerNormConfig(*base.values())), ctypes.byref(out))
    return rc, out.value


def _create_loss(**kw):
    base = dict(dtype=2, dim=64, scale=1.0)
    base.update(kw)
    out = ctypes.c_void_p(7)
    rc = tbe.load_library().tbe_softmax_loss_create(ctypes.byref(tbe._SoftmaxLossConfig(*base.values())),
                                                    ctypes.byref(out))
    return rc, out.value


@built
@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(dim=0), dict(dim=-4), dict(eps=-1e-9),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(has_weight=2),
                                dict(has_bias=-1)])
def test_norm_create_refuses_bad_arguments_without_cuda(kw):
    assert _create_norm(**kw) == (tbe.TBE_ERR_INVALID_ARG, None)


@built
@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(dim=0), dict(dim=-4), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_loss_create_refuses_bad_arguments_without_cuda(kw):
    assert _create_loss(**kw) == (tbe.TBE_ERR_INVALID_ARG, None)


@built
def test_create_refuses_what_is_outside_the_limits():
    assert _create_norm(dim=16385) == (tbe.TBE_ERR_UNSUPPORTED, None)
    assert _create_loss(dim=4097) == (tbe.TBE_ERR_UNSUPPORTED, None)


@built
def test_calls_refuse_null_handles():
    lib, bad = tbe.load_library(), tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_layer_norm_create(None, None) == bad
    assert lib.tbe_softmax_loss_create(None, None) == bad
    assert lib.tbe_layer_norm_workspace_bytes(None, 1) == 0
    assert lib.tbe_softmax_loss_workspace_bytes(None, 1, 1, 0) == 0
    assert lib.tbe_layer_norm_forward(None, None, 0, None, 0, None, None, 1, None, None, None, None) == bad
    assert lib.tbe_layer_norm_backward(None, None, 0, None, None, 0, None, 0, None, 1, None, None, None, None, 0,
                                       None) == bad
    assert lib.tbe_softmax_loss_forward(None, None, 0, None, 0, None, 1, 1, 1, None, None, None, 0, None) == bad
    assert lib.tbe_softmax_loss_backward(None, None, 0, None, 0, None, 1, 1, 1, None, None, None, None, None, 0,
                                         None) == bad
    assert lib.tbe_softmax_loss_get_error(None, None) == bad
    lib.tbe_layer_norm_destroy(None)
    lib.tbe_softmax_loss_destroy(None)


@pytest.mark.parametrize("dim", [2 ** 32 + 64, -2 ** 31 - 1])
def test_numbers_outside_int32_are_refused(dim, monkeypatch):
    monkeypatch.setattr(tbe, "load_library", lambda: pytest.fail("reached the library"))
    with pytest.raises(ValueError):
        tbe.tbe_layer_norm_create(dim, torch.float32)
    with pytest.raises(ValueError):
        tbe.tbe_softmax_loss_create(dim, torch.float32)
    with pytest.raises(ValueError):
        tbe.tbe_layer_norm_create(64, torch.int32)
    with pytest.raises(ValueError):
        tbe.tbe_softmax_loss_create(64, torch.float64)
