"""Layer norm on the GPU: rows and batches that the sizes of the other tests do not reach."""

import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe
import rows_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [3, 20, 40, 77, 136, 520, 1100, 4104])
def test_gradients_of_huge_rows_without_spread(dtype, dim):
    """Elements of 2^117 and eps 1e-10: mean * rstd is beyond fp32, xhat is 0, and the gradient is rstd (a - mean(a))."""
    if dim > 2000:
        value, eps = 2.0 ** 114, 1e-12  # (the row's sum stays within fp32; 2^114 * 1e6 does not)
    else:
        value, eps = 2.0 ** 116, 1e-10
    g = torch.Generator(device="cuda").manual_seed(dim)
    h = tbe.tbe_layer_norm_create(dim, dtype, eps)
    x = torch.full((5, dim), value, device="cuda", dtype=dtype)
    w, b, up = (torch.randn((n, dim), generator=g, device="cuda").to(dtype) for n in (1, 1, 5))
    out, total, stats = tbe.tbe_layer_norm_forward(h, x, w[0], b[0])
    assert torch.equal(out, b.expand(5, dim))
    gx, gw, gb = tbe.tbe_layer_norm_backward(h, total, stats, up, w[0])
    a = up.double() * w.double()
    want = (a - a.mean(1, keepdim=True)) * eps ** -0.5
    # the mean's sum: min(D, 80) roundings and three more, of the mean of |a|; the difference's, rstd's (2) and the result's
    n, u = min(dim, 80), ref.UNIT[dtype]
    room = ((n + 3) * ref.F * a.abs().mean(1, keepdim=True) + 4 * ref.F * a.abs()) * eps ** -0.5 \
        + (u + 8 * ref.F) * want.abs()
    assert bool(((gx.double() - want).abs() <= room).all())
    assert not gw.any()
    assert bool(((gb.double() - up.double().sum(0)).abs() <= u * up.double().sum(0).abs() + 8 * ref.F * up.double().abs().sum(0)).all())
