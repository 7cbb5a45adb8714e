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


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim", [(40000, 8), (40011, 24), (30007, 64), (20003, 77), (9001, 512), (6007, 1100),
                                      (3001, 4096)])
def test_in_place_of_many_rows(dtype, rows, dim):
    """Every thread takes many rows in turn, so rows fetched ahead lie beside others that are already overwritten (narrow
    ones in one cache line with them)."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    h = tbe.tbe_layer_norm_create(dim, dtype)
    x, r, grad, up = (torch.randn((rows, dim), generator=g, device="cuda").to(dtype) for _ in range(4))
    w, b = torch.randn((2, dim), generator=g, device="cuda").to(dtype)
    out, total, stats = tbe.tbe_layer_norm_forward(h, x, w, b, r)
    for names in (("out", "total"), ("total", "out")):
        places = dict(zip(names, (x.clone(), r.clone())))
        first, second = places[names[0]], places[names[1]]
        got = tbe.tbe_layer_norm_forward(h, first, w, b, second, **places)
        assert torch.equal(got[0], out) and torch.equal(got[1], total) and torch.equal(got[2], stats), names
    y = x.clone()
    want = tbe.tbe_layer_norm_forward(h, x, w, b)
    assert torch.equal(tbe.tbe_layer_norm_forward(h, y, w, b, out=y)[0], want[0])
    want = tbe.tbe_layer_norm_backward(h, total, stats, grad, w, up)
    for place in ("total", "grad_out", "grad_total"):
        args = dict(total=total, grad_out=grad, grad_total=up)
        args[place] = args[place].clone()
        got = tbe.tbe_layer_norm_backward(h, stats=stats, weight=w, grad_x=args[place], **args)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), place
