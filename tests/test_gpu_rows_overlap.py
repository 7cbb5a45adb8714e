"""Layer norm and the softmax loss refuse results that lie over each other or over operands that are still read."""

import pytest
import torch

import recommender_sparse_embeddings_gb300 as tbe

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def refused(call, *args, **kw):
    with pytest.raises(tbe.TBEError) as e:
        call(*args, **kw)
    assert e.value.code == tbe.TBE_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 264])
def test_no_rows_leave_a_table_given_as_its_gradient(dtype, d):
    h, table = tbe.tbe_softmax_loss_create(d, dtype), torch.randn((50, d), device="cuda").to(dtype)
    was = table.clone()
    x, targets = table[:0], torch.empty(0, dtype=torch.int64, device="cuda")
    lse = grad = torch.empty(0, device="cuda")
    refused(tbe.tbe_softmax_loss_backward, h, x, table, targets, lse, grad, grad_table=table)
    refused(tbe.tbe_softmax_loss_backward, h, x, table[:40], targets, lse, grad, grad_table=table[10:])
    assert torch.equal(table, was)
    _, gw = tbe.tbe_softmax_loss_backward(h, x, table, targets, lse, grad)
    assert gw.shape == table.shape and not gw.any()
    # no rows and no items: nothing is written wherever the results lie
    tbe.tbe_softmax_loss_backward(h, x, table[:0], targets, lse, grad, grad_x=x, grad_table=table[:0])


def norm(dtype, rows, d, weight=True):
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    h = tbe.tbe_layer_norm_create(d, dtype, weight=weight, bias=weight)
    return h, *(torch.randn((n, d), generator=g, device="cuda").to(dtype) for n in (rows, rows, 1, 1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 77])
def test_norm_results_over_each_other_or_over_operands(dtype, d):
    n = 40
    h, x, r, w, b = norm(dtype, n, d)
    room = torch.full(((2 * n + 8) * d + 64,), 7.0, dtype=dtype, device="cuda")
    was = room.clone()

    def at(first, rows=n):
        return room[first:first + rows * d].view(rows, d)

    def call(x=x, r=r, **kw):
        return tbe.tbe_layer_norm_forward(h, x, kw.pop("w", w)[0], kw.pop("b", b)[0], r, **kw)

    for first in (0, 1, d, (n - 1) * d, n * d - 1):  # out and total: the same, an element, rows apart, the last shared
        refused(call, out=at(0), total=at(first))
        refused(call, out=at(first), total=at(0))
    call(out=at(0), total=at(n * d))
    room.copy_(was)
    for first in (1, d, (n - 1) * d):  # results over other rows of an operand
        for kw in (dict(x=at(0), out=at(first)), dict(x=at(first), out=at(0)), dict(r=at(0), out=at(first)),
                   dict(x=at(0), total=at(first)), dict(r=at(first), total=at(0))):
            refused(call, **kw)
    wide = room[:n * 2 * d].view(n, 2 * d)  # over strided rows, a broadcast one, and the gaps between them
    refused(call, x=wide[:, :d], out=at(0))
    refused(call, r=wide[:, d:], total=at(0))
    refused(call, x=room[:d].expand(n, d), out=at(0))
    refused(call, w=at(3 * d), out=at(0))
    refused(call, b=at(n * d - d, 1), total=at(0))
    stats = room[:4 * n].view(torch.float32)[:2 * n].view(2, n)
    for kw in (dict(out=at(0)), dict(total=at(0)), dict(x=at(0)), dict(r=at(0)), dict(w=at(0, 1))):
        refused(call, stats=stats, **kw)
    assert torch.equal(room, was)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_results_beside_operands(dtype):
    """What shares no byte is taken: a result in a gap between strided rows, behind them, and the same row of one."""
    n, d = 3, 64
    h, x, r, w, b = norm(dtype, n, d)
    want = [t.clone() for t in tbe.tbe_layer_norm_forward(h, x, w[0], b[0], r)]
    wide = torch.zeros((n, 16 * d), dtype=dtype, device="cuda")
    wide[:, :d] = x
    flat = wide.view(-1)
    for first in (d, 12 * d, (2 * 16 + 1) * d):
        got = tbe.tbe_layer_norm_forward(h, wide[:, :d], w[0], b[0], r, out=flat[first:first + n * d].view(n, d))
        assert torch.equal(got[0], want[0]) and torch.equal(wide[:, :d], x)
    one = wide[:1, :d]  # a single row: its stride says nothing
    tbe.tbe_layer_norm_forward(h, one, w[0], b[0], r[:1], out=flat[:d].view(1, d))
    assert torch.equal(one, want[0][:1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 77])
def test_norm_gradients_over_each_other_or_over_operands(dtype, d):
    n = 40
    h, x, g, w, b = norm(dtype, n, d)
    _, total, stats = tbe.tbe_layer_norm_forward(h, x, w[0], b[0])
    want = [t.clone() for t in tbe.tbe_layer_norm_backward(h, total, stats, g, w[0], g)]
    room = torch.full(((2 * n + 8) * d + 64,), 7.0, dtype=dtype, device="cuda")
    was = room.clone()

    def at(first, rows=n):
        return room[first:first + rows * d].view(rows, d)

    def call(total=total, stats=stats, g=g, w=w, u=g, **kw):
        return tbe.tbe_layer_norm_backward(h, total, stats, g, w[0], u, **kw)

    for first in (1, d, (n - 1) * d):
        for name in ("total", "g", "u"):
            refused(call, **{name: at(0)}, grad_x=at(first))
            refused(call, **{name: at(first)}, grad_x=at(0))
    refused(call, g=room[:n * 2 * d].view(n, 2 * d)[:, :d], grad_x=at(0))
    refused(call, u=room[:d].expand(n, d), grad_x=at(0))
    refused(call, w=at(5 * d), grad_x=at(0))
    refused(call, stats=room[:4 * n].view(torch.float32)[:2 * n].view(2, n), grad_x=at(0))
    one = room[:d]
    refused(call, grad_weight=one, grad_bias=one)
    refused(call, grad_weight=one, grad_bias=room[d - 1:2 * d - 1])
    refused(call, grad_x=at(0), grad_weight=room[d * (n - 1) + 3:d * n + 3])
    refused(call, grad_x=at(0), grad_bias=one)
    assert torch.equal(room, was)
    for place in ("total", "g", "u"):  # the same rows in place, the weights' gradients over the weights
        at(0).copy_(total if place == "total" else g)
        ww = w.clone()
        got = call(**{place: at(0)}, w=ww, grad_x=at(0), grad_weight=ww[0], grad_bias=at(n * d, 1)[0])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), place
        assert torch.equal(ww[0], want[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_loss_over_lse_or_over_the_targets(dtype, index):
    n, h = 30, tbe.tbe_softmax_loss_create(48, dtype)
    x, table = torch.randn((n, 48), device="cuda").to(dtype), torch.randn((100, 48), device="cuda").to(dtype)
    targets, room = torch.arange(n, device="cuda").to(index), torch.full((2 * n,), 7.0, device="cuda")
    was = targets.clone()
    for kw in (dict(loss=room[:n], lse=room[:n]), dict(loss=room[:n], lse=room[n - 1:2 * n - 1]),
               dict(loss=targets.view(torch.float32)[:n]), dict(lse=targets.view(torch.float32)[-n:])):
        refused(tbe.tbe_softmax_loss_forward, h, x, table, targets, **kw)
    assert torch.equal(targets, was) and bool((room == 7.0).all())
    tbe.tbe_softmax_loss_forward(h, x, table, targets, loss=room[:n], lse=room[n:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_in_place_without_a_residual_keeps_no_stream(dtype):
    """What the call returns as the kept stream is the stream, or nothing: not the normalised rows in its place."""
    h, x, r, w, b = norm(dtype, 20, 72)
    was = x.clone()
    out, total, stats = tbe.tbe_layer_norm_forward(h, x, w[0], b[0])
    assert total is x and torch.equal(x, was)
    again, total, stats = tbe.tbe_layer_norm_forward(h, x, w[0], b[0], out=x)
    assert total is None and again is x and torch.equal(x, out)
    with pytest.raises(ValueError):
        tbe.tbe_layer_norm_backward(h, total, stats, out, w[0])
    x.copy_(was)
    want = tbe.tbe_layer_norm_forward(h, x, w[0], b[0], r)
    got = tbe.tbe_layer_norm_forward(h, x, w[0], b[0], r, out=x)  # with a residual the stream has a place of its own
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    empty = tbe.tbe_layer_norm_forward(h, x[:0], w[0], b[0])
    assert empty[1] is not None and empty[1].shape == (0, 72)
