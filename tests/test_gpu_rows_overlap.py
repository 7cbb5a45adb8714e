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
