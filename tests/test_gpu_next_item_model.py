"""The example's next-item model: tables, norms, attention and the loss over the
items together, against the same model written out for torch's autograd in 64 bits."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def written_out(model, ids, bags, offsets, targets):
    import history_model

    assert history_model.tbe.TBE_OK == 0
    p = {k: v.to(model.dtype).double().requires_grad_() for k, v in model.params.items()}
    table = model.table.double().requires_grad_()
    events, h, k, d = bags.numel() - 1, model.heads, model.kv_heads, model.head_dim
    rows = torch.nn.functional.embedding_bag(ids, model.table.double(), bags[:-1], mode="sum").requires_grad_()

    def norm(x, i):
        c = x - x.mean(1, keepdim=True)
        return c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["norm_w" + i] + p["norm_b" + i]

    qkv = (norm(rows, "1") @ p["w"]).view(events, h + 2 * k, d)
    starts = history_model.tbe.tbe_relative_buckets(16, 64)
    out = []
    for lo, hi in zip(offsets[:-1].tolist(), offsets[1:].tolist()):
        at = torch.arange(hi - lo, device=ids.device)
        dist = at[:, None] - at[None, :]
        bucket = sum((dist >= s).long() for s in starts).clamp(min=1) - 1
        q, key, v = qkv[lo:hi, :h], qkv[lo:hi, h:h + k], qkv[lo:hi, h + k:]
        s = torch.einsum("ihd,jhd->hij", q, key.repeat_interleave(h // k, 1)) * d ** -0.5
        s = s + p["bias"][bucket].permute(2, 0, 1)
        s = s.masked_fill((dist < 0) | ((dist >= 64) & (at[None, :] >= 2)), float("-inf"))
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v.repeat_interleave(h // k, 1)))
    y = norm(torch.cat(out).flatten(1) @ p["w_out"] + rows, "2")
    keep = targets >= 0
    loss = torch.nn.functional.cross_entropy(y[keep] @ table.t(), targets[keep])
    loss.backward()
    return loss.item(), {**{n: x.grad for n, x in p.items()}, "table": table.grad, "rows": rows.grad}


# 2-norms of errors: fp32 sums of up to 3000 terms drift by 1e-6 to 1e-5 a layer (six layers); 16-bit rounds each of
# about ten tensors on the way by at most 2^-9 (bf16) or 2^-12 (fp16) of it, which the norms and softmaxes pass on
# by factors of one to two, and weights of the matrix products lose as much
@pytest.mark.parametrize("dtype,tolerance", [(torch.float32, 1e-4), (torch.bfloat16, 0.08), (torch.float16, 0.01)])
def test_gradients_of_the_whole_model(dtype, tolerance):
    import history_model

    model = history_model.NextItemModel(items=700, dtype=dtype)
    ids, bags, offsets, _ = history_model.make_histories(40, 700, "cuda", 3)
    targets = history_model.next_items(ids, offsets)
    assert int((targets < 0).sum()) == 40
    scale = float(offsets[-1])
    loss, g = model.gradients(ids, bags, offsets, targets, scale)
    model.check()
    want_loss, want = written_out(model, ids, bags, offsets, targets)
    assert abs(float(loss) - want_loss) < tolerance * want_loss
    assert set(g) == set(want)
    for name, x in want.items():
        err = ((g[name].double() / scale - x).norm() / x.norm()).item()
        assert err < tolerance, (name, err)
    model.close()


def test_the_example_runs():
    import history_model

    losses = history_model.train_next_item(users=20, steps=3, verbose=False)
    assert len(losses) == 3 and all(x == x and x > 0 for x in losses)
