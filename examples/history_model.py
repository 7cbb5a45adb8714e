"""A small next-event model over user histories: the table-batched embedding
and the attention operators used together, trained and served.

Each user has a ragged history of events.  An event is a bag of item ids (the
item and its attributes), pooled by ``tbe_forward`` into one row; the rows are
projected to queries, keys and values; attention over the history (newest
``window`` events, first ``sinks`` events, learned bias by distance) gives the
state after each event, which predicts the next event's label.  One training
step runs every gradient through the library: ``tbe_attention_backward`` for
q, k, v and the bias table, ``tbe_backward_sgd`` for the item table.

Serving keeps the keys and values in a paged cache: the histories are appended
once, then each new event is appended and attends to its user's cache.

``NextItemModel`` predicts the next event's item instead: the pooled rows are a
stream that is normalised on its way into attention, attention's output is added
to it, and the normalised sum is scored against the item table itself
(``tbe_softmax_loss_forward``; the table gets the gradients of both its uses).

    python examples/history_model.py [--users 64] [--steps 20] [--next-item]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import recommender_sparse_embeddings_gb300 as tbe  # noqa: E402


class HistoryModel:
    def __init__(self, items=5000, dim=64, heads=4, kv_heads=2, head_dim=32, window=64, sinks=2, buckets=16,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device)

        self.dtype, self.heads, self.kv_heads, self.head_dim = dtype, heads, kv_heads, head_dim
        self.table = weight(items, dim, std=0.5)
        self.bags = tbe.tbe_create([self.table], "sum")
        self.w = weight(dim, (heads + 2 * kv_heads) * head_dim, std=dim ** -0.5)
        self.w_out = weight(heads * head_dim, 1, std=(heads * head_dim) ** -0.5)
        self.bias = weight(buckets, heads, std=0.1)
        self.attention = tbe.tbe_attention_create(heads, kv_heads, head_dim, dtype, window, sinks,
                                                  tbe.tbe_relative_buckets(buckets, window))

    def rows(self, ids, bag_offsets):
        """Pooled rows of the events and their q, k, v (views of one buffer)."""
        events = bag_offsets.numel() - 1
        x = tbe.tbe_forward(self.bags, ids, bag_offsets, events)
        qkv = (x @ self.w).to(self.dtype).view(events, self.heads + 2 * self.kv_heads, self.head_dim)
        h, k = self.heads, self.kv_heads
        return x, qkv[:, :h], qkv[:, h:h + k], qkv[:, h + k:]

    def step(self, ids, bag_offsets, offsets, labels, lr):
        """One training step on a batch of histories; returns the loss."""
        events = bag_offsets.numel() - 1
        x, q, k, v = self.rows(ids, bag_offsets)
        bias = self.bias.to(self.dtype)
        out, lse = tbe.tbe_attention_forward(self.attention, q, k, v, offsets, bias)
        flat = out.view(events, -1).float()
        logit = (flat @ self.w_out)[:, 0]
        loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, labels)
        d_logit = ((torch.sigmoid(logit) - labels) / events)[:, None]
        scale = float(events)  # the 16-bit gradients carry the sum, the updates divide
        d_out = (scale * d_logit @ self.w_out.t()).to(self.dtype).view_as(out)
        gq, gk, gv, gb = tbe.tbe_attention_backward(self.attention, q, k, v, offsets, out, lse, d_out, bias)
        d_qkv = torch.cat([gq, gk, gv], 1).view(events, -1).float() / scale
        d_x = (d_qkv @ self.w.t()).contiguous()
        workspace = tbe.make_workspace(self.bags, ids.numel(), events)
        self.w_out -= lr * flat.t() @ d_logit
        self.w -= lr * x.t() @ d_qkv
        self.bias -= lr * gb.float() / scale
        tbe.tbe_backward_sgd(self.bags, ids, bag_offsets, events, d_x, lr, workspace)
        return float(loss)

    def close(self):
        self.bags.close()
        self.attention.close()


class NextItemModel:
    """One pre-norm attention block over pooled rows, and the loss of the next
    item over the table that the rows come from."""

    def __init__(self, items=5000, dim=64, heads=4, kv_heads=2, head_dim=32, window=64, sinks=2, buckets=16,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def weight(*shape, std, mean=0.0):
            return (torch.randn(shape, generator=g) * std + mean).to(device)

        self.dtype, self.heads, self.kv_heads, self.head_dim = dtype, heads, kv_heads, head_dim
        self.table = weight(items, dim, std=0.3).to(dtype)
        self.bags = tbe.tbe_create([self.table], "sum")
        self.params = {"w": weight(dim, (heads + 2 * kv_heads) * head_dim, std=dim ** -0.5),
                       "w_out": weight(heads * head_dim, dim, std=(heads * head_dim) ** -0.5),
                       "bias": weight(buckets, heads, std=0.1)}
        for i in ("1", "2"):
            self.params |= {"norm_w" + i: weight(dim, std=0.1, mean=1.0), "norm_b" + i: weight(dim, std=0.1)}
        self.attention = tbe.tbe_attention_create(heads, kv_heads, head_dim, dtype, window, sinks,
                                                  tbe.tbe_relative_buckets(buckets, window))
        self.norm = tbe.tbe_layer_norm_create(dim, dtype)
        self.loss = tbe.tbe_softmax_loss_create(dim, dtype)

    def gradients(self, ids, bag_offsets, offsets, targets, scale=1.0):
        """(loss, gradients of the parameters and of the pooled rows) of the mean
        loss over the labelled events, times ``scale``; the table's gradient as a
        table of items is "table", its lookups' come from "rows"."""
        events, p = bag_offsets.numel() - 1, {k: v.to(self.dtype) for k, v in self.params.items()}
        h, k, dt = self.heads, self.kv_heads, self.dtype
        stream = tbe.tbe_forward(self.bags, ids, bag_offsets, events).to(dt)
        y1, _, stats1 = tbe.tbe_layer_norm_forward(self.norm, stream, p["norm_w1"], p["norm_b1"])
        qkv = (y1 @ p["w"]).view(events, h + 2 * k, self.head_dim)
        q, key, v = qkv[:, :h], qkv[:, h:h + k], qkv[:, h + k:]
        out, lse = tbe.tbe_attention_forward(self.attention, q, key, v, offsets, p["bias"])
        flat = out.view(events, -1)
        y2, total, stats2 = tbe.tbe_layer_norm_forward(self.norm, flat @ p["w_out"], p["norm_w2"], p["norm_b2"],
                                                       residual=stream)
        loss, lse2 = tbe.tbe_softmax_loss_forward(self.loss, y2, self.table, targets)
        labelled = (targets >= 0).sum().clamp(min=1)

        up = (scale / labelled.float()).expand(events).contiguous()
        g = {}
        gy2, g["table"] = tbe.tbe_softmax_loss_backward(self.loss, y2, self.table, targets, lse2, up)
        ga, g["norm_w2"], g["norm_b2"] = tbe.tbe_layer_norm_backward(self.norm, total, stats2, gy2, p["norm_w2"])
        g["w_out"] = flat.t() @ ga
        d_out = (ga @ p["w_out"].t()).view_as(out)
        gq, gk, gv, g["bias"] = tbe.tbe_attention_backward(self.attention, q, key, v, offsets, out, lse, d_out, p["bias"])
        d_qkv = torch.cat([gq, gk, gv], 1).view(events, -1)
        g["w"] = y1.t() @ d_qkv
        g["rows"], g["norm_w1"], g["norm_b1"] = tbe.tbe_layer_norm_backward(
            self.norm, stream, stats1, d_qkv @ p["w"].t(), p["norm_w1"], grad_total=ga)
        return loss.sum() / labelled, g

    def step(self, ids, bag_offsets, offsets, targets, lr):
        """One training step on a batch of histories; returns the loss."""
        scale = float(offsets[-1])  # the 16-bit gradients carry the sum, the updates divide
        loss, g = self.gradients(ids, bag_offsets, offsets, targets, scale)
        for name, x in self.params.items():
            x -= lr / scale * g[name].float()
        events = bag_offsets.numel() - 1
        workspace = tbe.make_workspace(self.bags, ids.numel(), events)
        tbe.tbe_backward_sgd(self.bags, ids, bag_offsets, events, g["rows"].float() / scale, lr, workspace)
        self.table -= (lr / scale * g["table"].float()).to(self.dtype)
        return float(loss)

    def check(self):
        codes = (tbe.tbe_get_error(self.bags), tbe.tbe_attention_get_error(self.attention),
                 tbe.tbe_softmax_loss_get_error(self.loss))
        if any(c != tbe.TBE_OK for c in codes):
            raise RuntimeError(f"device error {codes}")

    def close(self):
        for h in (self.bags, self.attention, self.norm, self.loss):
            h.close()


def next_items(ids, offsets):
    """The first id of the event after each one (three ids an event); -1 for a history's last."""
    targets = ids[::3].roll(-1)
    targets[offsets[1:] - 1] = -1
    return targets


def train_next_item(users=64, steps=20, items=500, lr=2.0, verbose=True):
    model = NextItemModel(items=items)
    ids, bags, offsets, _ = make_histories(users, items, "cuda", 1)
    targets = next_items(ids, offsets)
    losses = [model.step(ids, bags, offsets, targets, lr) for _ in range(steps)]
    model.check()
    if verbose:
        print(f"next item: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    model.close()
    return losses


class Cache:
    """A paged cache of a batch of users' keys and values."""

    def __init__(self, model, users, room, page=16, device="cuda"):
        width = (room + page - 1) // page
        shape = (users * width, page, model.kv_heads, model.head_dim)
        self.k = torch.empty(shape, dtype=model.dtype, device=device)
        self.v = torch.empty(shape, dtype=model.dtype, device=device)
        self.table = torch.randperm(users * width, device=device).to(torch.int32).view(users, width)
        self.lengths = torch.zeros(users, dtype=torch.int32, device=device)

    def append(self, model, k, v, offsets):
        tbe.tbe_attention_append(model.attention, k, v, offsets, self.lengths, self.k, self.v, self.table)
        self.lengths += (offsets[1:] - offsets[:-1]).to(torch.int32)


def make_histories(users, items, device, seed):
    """Ragged histories of 1 to 100 events, three ids an event; an event's label
    says whether its first id is even (learnable from the item table)."""
    g = torch.Generator().manual_seed(seed)
    lengths = torch.randint(1, 101, (users,), generator=g)
    events = int(lengths.sum())
    ids = torch.randint(0, items, (3 * events,), generator=g)
    labels = (ids[::3] % 2).float()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    return ids.to(device), torch.arange(0, 3 * events + 1, 3).to(device), offsets.to(device), labels.to(device)


def main(users=64, steps=20, items=500, lr=2.0, verbose=True):
    model = HistoryModel(items=items)
    ids, bags, offsets, labels = make_histories(users, items, "cuda", 1)
    losses = [model.step(ids, bags, offsets, labels, lr) for _ in range(steps)]
    if verbose:
        print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps over {offsets[-1].item()} events")

    # serving: all but each user's last event are cached, the last one arrives
    _, q, k, v = model.rows(ids, bags)
    bias = model.bias.to(model.dtype)
    want, _ = tbe.tbe_attention_forward(model.attention, q, k, v, offsets, bias)
    last = offsets[1:] - 1
    old = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    old[last] = False
    cache = Cache(model, users, 128)
    cache.append(model, k[old], v[old], offsets - torch.arange(users + 1, device="cuda"))
    cache.append(model, k[last], v[last], torch.arange(users + 1, device="cuda"))
    got = tbe.tbe_attention_decode(model.attention, q[last], cache.k, cache.v, cache.table, cache.lengths, bias)
    error = (got.float() - want[last].float()).abs().max().item()
    for h, check in ((model.bags, tbe.tbe_get_error), (model.attention, tbe.tbe_attention_get_error)):
        if check(h) != tbe.TBE_OK:
            raise RuntimeError("device error")
    if verbose:
        print(f"new events served from the cache: largest difference to the whole histories' pass {error:.2e}")
    model.close()
    return losses, error


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--users", type=int, default=64)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--next-item", action="store_true", help="train the next item's loss over the item table")
    a = p.parse_args()
    if a.next_item:
        train_next_item(a.users, a.steps)
    else:
        main(a.users, a.steps)
